// heads_host.cuh -- host side of strided operands: which loads apply, tensor maps.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "heads.cuh"
#include "host_common.cuh"

namespace ssscan {
namespace {

// 16-byte loads: data, every stride and the row itself whole units.
bool la_vec(const LaTensor& x, int d, int es) {
  const int64_t n = 16 / es;
  return aligned(x.ptr, 16) && x.sb % n == 0 && x.st % n == 0 && x.sh % n == 0 && d % n == 0;
}

// cuTensorMapEncodeTiled, looked up once through the runtime (no link-time libcuda).
PFN_cuTensorMapEncodeTiled_v12000 la_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
  }();
  return fn;
}

// Blocks of `rows` tokens x 64 columns of one head, 128-byte swizzle, zeros out of bounds.
bool la_map(CUtensorMap* m, const LaTensor& x, int64_t batch, int64_t seqlen, int heads, int d, int rows) {
  const auto enc = la_map_encoder();
  if (!enc) return false;
  const int64_t ext[4] = {d, seqlen, heads, batch}, str[4] = {1, x.st, x.sh, x.sb};
  cuuint64_t dims[4], strides[3];
  for (int i = 0; i < 4; ++i) {
    dims[i] = (cuuint64_t)ext[i];
    if (i == 0) continue;
    // an axis of one has any stride; a broadcast or reversed one is left to plain loads
    const int64_t bytes = ext[i] == 1 ? 16 : str[i] * 2;
    if (bytes <= 0 || bytes % 16 != 0 || bytes >= ((int64_t)1 << 40)) return false;
    strides[i - 1] = (cuuint64_t)bytes;
  }
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, step[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.ptr), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace ssscan

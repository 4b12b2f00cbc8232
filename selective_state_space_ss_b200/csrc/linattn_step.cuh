// linattn_step.cuh -- one token of the decayed linear attention:
//
//   S <- exp(g) S + k v^T,    o = scale * S^T q     for every (row, head).
//
// Bound by memory: the fp32 state is read and written once, 8 bytes for 4
// operations.  A block takes 32 value columns of one head's state with all their
// keys, so the sum over keys stays in the block, and holds its slice in registers
// between the read and the write; a small batch still gives heads x dv / 32 blocks
// a row.  Batch 128, 40 heads of 128 x 128 (674 MB): 102 us, 6.6 TB/s, the copy rate; a
// batch of 4 with 24 heads of 64 x 64 takes 2.5 us on the device.  By slots every block
// looks through the earlier rows' for its own: 4% there, 15% at batch 128 with 24 heads of
// 64 x 64 (19 -> 22 us), 36% at 4096 rows with 8 (195 -> 266 us).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "linattn_pass.cuh"

namespace ssscan {

constexpr int kLaStepThreads = 256;
constexpr int kLaStepCols = 32;  // value columns of a block

struct LaStepArgs {
  LaTensor q, k, v, g;  // token strides unused
  float* state;
  int64_t num_slots;
  const int* slots;
  void* out;
  int batch, heads, dk, dv;
  float scale;
};

// The state row of batch row b, or -1 for padding: outside the pool, or a slot that
// an earlier row has.  By the whole block.
__device__ __forceinline__ int64_t la_step_slot(const LaStepArgs& a, int b) {
  if (!a.slots) return b;
  const int slot = a.slots[b];
  bool skip = slot < 0 || slot >= a.num_slots;
  for (int i = threadIdx.x; i < b; i += blockDim.x) skip |= a.slots[i] == slot;
  return __syncthreads_or(skip) ? -1 : slot;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kLaStepThreads) linattn_step_kernel(const __grid_constant__ LaStepArgs a) {
  constexpr int TPR = kLaStepCols / VEC;         // threads of a key's row
  constexpr int ROWS = kLaStepThreads / TPR;     // keys at once
  constexpr int IT = 128 / ROWS;
  __shared__ float sq[128], sk[128];
  __shared__ float part[ROWS][kLaStepCols + 1];
  const int tid = threadIdx.x, b = blockIdx.y;
  const int tiles = (a.dv + kLaStepCols - 1) / kLaStepCols;
  const int h = blockIdx.x / tiles, v0 = (blockIdx.x % tiles) * kLaStepCols;
  const int64_t slot = la_step_slot(a, b);
  if (slot < 0) return;
  const int c = (tid % TPR) * VEC, r0 = tid / TPR;
  const bool mine = v0 + c < a.dv;
  float* st = a.state + ((slot * a.heads + h) * a.dk) * a.dv + v0 + c;
  const int64_t all = a.num_slots * a.heads * a.dk * a.dv;
  float x[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = r0 + i * ROWS;
    if (mine && r < a.dk && in_range(st + (int64_t)r * a.dv - a.state, VEC, all)) {
      if constexpr (VEC == 4) {
        const float4 y = __ldcs(reinterpret_cast<const float4*>(st + (int64_t)r * a.dv));
        x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
      } else {
        x[i][0] = st[(int64_t)r * a.dv];
      }
    }
  }
  if (tid < a.dk) {
    const char* qk[2] = {la_row(a.q, b, 0, h, sizeof(T)) + tid * sizeof(T), la_row(a.k, b, 0, h, sizeof(T)) + tid * sizeof(T)};
    if (la_inside(a.q, qk[0], 1, sizeof(T))) sq[tid] = to_f32(*reinterpret_cast<const T*>(qk[0]));
    if (la_inside(a.k, qk[1], 1, sizeof(T))) sk[tid] = to_f32(*reinterpret_cast<const T*>(qk[1]));
  }
  const char* g = la_row(a.g, b, 0, h, sizeof(T));
  const float decay = la_inside(a.g, g, 1, sizeof(T)) ? expf(to_f32(*reinterpret_cast<const T*>(g))) : 0.f;
  float vv[VEC], o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const char* v = la_row(a.v, b, 0, h, sizeof(T)) + (v0 + c + e) * sizeof(T);
    vv[e] = mine && la_inside(a.v, v, 1, sizeof(T)) ? to_f32(*reinterpret_cast<const T*>(v)) : 0.f;
    o[e] = 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = r0 + i * ROWS;
    if (mine && r < a.dk) {
      const float q = sq[r], k = sk[r];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[i][e] = fmaf(x[i][e], decay, k * vv[e]);
        o[e] = fmaf(q, x[i][e], o[e]);
      }
      if (!in_range(st + (int64_t)r * a.dv - a.state, VEC, all)) continue;
      if constexpr (VEC == 4)
        __stcs(reinterpret_cast<float4*>(st + (int64_t)r * a.dv), make_float4(x[i][0], x[i][1], x[i][2], x[i][3]));
      else
        st[(int64_t)r * a.dv] = x[i][0];
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) part[r0][c + e] = o[e];
  __syncthreads();
  if (tid < kLaStepCols && v0 + tid < a.dv) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s += part[i][tid];
    const int64_t at = ((int64_t)b * a.heads + h) * a.dv + v0 + tid;
    if (!in_range(at, (int64_t)a.batch * a.heads * a.dv)) return;
    if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(s * a.scale);
    else static_cast<float*>(a.out)[at] = s * a.scale;
  }
}

}  // namespace ssscan

// ss_winattn.cu -- the exported functions of include/ss_winattn.h: attention over a window
// with sinks (forward, backward, the newest tokens over a paged cache), the cache's
// appending and the rotation of positions.  libssscan.so's third translation unit; its
// kernels report through an error word of its own, which ss_last_device_error reads too.
#include <cuda_runtime.h>

#include <cstdint>

#include "ss_scan_debug.h"
#include "ss_winattn.h"
#include "winattn_host.cuh"

using namespace ssscan;

namespace ssscan {

// This unit's error word of the current device, read and cleared; false if CUDA failed.
bool take_winattn_error_word(unsigned int* word) {
  if (cudaMemcpyFromSymbol(word, g_error_word, sizeof *word) != cudaSuccess) return false;
  if (*word == 0) return true;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_error_word, &zero, sizeof zero) == cudaSuccess;
}

// ss_debug_inject's settings of this unit.
void set_winattn_debug(int what, long long value) {
  g_dbg_wa_skip_load.store(what == SS_DEBUG_WINATTN_SKIP_LOAD ? value : -1);
}

}  // namespace ssscan

extern "C" {

ss_status ss_winattn_fwd(const ss_heads* q, const ss_heads* k, const ss_heads* v, int64_t window, int64_t sinks,
                         float scale, const int32_t* lengths, void* o_out, float* lse_out, int64_t batch,
                         int64_t seqlen, int heads, int kv_heads, int d, ss_dtype in_dtype, cudaStream_t stream) {
  const WaShape s{batch, seqlen, heads, kv_heads, d, in_dtype, window, sinks};
  return winattn_fwd_impl(q, k, v, scale, lengths, o_out, lse_out, s, stream);
}

ss_status ss_winattn_bwd(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* o, const float* lse,
                         const ss_heads* d_o, int64_t window, int64_t sinks, float scale, const int32_t* lengths,
                         void* dq, void* dk_out, void* dv_out, int64_t batch, int64_t seqlen, int heads, int kv_heads,
                         int d, ss_dtype in_dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const WaShape s{batch, seqlen, heads, kv_heads, d, in_dtype, window, sinks};
  return winattn_bwd_impl(q, k, v, o, lse, d_o, scale, lengths, dq, dk_out, dv_out, s, workspace, workspace_bytes,
                          stream);
}

size_t ss_winattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int kv_heads, int d, int64_t window,
                                      int64_t sinks, ss_dtype in_dtype) {
  return winattn_bwd_bytes(WaShape{batch, seqlen, heads, kv_heads, d, in_dtype, window, sinks});
}

ss_status ss_winattn_step(const ss_heads* q, const ss_pages* pages, const int32_t* lengths, int64_t window,
                          int64_t sinks, float scale, void* o_out, int64_t batch, int64_t tokens, int heads,
                          int kv_heads, int d, ss_dtype in_dtype, cudaStream_t stream) {
  const WaShape s{batch, tokens, heads, kv_heads, d, in_dtype, window, sinks};
  return winattn_step_impl(q, pages, lengths, scale, o_out, s, stream);
}

ss_status ss_kv_append(const ss_heads* k, const ss_heads* v, const ss_heads* q, const ss_pages* pages,
                       const int32_t* starts, const int32_t* counts, const ss_rotation* rotation, void* q_out,
                       void* k_out, int64_t batch, int64_t tokens, int heads, int kv_heads, int d, ss_dtype in_dtype,
                       cudaStream_t stream) {
  if (!pages || !k || !v) return SS_ERR_INVALID_ARG;
  const WaShape s{batch, tokens, q ? heads : kv_heads, kv_heads, d, in_dtype, 1, 0};
  return rotate_impl(k, v, q, pages, starts, counts, rotation, 0, q_out, k_out, s, stream);
}

ss_status ss_rotate(const ss_heads* q, const ss_heads* k, const int32_t* starts, const int32_t* counts,
                    const ss_rotation* rotation, int inverse, void* q_out, void* k_out, int64_t batch, int64_t tokens,
                    int heads, int kv_heads, int d, ss_dtype in_dtype, cudaStream_t stream) {
  if (!q) return SS_ERR_INVALID_ARG;
  const WaShape s{batch, tokens, heads, k ? kv_heads : heads, d, in_dtype, 1, 0};
  return rotate_impl(k, nullptr, q, nullptr, starts, counts, rotation, inverse, q_out, k_out, s, stream);
}

}  // extern "C"

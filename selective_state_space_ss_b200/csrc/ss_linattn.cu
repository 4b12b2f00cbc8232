// ss_linattn.cu -- the exported functions of include/ss_linattn.h: the linear
// attention with a decay per head (forward, backward, single tokens) and the 8-bit
// state pool.  libssscan.so's second translation unit; its kernels report through
// an error word of its own, which ss_last_device_error reads along with the other.
#include <cuda_runtime.h>

#include <cstdint>

#include "ss_linattn.h"
#include "ss_scan_debug.h"
#include "linattn_host.cuh"

using namespace ssscan;

namespace ssscan {

// This unit's error word of the current device, read and cleared; false if CUDA failed.
bool take_linattn_error_word(unsigned int* word) {
  if (cudaMemcpyFromSymbol(word, g_error_word, sizeof *word) != cudaSuccess) return false;
  if (*word == 0) return true;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_error_word, &zero, sizeof zero) == cudaSuccess;
}

// ss_debug_inject's settings of this unit.
void set_linattn_debug(int what, long long value) {
  if (what == SS_DEBUG_LINATTN_SPIN_LIMIT) g_dbg_la_spin_limit.store(value);
  if (what == SS_DEBUG_LINATTN_SKIP_PUBLISH) g_dbg_la_skip_publish.store(value);
  if (what == SS_DEBUG_LINATTN_SKIP_LOAD) g_dbg_la_skip_load.store(value);
  if (what == SS_DEBUG_CLEAR) {
    g_dbg_la_spin_limit.store(0);
    g_dbg_la_skip_publish.store(-1);
    g_dbg_la_skip_load.store(-1);
  }
}

}  // namespace ssscan

extern "C" {

ss_status ss_linattn_fwd(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* log_decay,
                         float scale, const float* initial_state, const int32_t* lengths, void* o_out,
                         float* last_state_out, int64_t batch, int64_t seqlen, int heads, int qk_heads, int dk,
                         int dv, ss_dtype in_dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const LaShape s{batch, seqlen, heads, qk_heads, dk, dv, in_dtype == SS_BF16};
  return linattn_fwd_impl(q, k, v, log_decay, scale, initial_state, lengths, o_out, last_state_out, s, in_dtype,
                          workspace, workspace_bytes, stream);
}

size_t ss_linattn_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int qk_heads, int dk, int dv,
                                  ss_dtype in_dtype) {
  const LaShape s{batch, seqlen, heads, qk_heads, dk, dv, in_dtype == SS_BF16};
  if (la_check_shape(s, in_dtype) != SS_OK) return (size_t)-1;
  return la_seg_bytes(s, la_plan(s));
}

ss_status ss_linattn_bwd(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* log_decay,
                         const ss_heads* d_o, float scale, const float* initial_state, const float* dlast_state,
                         const int32_t* lengths, void* dq, void* dk_out, void* dv_out, void* dlog_decay,
                         float* dinitial_state, int64_t batch, int64_t seqlen, int heads, int qk_heads, int dk,
                         int dv, ss_dtype in_dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const LaShape s{batch, seqlen, heads, qk_heads, dk, dv, in_dtype == SS_BF16};
  return linattn_bwd_impl(q, k, v, log_decay, d_o, scale, initial_state, dlast_state, lengths, dq, dk_out, dv_out,
                          dlog_decay, dinitial_state, s, in_dtype, workspace, workspace_bytes, stream);
}

size_t ss_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads, int qk_heads, int dk, int dv,
                                      ss_dtype in_dtype) {
  const LaShape s{batch, seqlen, heads, qk_heads, dk, dv, in_dtype == SS_BF16};
  if (la_check_bwd_shape(s, in_dtype) != SS_OK) return (size_t)-1;
  return la_bwd_ws(s, la_plan(s)).bytes;
}

ss_status ss_linattn_step(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* log_decay,
                          float scale, float* state, int64_t num_slots, const int32_t* slots, void* o_out,
                          int64_t batch, int heads, int qk_heads, int dk, int dv, ss_dtype in_dtype,
                          cudaStream_t stream) {
  const LaShape s{batch, 1, heads, qk_heads, dk, dv, in_dtype == SS_BF16};
  return linattn_step_impl(q, k, v, log_decay, scale, state, num_slots, slots, o_out, s, in_dtype, stream);
}

ss_status ss_state_store8(const float* state, int8_t* codes, float* scales, int64_t num_slots, const int32_t* slots,
                          int64_t batch, int64_t rows, int width, cudaStream_t stream) {
  const ss_status st = pool_check(state, codes, scales, num_slots, slots, batch, rows, width);
  if (st != SS_OK) return st;
  return state_store8_impl(PoolArgs{const_cast<float*>(state), codes, scales, num_slots, slots, batch, rows, width},
                           stream);
}

ss_status ss_state_load8(const int8_t* codes, const float* scales, int64_t num_slots, const int32_t* slots,
                         float* state_out, int64_t batch, int64_t rows, int width, cudaStream_t stream) {
  const ss_status st = pool_check(state_out, codes, scales, num_slots, slots, batch, rows, width);
  if (st != SS_OK) return st;
  return state_load8_impl(PoolArgs{state_out, const_cast<int8_t*>(codes), const_cast<float*>(scales), num_slots,
                                   slots, batch, rows, width},
                          stream);
}

}  // extern "C"

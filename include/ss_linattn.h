/*
 * ss_linattn.h -- C ABI of libssscan.so: linear attention with one decay per
 * head, and the 8-bit pool for the states of sequences that wait.
 *
 * The selective scan of ss_scan.h decays every channel and state on its own.
 * With one decay for a whole head the same recurrence is a linear attention,
 * whose state is a dk x dv matrix (keys and queries in the place of B and C,
 * shared by a head's channels; values in the place of Delta * u):
 *
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = scale * S_t^T q_t
 *
 * for every batch row and head, S_0 = initial_state or zero.
 *
 * The conventions of ss_scan.h hold: device pointers, caller-owned; nothing is
 * allocated, nothing synchronised; calls are asynchronous on `stream` and may be
 * captured into a CUDA graph; the stream belongs to the current device, and so do
 * the buffers; arguments are checked on the host before any launch and a rejected
 * call launches nothing.  Values must be finite (fp32: below 3.38e38): a NaN or an
 * infinity in q, k or v spreads over the heads of its batch row that read it, from
 * the 64-token chunk that holds it on (gradients: to the chunks before it as well),
 * the chunk's earlier tokens included, and stays out of every other head and row.
 * fp32 inputs are multiplied as three bf16 parts, so below about 1e-33 their last
 * bits are lost.  Outputs must not overlap inputs or one another, but where it says
 * so.  A kernel whose waits give up (ss_last_device_error: SS_ERR_TIMEOUT) leaves
 * its outputs unspecified.
 */
#ifndef SS_LINATTN_H_
#define SS_LINATTN_H_

#include "ss_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A [batch, seqlen, heads, d] tensor whose last axis is contiguous; strides in
 * elements (a slice of a projection's output needs no copy; stride 0 repeats).
 * The log decays are [batch, seqlen, heads] with the same three strides: a decay
 * that is constant over time has token_stride 0.  In the single-token step the
 * token stride is not read.
 */
typedef struct {
  const void* data;
  int64_t batch_stride, token_stride, head_stride;
} ss_heads;

/*
 * ss_linattn_fwd -- a whole prompt.
 *
 *  q, k          [batch, seqlen, qk_heads, dk] in_dtype; head h of the heads
 *                reads head h / (heads / qk_heads)
 *  v             [batch, seqlen, heads, dv]    in_dtype
 *  log_decay     [batch, seqlen, heads]        in_dtype: g, normally <= 0; minus
 *                infinity forgets all before its token; a g > 0 grows the state
 *                and is the caller's to keep in range
 *  scale         multiplies the outputs (dk^-1/2, or 1)
 *  initial_state [batch, heads, dk, dv] float32, nullable (zero)
 *  lengths       [batch] int32, nullable: row b has lengths[b] tokens, taken into
 *                0 .. seqlen.  Nothing behind them is read, o_out keeps what it
 *                holds there, and last_state is the state after the last of them
 *                (the initial state for none)
 *  o_out         [batch, seqlen, heads, dv] in_dtype, contiguous.  Unlike the
 *                scan's y, which its gate and sums leave in fp32, it goes on as
 *                it is to a matrix product, and is rounded once, at the end
 *  last_state_out[batch, heads, dk, dv] float32, nullable; it may be the buffer of
 *                initial_state (then advanced in place); no other overlap
 *  1 <= dk, dv <= 128 (others: SS_ERR_UNSUPPORTED); heads a multiple of qk_heads and
 *                at most 65536, batch * heads at most 2^24, seqlen below 2^31 - 1024
 *  workspace     ss_linattn_workspace_bytes(...) bytes, 256-byte aligned (null
 *                when 0): states of the segments that a long sequence with few
 *                heads is cut into, or those that CTAs hand on where there are more
 *                heads than SMs.  Contents on entry do not matter; calls in
 *                flight at once, replays of captured ones among them, must not
 *                share one
 *
 * Any element alignment; 16-byte aligned data and strides take 16-byte loads.
 */
ss_status ss_linattn_fwd(const ss_heads* q, const ss_heads* k, const ss_heads* v,
                         const ss_heads* log_decay, float scale,
                         const float* initial_state, const int32_t* lengths,
                         void* o_out, float* last_state_out, int64_t batch,
                         int64_t seqlen, int heads, int qk_heads, int dk, int dv,
                         ss_dtype in_dtype, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace ss_linattn_fwd needs on the current device; (size_t)-1 for
 * sizes that it would reject. */
size_t ss_linattn_workspace_bytes(int64_t batch, int64_t seqlen, int heads,
                                  int qk_heads, int dk, int dv, ss_dtype in_dtype);

/*
 * ss_linattn_bwd -- the gradients of ss_linattn_fwd for an upstream gradient
 * d_o [batch, seqlen, heads, dv] (in_dtype, strided) of o and, nullable,
 * dlast_state [batch, heads, dk, dv] float32 of the last state.  No state is kept
 * from the forward; with R_t the gradient of S_t,
 *
 *   R_t  = scale q_t do_t^T + exp(g_{t+1}) R_{t+1}
 *   dq_t = scale S_t do_t (summed over the heads that share it)
 *   dk_t = R_t v_t        (summed over the heads that share it)
 *   dv_t = R_t^T k_t
 *   dg_t = exp(g_t) <R_t, S_{t-1}>
 *   dinitial_state = exp(g_1) R_1
 *
 * dq, dk [batch, seqlen, qk_heads, dk], dv_out [batch, seqlen, heads, dv],
 * dlog_decay [batch, seqlen, heads]: in_dtype, contiguous, required; as in the
 * forward nothing is written behind a row's length.  dinitial_state [batch, heads,
 * dk, dv] float32, nullable; it may be the buffer of dlast_state.  (A decay that was
 * broadcast over time gets its gradient token by token.)  dg_t is a sum of terms that
 * each hold exp(g_t), none of which cancels another's larger part: it is good relative
 * to their size, however much the decay leaves, and exactly zero where that is nothing
 * (minus infinity) and at t = 1 without an initial state.  Sums are in a fixed
 * order: the same call gives the same bits.  workspace:
 * ss_linattn_bwd_workspace_bytes(...) bytes, 256-byte aligned, most of it a state (dk
 * and dv made up to 64 or 128, float32) for every 64 tokens of every head.
 */
ss_status ss_linattn_bwd(const ss_heads* q, const ss_heads* k, const ss_heads* v,
                         const ss_heads* log_decay, const ss_heads* d_o, float scale,
                         const float* initial_state, const float* dlast_state,
                         const int32_t* lengths, void* dq, void* dk_out, void* dv_out,
                         void* dlog_decay, float* dinitial_state, int64_t batch,
                         int64_t seqlen, int heads, int qk_heads, int dk, int dv,
                         ss_dtype in_dtype, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream);

size_t ss_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int heads,
                                      int qk_heads, int dk, int dv, ss_dtype in_dtype);

/*
 * ss_linattn_step -- one token for every sequence, its state advanced in place.
 *
 *  state  [num_slots, heads, dk, dv] float32
 *  slots  [batch] int32, nullable: row b's state is state[slots[b]].  A slot
 *         outside 0 .. num_slots-1 marks a row of padding: nothing is read or
 *         written for it, o_out included.  Of rows with the same slot the first
 *         one is taken and the others are padding.  Null: row b's state is
 *         state[b], and num_slots is at least batch
 *  q, k [batch, qk_heads, dk], v [batch, heads, dv], log_decay [batch, heads]
 *         in_dtype, with the strides of ss_heads; o_out [batch, heads, dv]
 *         in_dtype, contiguous
 *
 * Sizes as ss_linattn_fwd, and batch <= 65535.  No workspace.
 */
ss_status ss_linattn_step(const ss_heads* q, const ss_heads* k, const ss_heads* v,
                          const ss_heads* log_decay, float scale, float* state,
                          int64_t num_slots, const int32_t* slots, void* o_out,
                          int64_t batch, int heads, int qk_heads, int dk, int dv,
                          ss_dtype in_dtype, cudaStream_t stream);

/*
 * ss_state_store8 / ss_state_load8 -- the states of sequences that wait (a dialogue
 * between its turns, a prefix that many prompts share), in 8 bits: each row of
 * `width` values (the last axis of the scan's [batch, dim, dstate] or of the
 * attention's [batch, heads, dk, dv]) as steps of a scale of its own,
 *
 *   scale = max |x| * (1 / 127) (float32),    code = x / scale to the nearest, ties to even
 *
 * and back as code * scale.  The code is the nearest to the quotient as it is, not
 * as fp32 rounds it, so a value read back is off by at most half a scale.
 *
 *  state  [batch, rows, width] float32, contiguous
 *  codes  [num_slots, rows, width] int8, scales [num_slots, rows] float32
 *  slots  [batch] int32, nullable (row b uses slot b, and num_slots is at least
 *         batch).  A slot outside 0 .. num_slots-1: the store leaves that sequence
 *         out, the load gives it a zero state (one that starts afresh).  Of
 *         sequences stored to the same slot the last one is kept; loads may share
 *
 * A row of zeros, or whose scale is below the smallest normal float32, is stored as
 * zeros; a row that holds a NaN or an infinity gets a NaN scale and reads back as
 * NaN.  1 <= width <= 1024 (others: SS_ERR_UNSUPPORTED), batch <= 65535,
 * rows * width < 2^31.  Any element alignment; 16-byte aligned state and codes and a
 * width that is a multiple of 4 take vector accesses.
 */
ss_status ss_state_store8(const float* state, int8_t* codes, float* scales,
                          int64_t num_slots, const int32_t* slots, int64_t batch,
                          int64_t rows, int width, cudaStream_t stream);
ss_status ss_state_load8(const int8_t* codes, const float* scales, int64_t num_slots,
                         const int32_t* slots, float* state_out, int64_t batch,
                         int64_t rows, int width, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SS_LINATTN_H_ */

// linattn_host.cuh -- host side of the linear attention: the cut into segments,
// workspaces, launches and the argument checks
// (host code of libssscan.so's second translation unit, ss_linattn.cu)
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "ss_linattn.h"
#include "host_common.cuh"
#include "linattn_decay_grad.cuh"
#include "linattn_pass.cuh"
#include "linattn_step.cuh"
#include "state_pool.cuh"

namespace ssscan {
namespace {

struct LaShape {
  int64_t batch, seqlen;
  int heads, qk_heads, dk, dv;
  bool bf16;
  int64_t bh() const { return batch * heads; }
  int64_t per_state() const { return (int64_t)dk * dv; }
  int es() const { return bf16 ? 2 : 4; }
};

ss_status la_check_shape(const LaShape& s, int in_dtype) {
  if (s.batch < 1 || s.seqlen < 1 || s.heads < 1 || s.qk_heads < 1 || s.dk < 1 || s.dv < 1) return SS_ERR_INVALID_ARG;
  if (s.heads % s.qk_heads != 0) return SS_ERR_INVALID_ARG;
  if (s.seqlen > INT_MAX - 1024 || s.batch > INT_MAX || s.heads > 65536 || s.batch * s.heads > (1 << 24))
    return SS_ERR_INVALID_ARG;
  if (s.dk > 128 || s.dv > 128) return SS_ERR_UNSUPPORTED;
  if (in_dtype != SS_F32 && in_dtype != SS_BF16) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}

int la_chunks(const LaShape& s) { return (int)((s.seqlen + kLaChunk - 1) / kLaChunk); }

bool la_check_heads(const ss_heads* x, int es) { return x && x->data && aligned(x->data, es); }

// `heads` heads of d values as the pass has them, every `share` of them one of the tensor's.
LaTensor la_tensor(const ss_heads& x, const LaShape& s, int share, int d) {
  LaTensor t{x.data, x.batch_stride, x.token_stride, x.head_stride, share};
#ifdef SS_BOUNDS_CHECK
  int64_t hi = d - 1;
  const int64_t ends[3] = {(s.batch - 1) * t.sb, (s.seqlen - 1) * t.st, (s.heads / share - 1) * t.sh};
  for (int64_t e : ends) (e < 0 ? t.lo : hi) += e;
  t.n = hi - t.lo + 1;
#endif
  return t;
}

// 16-byte loads: data, every stride and the row itself whole units.
bool la_vec(const LaTensor& x, int d, int es) {
  const int64_t n = 16 / es;
  return aligned(x.ptr, 16) && x.sb % n == 0 && x.st % n == 0 && x.sh % n == 0 && d % n == 0;
}

struct LaSegs {
  int nseg, chunks;  // segments of a head, and chunks of each
  int workers;       // > 0 (nseg 1): CTAs that share all chunks evenly
};

// How a pass is cut.  One CTA fits on an SM.  Uncut, batch x heads CTAs take all
// chunks of a head each.  With more heads than SMs a last wave that is not full is
// avoided by workers, one an SM, with an equal share of the chunks; each hands at
// most one state on.  With fewer, a head is cut into s segments: a first launch forms
// the states of s - 1 of them (no queries, scores or outputs: 0.53 to 0.67 of a chunk's
// time, 0.98 us of 1.62 with 64 x 64 bf16 heads, 1.26 of 2.34 with 128 x 128, 4.5 of 7.5
// and 8.8 of 15.4 in fp32), a second joins them and a third runs all segments at once.
// A CTA costs 7 to 13 us to start, the two extra launches about as much: in units of a
// chunk's time 4 (bf16) or 1.3 (fp32).
LaSegs la_plan(const LaShape& s) {
  const int64_t chunks = (s.seqlen + kLaChunk - 1) / kLaChunk, bh = s.bh();
  const int64_t slots = device_sms() > 0 ? device_sms() : 148;
  const double start = s.bf16 ? 4.0 : 1.3, extra = start;
  if (bh > slots) {
    const int64_t waves = (bh + slots - 1) / slots;
    const double share = (double)bh * chunks / slots;
    if (waves * (chunks + start) > share + 2 * start) return LaSegs{1, (int)chunks, (int)slots};
    return LaSegs{1, (int)chunks, 0};
  }
  double best = 0;
  int64_t at = 1;
  for (int64_t n = 1; n <= 64 && n <= chunks; ++n) {
    const int64_t per = (chunks + n - 1) / n;
    if ((chunks + per - 1) / per != n) continue;
    double cost = (double)((bh * n + slots - 1) / slots) * (per + start);
    if (n > 1) cost += (double)((bh * (n - 1) + slots - 1) / slots) * (0.6 * per + start) + extra;
    if (n == 1 || cost < best) best = cost, at = n;
  }
  return LaSegs{(int)at, (int)((chunks + at - 1) / at), 0};
}

struct LaSeg {  // a workspace's share for segments or workers
  float* states = nullptr;
  double* decay = nullptr;
  float* carry = nullptr;
  unsigned* flags = nullptr;
};
size_t la_carry_bytes(const LaShape& s, const LaSegs& g) {
  // sixteen back warps' states, for keys or (in a gradient) values up to 64 or 128 wide
  return align256((size_t)g.workers * 128 * (s.dk <= 64 && s.dv <= 64 ? 64 : 128) * 4);
}
size_t la_seg_bytes(const LaShape& s, const LaSegs& g) {
  if (g.workers > 0) return la_carry_bytes(s, g) + align256((1 + (size_t)g.workers * 16) * 4);
  if (g.nseg <= 1) return 0;
  return align256((size_t)s.bh() * g.nseg * s.per_state() * 4) + align256((size_t)s.bh() * g.nseg * 8);
}
LaSeg la_seg_at(char* ws, const LaShape& s, const LaSegs& g) {
  LaSeg r;
  if (g.workers > 0) {
    r.carry = reinterpret_cast<float*>(ws);
    r.flags = reinterpret_cast<unsigned*>(ws + la_carry_bytes(s, g));
  } else if (g.nseg > 1) {
    r.states = reinterpret_cast<float*>(ws);
    r.decay = reinterpret_cast<double*>(ws + align256((size_t)s.bh() * g.nseg * s.per_state() * 4));
  }
  return r;
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

// Blocks of 64 tokens x 64 columns of one head, 128-byte swizzle, zeros out of bounds.
bool la_map(CUtensorMap* m, const LaTensor& x, int64_t batch, int64_t seqlen, int heads, int d) {
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
  const cuuint32_t box[4] = {64, kLaChunk, 1, 1}, step[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.ptr), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int KD, int VD, LaMode MODE, bool FAST>
ss_status la_launch_as(const LaPassArgs& a, const LaMaps& maps, cudaStream_t stream) {
  using CF = LaCfg<T, KD, VD, MODE>;
  struct Tag : CF {};
  if (once_per_device<Tag>([] {
        return cudaFuncSetAttribute(linattn_pass_kernel<T, KD, VD, MODE, FAST>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, CF::kSmem) == cudaSuccess;
      }) != 1)
    return SS_ERR_CUDA;
  const int64_t grid = a.workers > 0 ? a.workers : (int64_t)a.bh * a.nseg;
  if (grid > INT_MAX) return SS_ERR_INVALID_ARG;
  if (a.workers > 0 &&
      cudaMemsetAsync(a.flags, 0, (1 + (size_t)a.workers * 16) * sizeof(unsigned), stream) != cudaSuccess)
    return SS_ERR_CUDA;
  linattn_pass_kernel<T, KD, VD, MODE, FAST><<<(unsigned)grid, CF::kThreads, CF::kSmem, stream>>>(a, maps);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <typename T, int KD, int VD, LaMode MODE>
ss_status la_launch(const LaPassArgs& a, const LaMaps& maps, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    const bool stores = MODE == kLaStates || a.out_vec || (MODE == kLaProducts && a.out_f32);
    if (a.tma && !a.lengths && stores && (MODE != kLaProducts || a.x_vec))
      return la_launch_as<T, KD, VD, MODE, true>(a, maps, stream);
  }
  return la_launch_as<T, KD, VD, MODE, false>(a, maps, stream);
}

template <typename T, LaMode MODE>
ss_status la_dispatch(LaPassArgs a, int64_t batch, cudaStream_t stream) {
  const int es = sizeof(T);
  a.vec = la_vec(a.k, a.dk, es) && la_vec(a.v, a.dv, es) && (MODE == kLaStates || la_vec(a.q, a.dk, es));
  a.out_vec = es == 2 && !a.out_f32 && a.out && aligned(a.out, 16) && a.dv % 8 == 0;
  a.x_vec = es == 2 && a.x.ptr && la_vec(a.x, a.dv, es);
  LaMaps m = {};
  if (es == 2 && a.vec) {
    auto map = [&](CUtensorMap* to, const LaTensor& x, int d) {
      return la_map(to, x, batch, a.seqlen, a.heads / x.share, d);
    };
    a.tma = map(&m.k, a.k, a.dk) && map(&m.v, a.v, a.dv) && (MODE == kLaStates || map(&m.q, a.q, a.dk));
  }
  if (a.dk <= 64) return a.dv <= 64 ? la_launch<T, 64, 64, MODE>(a, m, stream) : la_launch<T, 64, 128, MODE>(a, m, stream);
  return a.dv <= 64 ? la_launch<T, 128, 64, MODE>(a, m, stream) : la_launch<T, 128, 128, MODE>(a, m, stream);
}

template <LaMode MODE>
ss_status la_pass(const LaPassArgs& a, bool bf16, int64_t batch, cudaStream_t stream) {
  return bf16 ? la_dispatch<__nv_bfloat16, MODE>(a, batch, stream) : la_dispatch<float, MODE>(a, batch, stream);
}

// The starting states of every segment of pass `a` (its k, v, g and directions) into seg.
ss_status la_segment_states(LaPassArgs a, const LaShape& s, const LaSegs& g, const LaSeg& seg, const float* s0,
                            cudaStream_t stream) {
  a.nseg = g.nseg - 1;
  a.seg_chunks = g.chunks;
  a.s_in = nullptr;
  a.s_out = seg.states;
  a.s_out_head = (int64_t)g.nseg * s.per_state();
  a.s_out_seg = s.per_state();
  a.seg_decay = seg.decay;
  const ss_status st = la_pass<kLaStates>(a, s.bf16, s.batch, stream);
  if (st != SS_OK) return st;
  // (segments are cut where there are no more heads than SMs, so they fit the grid's rows)
  linattn_join_kernel<<<dim3((unsigned)((s.per_state() + 255) / 256), (unsigned)s.bh()), 256, 0, stream>>>(
      seg.states, seg.decay, s0, g.nseg, s.per_state());
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

// Test hooks (ss_scan_debug.h): consumed by the next forward or backward call.
std::atomic<long long> g_dbg_la_spin_limit{0};
std::atomic<long long> g_dbg_la_skip_publish{-1};
std::atomic<long long> g_dbg_la_skip_load{-1};

LaPassArgs la_base(const LaShape& s, const ss_heads* g, const int32_t* lengths, const LaSegs& segs) {
  LaPassArgs a = {};
  const long long spin = g_dbg_la_spin_limit.exchange(0);
  a.carry_spin_limit = spin > 0 ? (uint32_t)spin : kLaCarrySpinLimit;
  a.skip_publish = (int)g_dbg_la_skip_publish.exchange(-1);
  a.skip_load = (int)g_dbg_la_skip_load.exchange(-1);
  a.g = la_tensor(*g, s, 1, 1);
  a.lengths = lengths;
  a.heads = s.heads;
  a.seqlen = (int)s.seqlen;
  a.bh = (int)s.bh();
  a.nseg = segs.nseg;
  a.seg_chunks = segs.chunks;
  a.chunks = la_chunks(s);
  a.scale_p = a.scale_o = a.scale_w = 1.f;
  return a;
}

// Where a pass starts: the segments' states, or the caller's.
void la_start(LaPassArgs& a, const LaShape& s, const LaSegs& g, const LaSeg& seg, const float* s0) {
  a.workers = g.workers;
  a.carry = seg.carry;
  a.flags = seg.flags;
  a.s_in = g.nseg > 1 ? seg.states : s0;
  a.s_in_head = (int64_t)g.nseg * s.per_state();
  a.s_in_seg = s.per_state();
  a.s_out_head = s.per_state();
  a.s_out_seg = 0;
}

ss_status linattn_fwd_impl(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* g, float scale,
                           const float* s0, const int32_t* lengths, void* o, float* last, const LaShape& s,
                           int in_dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const ss_status shape = la_check_shape(s, in_dtype);
  if (shape != SS_OK) return shape;
  const int es = s.es();
  if (!la_check_heads(q, es) || !la_check_heads(k, es) || !la_check_heads(v, es) || !la_check_heads(g, es) || !o)
    return SS_ERR_INVALID_ARG;
  if (!aligned(o, es) || !aligned(s0, 4) || !aligned(last, 4) || !aligned(lengths, 4)) return SS_ERR_INVALID_ARG;
  const LaSegs segs = la_plan(s);
  const size_t need = la_seg_bytes(s, segs);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 256))) return SS_ERR_INVALID_ARG;
  const LaSeg seg = la_seg_at(static_cast<char*>(ws), s, segs);
  LaPassArgs a = la_base(s, g, lengths, segs);
  const int share = s.heads / s.qk_heads;
  a.q = la_tensor(*q, s, share, s.dk);
  a.k = la_tensor(*k, s, share, s.dk);
  a.v = la_tensor(*v, s, 1, s.dv);
  a.dk = s.dk;
  a.dv = s.dv;
  a.sk = s.dv;
  a.sv = 1;
  if (segs.nseg > 1) {
    const ss_status st = la_segment_states(a, s, segs, seg, s0, stream);
    if (st != SS_OK) return st;
  }
  la_start(a, s, segs, seg, s0);
  a.s_out = last;
  a.out = o;
  a.scale_p = a.scale_o = scale;
  return la_pass<kLaOutputs>(a, s.bf16, s.batch, stream);
}

// ---- backward

ss_status la_check_bwd_shape(const LaShape& s, int in_dtype) {
  const ss_status st = la_check_shape(s, in_dtype);
  if (st != SS_OK) return st;
  // a block of the decays' gradient each (the gradients of so many alone are 256 GB)
  return s.bh() * la_chunks(s) > INT_MAX ? SS_ERR_INVALID_ARG : SS_OK;
}

struct LaBwdWs {
  size_t dots_q = 0, dots_k = 0, flow = 0, dump = 0, part = 0, bytes = 0;
};
LaBwdWs la_bwd_ws(const LaShape& s, const LaSegs& g) {
  LaBwdWs w;
  size_t at = la_seg_bytes(s, g);
  auto take = [&at](size_t n) {
    const size_t r = at;
    at += align256(n);
    return r;
  };
  const size_t rows = (size_t)s.bh() * s.seqlen, chunks = (size_t)s.bh() * la_chunks(s);
  w.dots_q = take(rows * 16);
  w.dots_k = take(rows * 16);
  w.flow = take(chunks * 16 * 4);
  // a state for every chunk, as the warps hold it
  w.dump = take(chunks * (s.dk <= 64 ? 64 : 128) * (s.dv <= 64 ? 64 : 128) * 4);
  w.part = take(s.heads > s.qk_heads ? rows * s.dk * 4 : 0);
  w.bytes = at;
  return w;
}

template <typename T, int VEC, typename I>
ss_status la_launch_share(const float* part, void* out, const int32_t* lengths, const LaShape& s, int64_t total,
                          cudaStream_t stream) {
  const int64_t blocks = (total + 255) / 256;
  if (blocks > INT_MAX) return SS_ERR_INVALID_ARG;
  linattn_share_kernel<T, VEC, I><<<(unsigned)blocks, 256, 0, stream>>>(
      part, static_cast<T*>(out), lengths, (I)s.seqlen, (I)total, s.heads, s.heads / s.qk_heads, s.dk);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <typename T>
ss_status la_share_sum(const float* part, void* out, const int32_t* lengths, const LaShape& s, cudaStream_t stream) {
  const bool vec = s.dk % 4 == 0 && aligned(out, 4 * sizeof(T));
  const int64_t total = s.batch * s.seqlen * s.qk_heads * (vec ? s.dk / 4 : s.dk);
  const bool small = s.batch * s.seqlen * s.qk_heads * s.dk < INT_MAX;  // 32-bit divisions
  if (vec) return small ? la_launch_share<T, 4, uint32_t>(part, out, lengths, s, total, stream)
                        : la_launch_share<T, 4, uint64_t>(part, out, lengths, s, total, stream);
  return small ? la_launch_share<T, 1, uint32_t>(part, out, lengths, s, total, stream)
               : la_launch_share<T, 1, uint64_t>(part, out, lengths, s, total, stream);
}

template <typename T, bool VEC>
ss_status la_launch_decay_grad(const LaGradArgs& a, const LaShape& s, cudaStream_t stream) {
  struct Tag {};
  if (once_per_device<Tag>([] {
        return cudaFuncSetAttribute(linattn_decay_grad_kernel<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    la_grad_smem(128, 128, sizeof(T))) == cudaSuccess;
      }) != 1)
    return SS_ERR_CUDA;
  linattn_decay_grad_kernel<T, VEC>
      <<<(unsigned)(s.bh() * a.chunks), kLaGradThreads, la_grad_smem(s.dk, s.dv, sizeof(T)), stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

template <typename T>
ss_status la_decay_grad(const LaGradArgs& a, const LaShape& s, cudaStream_t stream) {
  const int es = sizeof(T);
  const bool vec = la_vec(a.q, s.dk, es) && la_vec(a.k, s.dk, es) && la_vec(a.v, s.dv, es) && la_vec(a.d, s.dv, es);
  return vec ? la_launch_decay_grad<T, true>(a, s, stream) : la_launch_decay_grad<T, false>(a, s, stream);
}

ss_status linattn_bwd_impl(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* g,
                           const ss_heads* d_o, float scale, const float* s0, const float* dlast,
                           const int32_t* lengths, void* dq, void* dk, void* dv, void* dg, float* ds0,
                           const LaShape& s, int in_dtype, void* ws, size_t ws_bytes, cudaStream_t stream) {
  ss_status st = la_check_bwd_shape(s, in_dtype);
  if (st != SS_OK) return st;
  const int es = s.es();
  for (const ss_heads* x : {q, k, v, g, d_o})
    if (!la_check_heads(x, es)) return SS_ERR_INVALID_ARG;
  for (const void* x : {dq, dk, dv, dg})
    if (!x || !aligned(x, es)) return SS_ERR_INVALID_ARG;
  if (!aligned(s0, 4) || !aligned(dlast, 4) || !aligned(lengths, 4) || !aligned(ds0, 4)) return SS_ERR_INVALID_ARG;
  const LaSegs segs = la_plan(s);
  const LaBwdWs w = la_bwd_ws(s, segs);
  if (!ws || ws_bytes < w.bytes || !aligned(ws, 256)) return SS_ERR_INVALID_ARG;
  char* base = static_cast<char*>(ws);
  const LaSeg seg = la_seg_at(base, s, segs);
  const int share = s.heads / s.qk_heads;
  const LaTensor tq = la_tensor(*q, s, share, s.dk), tk = la_tensor(*k, s, share, s.dk), tv = la_tensor(*v, s, 1, s.dv),
                 td = la_tensor(*d_o, s, 1, s.dv);
  float* part = reinterpret_cast<float*>(base + w.part);

  // dq: a forward pass with (do, v, k); its state is S with the two indices exchanged
  LaPassArgs a = la_base(s, g, lengths, segs);
  a.dump = reinterpret_cast<float*>(base + w.dump);
  a.flow = reinterpret_cast<float*>(base + w.flow);
  a.q = td;
  a.k = tv;
  a.v = tk;
  a.dk = s.dv;
  a.dv = s.dk;
  a.sk = 1;
  a.sv = s.dv;
  if (segs.nseg > 1 && (st = la_segment_states(a, s, segs, seg, s0, stream)) != SS_OK) return st;
  la_start(a, s, segs, seg, s0);
  a.scale_p = a.scale_o = scale;
  a.out = share > 1 ? part : dq;
  a.out_f32 = share > 1;
  a.x = tq;
  a.dots = reinterpret_cast<float*>(base + w.dots_q);
  if ((st = la_pass<kLaProducts>(a, s.bf16, s.batch, stream)) != SS_OK) return st;
  if (share > 1 && (st = s.bf16 ? la_share_sum<__nv_bfloat16>(part, dq, lengths, s, stream)
                                : la_share_sum<float>(part, dq, lengths, s, stream)) != SS_OK)
    return st;

  // dk: reversed with (v, do, q); the state is R, the gradient of S
  a.reverse = 1;
  a.q = tv;
  a.k = td;
  a.v = tq;
  a.scale_p = a.scale_w = scale;
  a.scale_o = 1.f;
  if (segs.nseg > 1 && (st = la_segment_states(a, s, segs, seg, dlast, stream)) != SS_OK) return st;
  la_start(a, s, segs, seg, dlast);
  a.out = share > 1 ? part : dk;
  a.x = tk;
  a.dots = reinterpret_cast<float*>(base + w.dots_k);
  // the initial state's gradient waits for the last pass where it overwrites dlast
  if ((st = la_pass<kLaProducts>(a, s.bf16, s.batch, stream)) != SS_OK) return st;
  if (share > 1 && (st = s.bf16 ? la_share_sum<__nv_bfloat16>(part, dk, lengths, s, stream)
                                : la_share_sum<float>(part, dk, lengths, s, stream)) != SS_OK)
    return st;
  LaGradArgs dec = {};
  dec.q = tq, dec.k = tk, dec.v = tv, dec.d = td, dec.g = a.g;
  dec.lengths = lengths;
  dec.dots_q = reinterpret_cast<float*>(base + w.dots_q);
  dec.dots_k = a.dots;
  dec.flow = a.flow;
  dec.out = dg;
  dec.heads = s.heads, dec.seqlen = a.seqlen, dec.dk = s.dk, dec.dv = s.dv, dec.chunks = a.chunks;
  dec.scale = scale;
  if ((st = s.bf16 ? la_decay_grad<__nv_bfloat16>(dec, s, stream) : la_decay_grad<float>(dec, s, stream)) != SS_OK) return st;

  // dv: reversed with (k, q, do)
  a.q = tk;
  a.k = tq;
  a.v = td;
  a.dk = s.dk;
  a.dv = s.dv;
  a.sk = s.dv;
  a.sv = 1;
  a.out = dv;
  a.out_f32 = 0;
  a.x = LaTensor{};
  a.x.share = 1;
  a.dots = nullptr;
  a.dump = nullptr;
  a.s_out = ds0;
  return la_pass<kLaOutputs>(a, s.bf16, s.batch, stream);
}

// ---- single tokens

template <typename T>
ss_status la_launch_step(const LaStepArgs& a, bool vec, cudaStream_t stream) {
  const dim3 grid((unsigned)(a.heads * ((a.dv + kLaStepCols - 1) / kLaStepCols)), (unsigned)a.batch);
  if (vec) linattn_step_kernel<T, 4><<<grid, kLaStepThreads, 0, stream>>>(a);
  else linattn_step_kernel<T, 1><<<grid, kLaStepThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

ss_status linattn_step_impl(const ss_heads* q, const ss_heads* k, const ss_heads* v, const ss_heads* g, float scale,
                            float* state, int64_t num_slots, const int32_t* slots, void* o, const LaShape& s,
                            int in_dtype, cudaStream_t stream) {
  const ss_status shape = la_check_shape(s, in_dtype);
  if (shape != SS_OK) return shape;
  const int es = s.es();
  for (const ss_heads* x : {q, k, v, g})
    if (!la_check_heads(x, es)) return SS_ERR_INVALID_ARG;
  if (!o || !aligned(o, es) || !state || !aligned(state, 4) || !aligned(slots, 4)) return SS_ERR_INVALID_ARG;
  if (s.batch > 65535 || num_slots < 1 || (!slots && num_slots < s.batch)) return SS_ERR_INVALID_ARG;
  LaStepArgs a = {};
  const int share = s.heads / s.qk_heads;
  a.q = la_tensor(*q, s, share, s.dk);
  a.k = la_tensor(*k, s, share, s.dk);
  a.v = la_tensor(*v, s, 1, s.dv);
  a.g = la_tensor(*g, s, 1, 1);
  a.state = state;
  a.num_slots = num_slots;
  a.slots = slots;
  a.out = o;
  a.batch = (int)s.batch;
  a.heads = s.heads;
  a.dk = s.dk;
  a.dv = s.dv;
  a.scale = scale;
  const bool vec = aligned(state, 16) && s.dv % 4 == 0;
  return s.bf16 ? la_launch_step<__nv_bfloat16>(a, vec, stream) : la_launch_step<float>(a, vec, stream);
}

// ---- the pool

ss_status pool_check(const void* state, const void* codes, const void* scales, int64_t num_slots, const int32_t* slots,
                     int64_t batch, int64_t rows, int width) {
  if (!state || !codes || !scales || batch < 1 || rows < 1 || width < 1 || num_slots < 1) return SS_ERR_INVALID_ARG;
  if (!aligned(state, 4) || !aligned(scales, 4) || !aligned(slots, 4)) return SS_ERR_INVALID_ARG;
  if (batch > 65535 || (!slots && num_slots < batch)) return SS_ERR_INVALID_ARG;
  if (width > 1024) return SS_ERR_UNSUPPORTED;
  if (rows > (INT_MAX - 1024) / width) return SS_ERR_INVALID_ARG;
  return SS_OK;
}

template <int LANES, int VEC, int REGS>
ss_status pool_store(const PoolArgs& a, cudaStream_t stream) {
  const int64_t tiles = (a.rows + kPoolThreads / LANES - 1) / (kPoolThreads / LANES);
  state_store8_kernel<LANES, VEC, REGS><<<dim3((unsigned)tiles, (unsigned)a.batch), kPoolThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

ss_status state_store8_impl(const PoolArgs& a, cudaStream_t stream) {
  const bool vec = a.width % 4 == 0 && aligned(a.state, 16) && aligned(a.codes, 4);
  if (vec) {
    if (a.width <= 16) return pool_store<4, 4, 1>(a, stream);
    if (a.width <= 32) return pool_store<8, 4, 1>(a, stream);
    if (a.width <= 64) return pool_store<8, 4, 2>(a, stream);
    if (a.width <= 128) return pool_store<8, 4, 4>(a, stream);
    if (a.width <= 256) return pool_store<16, 4, 4>(a, stream);
    if (a.width <= 512) return pool_store<32, 4, 4>(a, stream);
    return pool_store<32, 4, 8>(a, stream);
  }
  if (a.width <= 32) return pool_store<8, 1, 4>(a, stream);
  if (a.width <= 128) return pool_store<32, 1, 4>(a, stream);
  if (a.width <= 512) return pool_store<32, 1, 16>(a, stream);
  return pool_store<32, 1, 32>(a, stream);
}

template <int LANES, int REGS, int ROWS>
ss_status pool_load(const PoolArgs& a, cudaStream_t stream) {
  const int64_t per = kPoolThreads / LANES * ROWS, blocks = (a.rows + per - 1) / per;
  state_load8_kernel<LANES, REGS, ROWS><<<dim3((unsigned)blocks, (unsigned)a.batch), kPoolThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

ss_status state_load8_impl(const PoolArgs& a, cudaStream_t stream) {
  if (a.width % 4 == 0 && aligned(a.state, 16) && aligned(a.codes, 4)) {
    if (a.width <= 16) return pool_load<4, 1, 8>(a, stream);
    if (a.width <= 32) return pool_load<8, 1, 8>(a, stream);
    if (a.width <= 64) return pool_load<16, 1, 8>(a, stream);
    if (a.width <= 128) return pool_load<32, 1, 8>(a, stream);
    if (a.width <= 256) return pool_load<32, 2, 4>(a, stream);
    if (a.width <= 512) return pool_load<32, 4, 2>(a, stream);
    return pool_load<32, 8, 1>(a, stream);
  }
  const int64_t blocks = (a.rows * a.width + kPoolThreads - 1) / kPoolThreads;
  state_load8_plain_kernel<<<dim3((unsigned)blocks, (unsigned)a.batch), kPoolThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SS_OK : SS_ERR_CUDA;
}

}  // namespace
}  // namespace ssscan

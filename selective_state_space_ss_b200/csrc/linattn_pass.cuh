// linattn_pass.cuh -- one pass of the decayed linear attention over a sequence,
// the kernel behind ss_linattn_fwd and behind each gradient of ss_linattn_bwd.
//
// For every batch row and head, with queries q, keys k, values v and log decays g,
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,     o_t = S_t^T q_t.
//
// In chunks of C = 64 tokens, with G the running sum of g inside the chunk and S
// the state before it:
//
//   O  = ((Q K^T) . D) V + diag(e^G) Q S,     D_ij = e^{G_i - G_j} for j <= i, else 0
//   S <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
//
// A reversed pass (each token sees itself and the later ones; the state runs from
// the end) is the same with the two row factors exchanged and the mask and the
// sign of the exponent turned round:
//
//   D_ji = e^{G_i - G_j} for i >= j,  rows take e^{G_C - G_j},  keys take e^{G_i}.
//
// The gradients of the attention are such passes themselves: with do for q, v for
// k and k for v, a forward pass gives dq; (v, do, q) and (k, q, do) reversed give
// dk and dv.  So one kernel serves all four.
//
// Precision.  The tensor core multiplies bf16 and adds in fp32.  A value that is
// not bf16 already is split into bf16 planes (split2): bf16 inputs stay as they
// are, what is computed here (the masked products P, the weighted keys, the state)
// takes two planes, 16 bits, a relative error of about 1e-6 at every product; fp32
// inputs and everything behind them take three planes, 24 bits, and the six
// products of planes whose weight reaches that far.  The state itself stays fp32 in
// registers.  Running sums of the decays are fp64, kept as two floats.
//
// Layout.  Scores are Q K^T with tokens in the lanes.  O and S are kept transposed
// (value index in the lanes), so that S^T is the MMA's A operand straight from
// tensor memory: it is written there by the threads that hold it and never goes
// through shared memory.  M is 128 throughout; where only 64 rows mean something
// (tokens, 64-wide values) the other lanes hold sums of whatever follows in shared
// memory and nobody reads them.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "scan_common.cuh"
#include "tc5.cuh"

namespace ssscan {

constexpr int kLaChunk = 64;
constexpr int kLaBlock = kLaChunk * kTileRow;  // bytes of one plane's 64 x 64 block
constexpr uint32_t kLaSpinLimit = 1u << 20;

// A [batch, seqlen, heads, d] tensor, last axis contiguous, strides in elements;
// `share` consecutive heads of the pass read one of its heads.
struct LaTensor {
  const void* ptr;
  int64_t sb, st, sh;
  int share;
};

struct LaPassArgs {
  LaTensor q, k, v;
  LaTensor g;           // log decays [batch, seqlen, heads]
  const int* lengths;   // [batch] or null
  const float* s_in;    // states before the first chunk, or null (zero)
  float* s_out;         // states behind the last chunk, or null
  int64_t s_in_head, s_in_seg, s_out_head, s_out_seg;  // strides per (batch, head), per segment
  int64_t sk, sv;       // strides of a state's key and value index
  double* seg_decay;    // states-only: each segment's sum of g (base 2)
  void* out;            // [batch, seqlen, heads, dv] contiguous
  int out_f32;          // out is float32 whatever the inputs
  LaTensor x;           // rows to take the inner product of each output row with (ptr null: none)
  float* dots;          // [batch * heads, seqlen, 4] partial products of x
  float* dump;          // forward: where the states at anchors go; reversed: where they come from
  float* anchor;        // reversed: [batch * heads, anchors, 8] partial products <R, S> at anchors
  int anchor_chunks;    // an anchor behind every so many chunks
  int anchors;          // anchors of the longest row
  int heads, seqlen, dk, dv;
  int nseg, seg_chunks;
  int reverse;
  int vec;              // 16-byte loads apply to q, k and v
  float scale_p, scale_o, scale_w;
};

template <typename T, int KD, int VD>
struct LaCfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPI = kBf16 ? 1 : 3;  // planes of the inputs
  static constexpr int NPX = kBf16 ? 2 : 3;  // planes of what is computed here
  static constexpr int NPMAX = NPX;          // products of planes a, b with a + b < NPMAX
  static constexpr int KB = KD / 64, VB = VD / 64;
  static constexpr int kStages = kBf16 ? 2 : 1;
  static constexpr int kQ = 0, kK = KB * NPI * kLaBlock, kV = 2 * kK;
  static constexpr int kStageBytes = kV + VB * NPI * kLaBlock;
  static constexpr int kP = kStages * kStageBytes;
  static constexpr int kW = kP + NPX * kLaBlock;
  static constexpr int kFac = kW + NPX * KB * kLaBlock;
  static constexpr int kSmem = kFac + kStages * (4 * kLaChunk + 4) * 4 + 256 + 1024;
  // tensor memory columns
  static constexpr int cDS = 0, cSP = KD, cO1 = cSP + NPX * KD / 2, cO2 = cO1 + 64, cQK = cO2 + 64;
  static constexpr int kCols = cQK + 64 <= 256 ? 256 : 512;
  static_assert(cQK + 64 <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr int kComputeWarps = 8, kLoadWarps = 3;
  static constexpr int kThreads = 32 * (kComputeWarps + 1 + kLoadWarps);
};

// Waits of one CTA: when one gives up, the others stop waiting too, and the kernel
// runs to its end on whatever is there, inside its buffers.
__device__ __forceinline__ void la_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return;
  for (uint32_t i = 0; i < kLaSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if (*dead) return;
  }
  atomicOr(&g_error_word, kErrTmaWait);
  *dead = 1;
}

__device__ __forceinline__ int la_length(const LaPassArgs& a, int64_t b) {
  if (!a.lengths) return a.seqlen;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n < a.seqlen ? n : a.seqlen;
}

__device__ __forceinline__ const char* la_row(const LaTensor& x, int64_t b, int64_t t, int h, int es) {
  return static_cast<const char*>(x.ptr) + (b * x.sb + t * x.st + (int64_t)(h / x.share) * x.sh) * es;
}

// One tile of 64 tokens into shared memory: rows from `len` on and columns from `d`
// on are zero.  bf16 with 16-byte rows: asynchronous copies (the caller waits);
// everything else through registers.
template <typename T, int DP>
__device__ __forceinline__ void la_load_tile(char* dst, const LaTensor& x, int64_t b, int h, int t0,
                                             int len, int d, bool vec, int tid, int nthreads) {
  constexpr int B = DP / 64;
  constexpr int UNITS = kLaChunk * B * 8;
  for (int u = tid; u < UNITS; u += nthreads) {
    const int row = u / (B * 8), unit = u % (B * 8), col = unit * 8;
    const bool in = t0 + row < len && col < d && in_range(t0 + row, len);
    char* to = dst + (unit / 8) * kLaBlock + tile_unit(row, unit % 8);
    const char* from = la_row(x, b, in ? t0 + row : 0, h, sizeof(T)) + (in ? col : 0) * (int)sizeof(T);
    if constexpr (sizeof(T) == 2) {
      if (vec) {
        const uint32_t bytes = in ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(to)), "l"(from), "r"(bytes)
                     : "memory");
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(from) + 2 * i;
          const uint32_t lo = in && col + 2 * i < d ? p[0] : 0;
          const uint32_t hi = in && col + 2 * i + 1 < d ? p[1] : 0;
          w[i] = lo | hi << 16;
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      float f[8];
      const float* p = reinterpret_cast<const float*>(from);
      if (vec) {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 f0 = in ? reinterpret_cast<const float4*>(p)[0] : z;
        const float4 f1 = in && col + 4 < d ? reinterpret_cast<const float4*>(p)[1] : z;
        f[0] = f0.x, f[1] = f0.y, f[2] = f0.z, f[3] = f0.w, f[4] = f1.x, f[5] = f1.y, f[6] = f1.z, f[7] = f1.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = in && col + i < d ? p[i] : 0.f;
      }
      uint32_t w[3][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t s[3];
        split2<3>(f[2 * i], f[2 * i + 1], s);
        w[0][i] = s[0], w[1][i] = s[1], w[2][i] = s[2];
      }
#pragma unroll
      for (int p3 = 0; p3 < 3; ++p3)
        *reinterpret_cast<uint4*>(to + p3 * B * kLaBlock) = make_uint4(w[p3][0], w[p3][1], w[p3][2], w[p3][3]);
    }
  }
}

// A chunk's decays: running sums (base 2) as two floats, the factors of the rows and
// of the keys, and the chunk's whole decay.  One warp, two tokens a lane.  A log
// decay below -1400 leaves nothing in fp32 and is taken as that, so that minus
// infinity (a reset) does not turn differences of sums into NaN.
template <typename T>
__device__ __forceinline__ double la_decays(float* fac, const LaPassArgs& a, int64_t b, int h, int t0, int len,
                                            int lane, bool active) {
  double g[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = t0 + 2 * lane + i;
    float x = 0.f;
    if (active && t < len && in_range(t, len)) {
      const char* p = la_row(a.g, b, t, h, sizeof(T));
      x = to_f32(*reinterpret_cast<const T*>(p));
    }
    x = x < -1400.f ? -1400.f : x;
    g[i] = (double)x * 1.4426950408889634;
  }
  double sum = g[0] + g[1];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const double up = __shfl_up_sync(kFullMask, sum, o);
    if (lane >= o) sum += up;
  }
  const double total = __shfl_sync(kFullMask, sum, 31);
  const double at[2] = {sum - g[1], sum};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * lane + i;
    const float hi = (float)at[i];
    fac[r] = hi;
    fac[kLaChunk + r] = (float)(at[i] - (double)hi);
    const float from_start = (float)exp2(at[i]), to_end = (float)exp2(total - at[i]);
    fac[2 * kLaChunk + r] = a.reverse ? to_end : from_start;  // rows
    fac[3 * kLaChunk + r] = a.reverse ? from_start : to_end;  // keys
  }
  if (lane == 0) fac[4 * kLaChunk] = (float)exp2(total);
  return total;
}

// Sum over the lanes of v[i], for every i at once: lane i gets the sum of v[i].
__device__ __forceinline__ float la_column_sums(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(kFullMask, send, o);
    }
  }
  return v[0];
}

// STATES: only the states (the sequence's segments, each from zero, all at once).
template <typename T, int KD, int VD, bool STATES>
__global__ void __launch_bounds__(LaCfg<T, KD, VD>::kThreads, 1) linattn_pass_kernel(const __grid_constant__ LaPassArgs a) {
  using CF = LaCfg<T, KD, VD>;
  constexpr int NPI = CF::NPI, NPX = CF::NPX, ST = CF::kStages;
  extern __shared__ char la_smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(la_smem_raw) + 1023) & ~uintptr_t(1023));
  float* fac_all = reinterpret_cast<float*>(smem + CF::kFac);
  uint64_t* bars = reinterpret_cast<uint64_t*>(fac_all + ST * (4 * kLaChunk + 4));
  uint64_t *b_full = bars, *b_empty = bars + 2, *b_qk = bars + 4, *b_pk = bars + 5, *b_s = bars + 6, *b_ds = bars + 7;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(bars + 8);
  volatile int* dead = reinterpret_cast<int*>(tmem_at + 1);

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int64_t bh = blockIdx.x / a.nseg;
  const int step = (int)(blockIdx.x % a.nseg);  // the segment's place in the order of processing
  const int64_t b = bh / a.heads;
  const int h = (int)(bh % a.heads);
  const int len = la_length(a, b);
  const int all_chunks = (len + kLaChunk - 1) / kLaChunk;
  const int total_segs = STATES ? a.nseg + 1 : a.nseg;  // the last one's states are nobody's start
  const int seg = a.reverse ? total_segs - 1 - step : step;
  const int64_t first64 = (int64_t)seg * a.seg_chunks;
  const int first = first64 < all_chunks ? (int)first64 : all_chunks;
  const int last = first64 + a.seg_chunks < all_chunks ? (int)(first64 + a.seg_chunks) : all_chunks;
  const int n_chunks = last - first;
  auto chunk_at = [&](int n) { return a.reverse ? last - 1 - n : first + n; };

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&b_full[i], 32 * CF::kLoadWarps);
      mbar_init(&b_empty[i], CF::kComputeWarps);
    }
    mbar_init(b_qk, 1);
    mbar_init(b_pk, CF::kComputeWarps);
    mbar_init(b_s, CF::kComputeWarps);
    mbar_init(b_ds, 1);
    fence_mbar_init();
    *dead = 0;
  }
  if (warp == CF::kComputeWarps) tmem_alloc(tmem_at, CF::kCols);
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = *tmem_at;

  if (warp > CF::kComputeWarps) {
    // ---- loaders
    const int ltid = tid - 32 * (CF::kComputeWarps + 1);
    double sum = 0.0;
    for (int n = 0; n <= n_chunks; ++n) {
      if (n < n_chunks) {
        const int s = n % ST;
        if (n >= ST) la_wait(&b_empty[s], (uint32_t)((n / ST - 1) & 1), dead);
        const int t0 = chunk_at(n) * kLaChunk;
        char* st = smem + s * CF::kStageBytes;
        la_load_tile<T, KD>(st + CF::kK, a.k, b, h, t0, len, a.dk, a.vec, ltid, 32 * CF::kLoadWarps);
        if (!STATES) la_load_tile<T, KD>(st + CF::kQ, a.q, b, h, t0, len, a.dk, a.vec, ltid, 32 * CF::kLoadWarps);
        la_load_tile<T, VD>(st + CF::kV, a.v, b, h, t0, len, a.dv, a.vec, ltid, 32 * CF::kLoadWarps);
        if (ltid < 32) sum += la_decays<T>(fac_all + s * (4 * kLaChunk + 4), a, b, h, t0, len, lane, true);
        cp_async_commit();
      }
      // the tiles that are signalled now: with two stages the previous chunk's
      const int m = ST == 1 ? n : n - 1;
      if (m >= 0 && m < n_chunks) {
        if (ST == 1 || n == n_chunks) asm volatile("cp.async.wait_group 0;\n" ::: "memory");
        else asm volatile("cp.async.wait_group 1;\n" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(&b_full[m % ST]);
      }
    }
    if (STATES && ltid == 0) a.seg_decay[bh * total_segs + step] = sum;
  } else if (warp == CF::kComputeWarps) {
    // ---- MMA issue, one thread
    if (lane == 0) {
      const uint32_t base = smem_u32(smem);
      auto tile = [&](int s, int what, int blocks, int plane) {
        return base + s * CF::kStageBytes + what + plane * blocks * kLaBlock;
      };
      auto scores = [&](int n) {
        const int s = n % ST;
        la_wait(&b_full[s], (uint32_t)((n / ST) & 1), dead);
        tc5_fence_after();
        constexpr uint32_t id = mma_idesc(64, false, false);
        bool add = false;
        for (int pa = NPI - 1; pa >= 0; --pa)
          for (int pb = (NPI < CF::NPMAX - pa ? NPI : CF::NPMAX - pa) - 1; pb >= 0; --pb)
#pragma unroll
            for (int kk = 0; kk < KD; kk += 16) {
              const uint32_t off = (kk / 64) * kLaBlock + (kk % 64) * 2;
              mma_ss(tmem + CF::cQK, tile_desc(tile(s, CF::kQ, CF::KB, pa) + off, 0),
                     tile_desc(tile(s, CF::kK, CF::KB, pb) + off, 0), id, add);
              add = true;
            }
        mma_commit(b_qk);
      };
      if (!STATES && n_chunks > 0) scores(0);
      for (int n = 0; n < n_chunks; ++n) {
        const int s = n % ST;
        if (!STATES) {
          // O2^T = S^T Q^T
          la_wait(b_s, (uint32_t)(n & 1), dead);
          tc5_fence_after();
          constexpr uint32_t id = mma_idesc(64, false, false);
          bool add = false;
          for (int pa = NPX - 1; pa >= 0; --pa)
            for (int pb = (NPI < CF::NPMAX - pa ? NPI : CF::NPMAX - pa) - 1; pb >= 0; --pb)
#pragma unroll
              for (int kk = 0; kk < KD; kk += 16) {
                const uint32_t off = (kk / 64) * kLaBlock + (kk % 64) * 2;
                mma_ts(tmem + CF::cO2, tmem + CF::cSP + pa * (KD / 2) + kk / 2,
                       tile_desc(tile(s, CF::kQ, CF::KB, pb) + off, 0), id, add);
                add = true;
              }
        } else {
          la_wait(&b_full[s], (uint32_t)((n / ST) & 1), dead);
        }
        la_wait(b_pk, (uint32_t)(n & 1), dead);
        tc5_fence_after();
        {
          // dS^T = V^T (w . K)
          constexpr uint32_t id = mma_idesc(KD, true, true);
          bool add = false;
          for (int pa = NPI - 1; pa >= 0; --pa)
            for (int pb = (NPX < CF::NPMAX - pa ? NPX : CF::NPMAX - pa) - 1; pb >= 0; --pb)
#pragma unroll
              for (int j = 0; j < kLaChunk; j += 16) {
                mma_ss(tmem + CF::cDS, tile_desc(tile(s, CF::kV, CF::VB, pa) + j * kTileRow, kLaBlock),
                       tile_desc(base + CF::kW + pb * CF::KB * kLaBlock + j * kTileRow, kLaBlock), id, add);
                add = true;
              }
        }
        if (!STATES) {
          // O1^T = V^T P^T
          constexpr uint32_t id = mma_idesc(64, true, false);
          bool add = false;
          for (int pa = NPI - 1; pa >= 0; --pa)
            for (int pb = (NPX < CF::NPMAX - pa ? NPX : CF::NPMAX - pa) - 1; pb >= 0; --pb)
#pragma unroll
              for (int j = 0; j < kLaChunk; j += 16) {
                mma_ss(tmem + CF::cO1, tile_desc(tile(s, CF::kV, CF::VB, pa) + j * kTileRow, kLaBlock),
                       tile_desc(base + CF::kP + pb * kLaBlock + j * 2, 0), id, add);
                add = true;
              }
        }
        mma_commit(b_ds);
        if (!STATES && n + 1 < n_chunks) scores(n + 1);
      }
    }
    __syncwarp();
  } else {
    // ---- compute
    const int quad = warp % 4, half = warp / 4;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int vi = quad * 32 + lane;          // this thread's value index
    const bool holds = quad * 32 < VD;        // warps whose lanes hold a state
    constexpr int KH = KD / 2;                // its key indices: half * KH ...
    float S[KH];
    auto store_planes = [&]() {
#pragma unroll
      for (int c = 0; c < KH; c += 32) {
        uint32_t w[NPX][16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t s[NPX];
          split2<NPX>(S[c + 2 * i], S[c + 2 * i + 1], s);
#pragma unroll
          for (int p = 0; p < NPX; ++p) w[p][i] = s[p];
        }
#pragma unroll
        for (int p = 0; p < NPX; ++p)
          tmem_st16(lanes + CF::cSP + p * (KD / 2) + half * (KD / 4) + c / 2, w[p]);
      }
      tmem_wait_st();
    };
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    {
      const float* from = a.s_in && !STATES ? a.s_in + bh * a.s_in_head + step * a.s_in_seg : nullptr;
#pragma unroll
      for (int c = 0; c < KH; ++c) {
        const int kk = half * KH + c;
        S[c] = from && holds && vi < a.dv && kk < a.dk ? from[kk * a.sk + vi * a.sv] : 0.f;
      }
      if (!STATES) {
        if (holds) store_planes();
        tc5_fence_before();
        arrive(b_s);
      }
    }
    for (int n = 0; n < n_chunks; ++n) {
      const int s = n % ST;
      const int chunk = chunk_at(n), t0 = chunk * kLaChunk;
      const float* fac = fac_all + s * (4 * kLaChunk + 4);
      char* st = smem + s * CF::kStageBytes;
      const bool anchor_here = a.dump && ((chunk + 1) % a.anchor_chunks == 0 || chunk == all_chunks - 1);
      if (!STATES && a.reverse && anchor_here) {
        // <R, S> behind this chunk: R is the state here, S the forward pass's
        float sum = 0.f;
        const int64_t an = bh * a.anchors + chunk / a.anchor_chunks;
        if (holds) {
          const float* from = a.dump + (an * 8 + warp) * (KH * 32);
#pragma unroll
          for (int c = 0; c < KH; c += 4) {
            const float4 x = reinterpret_cast<const float4*>(from)[c / 4 * 32 + lane];
            sum += S[c] * x.x + S[c + 1] * x.y + S[c + 2] * x.z + S[c + 3] * x.w;
          }
        }
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
        if (lane == 0) a.anchor[an * 8 + warp] = sum;
      }
      la_wait(&b_full[s], (uint32_t)((n / ST) & 1), dead);
      if (!STATES && quad < 2) {
        // P = (Q K^T) . D, rows in the lanes
        la_wait(b_qk, (uint32_t)(n & 1), dead);
        tc5_fence_after();
        uint32_t x[32];
        tmem_ld32(x, lanes + CF::cQK + half * 32);
        tmem_wait_ld(x);
        const int row = quad * 32 + lane;
        const float ghi = fac[row], glo = fac[kLaChunk + row];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[NPX][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float p[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = u * 8 + i * 2 + e, j = half * 32 + c;
              const float d = (ghi - fac[j]) + (glo - fac[kLaChunk + j]);
              const float y = __uint_as_float(x[c]) * a.scale_p * ex2_approx(a.reverse ? -d : d);
              p[e] = (a.reverse ? j >= row : j <= row) ? y : 0.f;
            }
            uint32_t sp[NPX];
            split2<NPX>(p[0], p[1], sp);
#pragma unroll
            for (int q = 0; q < NPX; ++q) w[q][i] = sp[q];
          }
#pragma unroll
          for (int q = 0; q < NPX; ++q)
            *reinterpret_cast<uint4*>(smem + CF::kP + q * kLaBlock + tile_unit(row, half * 4 + u)) =
                make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
        }
        tc5_fence_before();
      } else {
        // the keys weighted by their decay to the chunk's end (reversed: start)
        const int me = STATES ? warp * 32 + lane : (half * 2 + quad - 2) * 32 + lane;
        constexpr int NT = STATES ? 256 : 128;
        for (int u = me; u < CF::KB * 512; u += NT) {
          const int row = (u % 512) / 8;
          const float wj = fac[3 * kLaChunk + row] * a.scale_w;
          const int off = (u / 512) * kLaBlock + row * kTileRow + (u % 8) * 16;
          uint32_t in[NPI][4];
#pragma unroll
          for (int p = 0; p < NPI; ++p) {
            const uint4 y = *reinterpret_cast<const uint4*>(st + CF::kK + p * CF::KB * kLaBlock + off);
            in[p][0] = y.x, in[p][1] = y.y, in[p][2] = y.z, in[p][3] = y.w;
          }
          uint32_t w[NPX][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int p = NPI - 1; p >= 0; --p) {  // the planes add up exactly from the smallest
              lo += __uint_as_float(in[p][i] << 16);
              hi += __uint_as_float(in[p][i] & 0xffff0000u);
            }
            uint32_t sp[NPX];
            split2<NPX>(lo * wj, hi * wj, sp);
#pragma unroll
            for (int p = 0; p < NPX; ++p) w[p][i] = sp[p];
          }
#pragma unroll
          for (int p = 0; p < NPX; ++p)
            *reinterpret_cast<uint4*>(smem + CF::kW + p * CF::KB * kLaBlock + off) =
                make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
        }
      }
      fence_proxy_async_smem();
      arrive(b_pk);

      la_wait(b_ds, (uint32_t)(n & 1), dead);
      tc5_fence_after();
      const float decay = fac[4 * kLaChunk];
      if (!STATES && holds) {
        uint32_t x1[32], x2[32];
        tmem_ld32(x1, lanes + CF::cO1 + half * 32);
        tmem_ld32(x2, lanes + CF::cO2 + half * 32);
        tmem_wait_ld(x1);
        tmem_wait_ld(x2);
        float o[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)
          o[c] = fmaf(__uint_as_float(x2[c]), fac[2 * kLaChunk + half * 32 + c] * a.scale_o, __uint_as_float(x1[c]));
        const int tb = t0 + half * 32;
        if (vi < a.dv) {
          const int64_t rs = (int64_t)a.heads * a.dv;
          const int64_t at = ((b * a.seqlen + tb) * a.heads + h) * a.dv + vi;
          if (sizeof(T) == 4 || a.out_f32) {
            float* to = static_cast<float*>(a.out) + at;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (tb + c < len && in_range(tb + c, a.seqlen)) to[c * rs] = o[c];
          } else {
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (tb + c < len && in_range(tb + c, a.seqlen)) to[c * rs] = __float2bfloat16_rn(o[c]);
          }
        }
        if (a.x.ptr) {
          const char* from = la_row(a.x, b, tb, h, sizeof(T)) + (int64_t)vi * sizeof(T);
          const int64_t rs = a.x.st * (int64_t)sizeof(T);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            o[c] = vi < a.dv && tb + c < len ? o[c] * to_f32(*reinterpret_cast<const T*>(from + c * rs)) : 0.f;
          const float sum = la_column_sums(o, lane);
          if (tb + lane < len) a.dots[(bh * a.seqlen + tb + lane) * 4 + quad] = sum;
        }
      } else if (!STATES && a.x.ptr && t0 + half * 32 + lane < len) {
        a.dots[(bh * a.seqlen + t0 + half * 32 + lane) * 4 + quad] = 0.f;
      }
      if (holds) {
#pragma unroll
        for (int c = 0; c < KH; c += 32) {
          uint32_t x[32];
          tmem_ld32(x, lanes + CF::cDS + half * KH + c);
          tmem_wait_ld(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) S[c + i] = fmaf(S[c + i], decay, __uint_as_float(x[i]));
        }
        if (!STATES && n + 1 < n_chunks) store_planes();
      }
      tc5_fence_before();
      arrive(&b_empty[s]);
      if (!STATES) arrive(b_s);
      if (!STATES && !a.reverse && anchor_here && holds) {
        const int64_t an = bh * a.anchors + chunk / a.anchor_chunks;
        float* to = a.dump + (an * 8 + warp) * (KH * 32);
#pragma unroll
        for (int c = 0; c < KH; c += 4)
          reinterpret_cast<float4*>(to)[c / 4 * 32 + lane] = make_float4(S[c], S[c + 1], S[c + 2], S[c + 3]);
      }
    }
    if (a.s_out && (STATES || step == a.nseg - 1) && holds && vi < a.dv) {
      float* to = a.s_out + bh * a.s_out_head + step * a.s_out_seg;
#pragma unroll
      for (int c = 0; c < KH; ++c) {
        const int kk = half * KH + c;
        if (kk < a.dk) to[kk * a.sk + vi * a.sv] = S[c];
      }
    }
  }
  // every MMA was waited for (b_ds of the last chunk) unless a wait gave up: then
  // this one, bounded too, stands between the MMAs in flight and the end
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  if (warp == CF::kComputeWarps) {
    if (*dead) {
      if (lane == 0) {
        mma_commit(b_qk);
        for (int i = 0; i < 1024 && !mbar_try_wait(b_qk, 0); ++i) {}
      }
      __syncwarp();
    }
    tmem_free(tmem, CF::kCols);
  }
}

// Segments joined: the state before each segment from the one before the first and
// what each adds, s <- e^{G} s + local, every element on its own.  `states` [bh][nseg]
// of dk x dv holds the local states and gets the starting ones.
__global__ void linattn_join_kernel(float* states, const double* seg_decay, const float* s0, int64_t s0_head,
                                    int nseg, int64_t per_state) {
  const int64_t bh = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= per_state) return;
  float s = s0 ? s0[bh * s0_head + i] : 0.f;
  float* at = states + bh * nseg * per_state + i;
  for (int n = 0; n < nseg; ++n) {
    const float local = n + 1 < nseg ? at[n * per_state] : 0.f;
    at[n * per_state] = s;
    if (n + 1 < nseg) s = fmaf(s, (float)exp2(seg_decay[bh * nseg + n]), local);
  }
}

// Gradients of shared heads: float partials [rows, heads, d] summed over the `share`
// heads that read one, in order.
template <typename T>
__global__ void linattn_share_kernel(const float* part, T* out, const int* lengths, int64_t seqlen, int64_t total,
                                     int heads, int share, int d) {
  const int groups = heads / share;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int c = (int)(i % d);
    const int gr = (int)(i / d % groups);
    const int64_t row = i / d / groups;
    if (lengths && row % seqlen >= lengths[row / seqlen]) continue;
    const float* p = part + (row * heads + (int64_t)gr * share) * d + c;
    float s = 0.f;
    for (int j = 0; j < share; ++j) s += p[(int64_t)j * d];
    if constexpr (sizeof(T) == 2) out[i] = __float2bfloat16_rn(s);
    else out[i] = s;
  }
}

// dg_t = sum_{s = t..e} (q_s . dq_s - k_s . dk_s) + <R_e, S_e>, e the next anchor at or
// behind t, R_e what the later tokens send back to the state S_e.  Each anchor's
// sums start anew, so that what cancels in the differences is no longer than the
// stretch between two.  One warp a stretch, from its end; sums in fp64.
template <typename T>
__global__ void linattn_decay_grad_kernel(const float* dots_q, const float* dots_k, const float* anchor, T* out,
                                          const int* lengths, int64_t bhs, int heads, int seqlen, int anchors,
                                          int anchor_tokens) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x % 32;
  const int64_t bh = w / anchors;
  const int an = (int)(w % anchors);
  if (bh >= bhs) return;
  const int64_t b = bh / heads;
  const int h = (int)(bh % heads);
  int len = lengths ? lengths[b] : seqlen;
  len = len < 0 ? 0 : len < seqlen ? len : seqlen;
  const int64_t begin = (int64_t)an * anchor_tokens;
  if (begin >= len) return;
  const int end = begin + anchor_tokens < len ? (int)(begin + anchor_tokens) : len;
  double carry = 0.0;
  for (int i = 0; i < 8; ++i) carry += anchor[(bh * anchors + an) * 8 + i];
  for (int hi = end; hi > begin; hi -= 32) {
    const int t = hi - 1 - lane;  // lane 0 the latest
    double x = 0.0;
    if (t >= begin) {
      const float4 q = reinterpret_cast<const float4*>(dots_q)[bh * seqlen + t];
      const float4 k = reinterpret_cast<const float4*>(dots_k)[bh * seqlen + t];
      x = ((double)q.x + q.y + q.z + q.w) - ((double)k.x + k.y + k.z + k.w);
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const double up = __shfl_up_sync(kFullMask, x, o);
      if (lane >= o) x += up;
    }
    x += carry;
    if (t >= begin) {
      const float y = (float)x;
      T* to = out + (b * seqlen + t) * heads + h;
      if constexpr (sizeof(T) == 2) *to = __float2bfloat16_rn(y);
      else *to = y;
    }
    carry = __shfl_sync(kFullMask, x, 31);
  }
}

}  // namespace ssscan

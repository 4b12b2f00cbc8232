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
// registers.  Running sums of the decays are whole numbers of 2^-32.
//
// Layout.  Scores are Q K^T with tokens in the lanes.  O and S are kept transposed
// (value index in the lanes), so that S^T is the MMA's A operand straight from
// tensor memory: it is written there by the threads that hold it and never goes
// through shared memory.  M is 128 there; where values are 64 wide the other lanes
// hold sums of whatever follows in shared memory and nobody reads them.
//
// Roles.  Loaders (two warps) fill rings of K, V and Q tiles, one warp works out the
// decays, one thread issues the MMAs; the front warps (eight) turn scores into P and
// keys into weighted keys one chunk ahead of the back warps (sixteen), which hold the
// state: they take O and the state's increment from tensor memory, give the state
// back as planes, and write O out while the next chunk's products run.
//
// Schedule.  A head's chunks depend on one another through S alone.  With fewer heads
// than SMs the sequence is cut into segments whose starting states a first launch
// works out (STATES).  With more, every CTA takes an equal range of the chunks of all
// heads laid end to end; a head cut between two CTAs is begun by the first of them
// before anything else and carried on by the second after all else, so the state
// handed over is there when it is needed.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "scan_common.cuh"
#include "tc5.cuh"

namespace ssscan {

constexpr int kLaChunk = 64;
constexpr int kLaBlock = kLaChunk * kTileRow;  // bytes of one plane's 64 x 64 block
constexpr uint32_t kLaSpinLimit = 1u << 9;        // polls of a barrier: a few seconds
constexpr uint32_t kLaCarrySpinLimit = 1u << 24;  // of the previous worker's flag: likewise

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
  float* dots;          // [batch * heads, seqlen, 4] partial products of x, one a lane quadrant
  float* dump;          // forward: where the states at anchors go; reversed: where they come from
  float* anchor;        // reversed: [batch * heads, anchors, 16] partial products <R, S>, one a back warp
  int anchor_chunks;    // an anchor behind every so many chunks
  int anchors;          // anchors of the longest row
  int heads, seqlen, dk, dv;
  int bh;               // batch * heads
  int nseg, seg_chunks; // segments of a head, or
  int workers;          // > 0: CTAs that share all chunks evenly
  float* carry;         // [workers] states handed to the next worker
  unsigned* flags;      // [0] hands out worker numbers, then [workers][16] one a back warp; zero at launch
  int reverse;
  int vec;              // 16-byte loads apply to q, k and v
  int out_vec;          // 16-byte stores to out
  int tma;              // so do the tensor maps
  float scale_p, scale_o, scale_w;
};

struct LaMaps {
  CUtensorMap q, k, v;
};

template <typename T, int KD, int VD>
struct LaCfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPI = kBf16 ? 1 : 3;  // planes of the inputs
  static constexpr int NPX = kBf16 ? 2 : 3;  // planes of the scores and of the state as operands
  static constexpr int NPW = 3;              // planes of the weighted keys
  static constexpr int KB = KD / 64, VB = VD / 64;
  // Tiles in each ring.  A key tile lives until its chunk's increment is formed (the
  // weighted keys' first planes replace it in place), a query tile until S Q is.
  static constexpr int RK = kBf16 ? 3 : 2, RQ = kBf16 ? 3 : 1, RV = kBf16 ? (KB == 2 && VB == 2 ? 2 : 3) : 1;
  static constexpr int RW = 2;               // the weighted keys' further planes
  static constexpr int RF = 4;               // decays
  static constexpr int kRing = 4;
  static_assert(RK <= kRing && RV <= kRing && RQ <= kRing && RF <= kRing, "barriers of a ring");
  static constexpr int kTileK = KB * NPI * kLaBlock, kTileV = VB * NPI * kLaBlock, kTileW = KB * (NPW - NPI) * kLaBlock;
  static constexpr int kQ = 0, kK = RQ * kTileK, kV = kK + RK * kTileK, kP = kV + RV * kTileV;
  static constexpr int kW = kP + NPX * kLaBlock;
  static constexpr int kFacFloats = 4 * kLaChunk + 4;
  static constexpr int kFac = kW + RW * kTileW;
  static constexpr int kStage = kFac + (RF * kFacFloats * 4 + 127) / 128 * 128;  // 512 bytes a back warp
  static constexpr int kBars = kStage + (kBf16 ? 16 * 512 : 0);
  static constexpr int kSmem = kBars + (8 * kRing + 8) * 8 + 16;
  // tensor memory columns
  static constexpr int cDS = 0, cSP = KD, cO1 = cSP + NPX * KD / 2, cO2 = cO1 + 64, cQK = cO2 + 64;
  static constexpr int kAhead = kBf16 ? 2 : 1;  // chunks that scores run ahead, one place for each
  static constexpr int kCols = cQK + 64 * kAhead <= 256 ? 256 : 512;
  static_assert(cQK + 64 * kAhead <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr int kQuads = VD / 32;        // lane quadrants that hold values
  static constexpr int kHolders = 4 * kQuads;   // back warps at work
  static constexpr int kLoaders = 64;           // loader threads
  static constexpr int kThreads = 896;
};
constexpr int kLaBackWarps = 16, kLaFrontWarps = 8;
constexpr int kLaMmaWarp = 24, kLaLoadWarp = 25, kLaDecayWarp = 27;
// registers a thread of the three kinds of warpgroup: 4 x 88 + 2 x 56 + 40 = 7 x 72 at launch
constexpr int kLaBackRegs = 88, kLaFrontRegs = 56, kLaAuxRegs = 40;

// Waits of one CTA: when one gives up, the others stop waiting too, and the kernel
// runs to its end on whatever is there, inside its buffers.  A poll may suspend the
// thread for up to 10 ms, so that those that wait leave the issue slots to the others.
__device__ __forceinline__ void la_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
#pragma unroll 1
  for (uint32_t i = 0; i < kLaSpinLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(10000000)
        : "memory");
    if (ok || *dead) return;
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
#pragma unroll 1
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
        split2<3>(pair(f[2 * i], f[2 * i + 1]), s);
        w[0][i] = s[0], w[1][i] = s[1], w[2][i] = s[2];
      }
#pragma unroll
      for (int p3 = 0; p3 < 3; ++p3)
        *reinterpret_cast<uint4*>(to + p3 * B * kLaBlock) = make_uint4(w[p3][0], w[p3][1], w[p3][2], w[p3][3]);
    }
  }
}

// A lane's two log decays of a chunk as they are stored, zero behind the row's end.
template <typename T>
__device__ __forceinline__ void la_fetch_decays(T (&x)[2], const LaPassArgs& a, int b, int h, int t0, int len, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = t0 + 2 * lane + i;
    x[i] = zero_elem<T>();
    if (t < len && in_range(t, len)) x[i] = *reinterpret_cast<const T*>(la_row(a.g, b, t, h, sizeof(T)));
  }
}

// 2^x of a number with 32 bits behind the point: the fraction by ex2, the integer
// through the exponent; what is below the normal numbers is zero, as ex2 has it.
__device__ __forceinline__ float la_exp2(int64_t x) {
  const int n = (int)(x >> 32);
  const float y = ex2_approx((float)(uint32_t)x * 0x1p-32f);  // 1 to 2
  const float z = y * __int_as_float((n + 127) << 23);
  return n < -126 ? 0.f : n > 127 ? __int_as_float(0x7f800000) : z;
}

// A chunk's decays: running sums, base 2, as integer and fraction, the factors of the
// rows and of the keys, and the chunk's whole decay, which is returned.  One warp, two
// tokens a lane.  The sums are whole numbers of 2^-32, so differences of large sums
// lose nothing.  A log decay beyond +-1400 leaves nothing, or too much, in fp32 and is
// taken as that: minus infinity (a reset) is a number like any other here.
__device__ __forceinline__ int64_t la_decays(float* fac, float x0, float x1, bool reverse, float scale_o, float scale_w,
                                             int lane) {
  const float x[2] = {x0, x1};
  int64_t g[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    g[i] = __double2ll_rn((double)fminf(fmaxf(x[i], -1400.f), 1400.f) * (1.4426950408889634 * 4294967296.0));
  int64_t sum = g[0] + g[1];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t up = __shfl_up_sync(kFullMask, sum, o);
    if (lane >= o) sum += up;
  }
  const int64_t total = __shfl_sync(kFullMask, sum, 31);
  const int64_t at[2] = {sum - g[1], sum};
  // a NaN among them is not to vanish
  const float bad = __any_sync(kFullMask, x0 != x0 || x1 != x1) ? __int_as_float(0x7fffffff) : 1.f;
  float2 hi, lo, rows, keys;
  float* out[4] = {&hi.x, &lo.x, &rows.x, &keys.x};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float from_start = la_exp2(at[i]), to_end = la_exp2(total - at[i]);
    out[0][i] = (float)(int)(at[i] >> 32);
    out[1][i] = (float)(uint32_t)at[i] * 0x1p-32f * bad;
    out[2][i] = (reverse ? to_end : from_start) * scale_o * bad;
    out[3][i] = (reverse ? from_start : to_end) * scale_w * bad;
  }
  reinterpret_cast<float2*>(fac)[lane] = hi;
  reinterpret_cast<float2*>(fac + kLaChunk)[lane] = lo;
  reinterpret_cast<float2*>(fac + 2 * kLaChunk)[lane] = rows;
  reinterpret_cast<float2*>(fac + 3 * kLaChunk)[lane] = keys;
  if (lane == 0) fac[4 * kLaChunk] = la_exp2(total) * bad;
  return total;
}

template <int N>
struct LaWidth {
  static constexpr int value = N;
};

// 32 values x 16 tokens of a back warp to the output, and their products with the
// rows of x.  o[h][4 i + z]: value v0 + 16 h + 8 (z / 2) + lane / 4, token
// t0 + 8 i + 2 (lane % 4) + z % 2.  bf16 rows go through 512 bytes of shared memory, 8
// tokens at a time, so that a token's 32 values leave as 64 bytes in 16-byte stores.
template <typename T>
__device__ __forceinline__ void la_emit(const LaPassArgs& a, const float (&o)[2][8], char* stage, int64_t b, int64_t bh,
                                        int h, int t0, int len, int v0, int quad, int lane) {
  const int64_t rs = (int64_t)a.heads * a.dv;
  const int64_t at = ((b * a.seqlen + t0) * a.heads + h) * a.dv + v0;
  if (sizeof(T) == 2 && !a.out_f32 && a.out_vec) {
    const uint32_t to = smem_u32(stage) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
    const int tok = lane / 4, c = lane % 4;
    const char* from = stage + tok * 64 + ((c ^ ((tok >> 1) & 3)) << 4);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + at + tok * rs + c * 8;
    const bool mine = v0 + c * 8 < a.dv;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      store_blocks_t(to, to_bf16x2(o[0][4 * i], o[0][4 * i + 1]), to_bf16x2(o[0][4 * i + 2], o[0][4 * i + 3]),
                     to_bf16x2(o[1][4 * i], o[1][4 * i + 1]), to_bf16x2(o[1][4 * i + 2], o[1][4 * i + 3]));
      __syncwarp();
      const uint4 y = *reinterpret_cast<const uint4*>(from);
      const int t = t0 + i * 8 + tok;
      if (mine && t < len && in_range(t, a.seqlen)) *reinterpret_cast<uint4*>(out + i * 8 * rs) = y;
      __syncwarp();
    }
  } else {
    const int v = v0 + lane / 4, t = t0 + 2 * (lane % 4);
    const int64_t mine = at + lane / 4 + 2 * (lane % 4) * rs;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int64_t row = mine + (8 * i + z) * rs;
        if (t + 8 * i + z < len && in_range(t + 8 * i + z, a.seqlen)) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (v + 8 * u < a.dv) {
              const float y = o[u / 2][4 * i + 2 * (u % 2) + z];
              if (sizeof(T) == 4 || a.out_f32) static_cast<float*>(a.out)[row + 8 * u] = y;
              else static_cast<__nv_bfloat16*>(a.out)[row + 8 * u] = __float2bfloat16_rn(y);
            }
        }
      }
  }
  if (a.x.ptr) {
    const int v = v0 + lane / 4, t = t0 + 2 * (lane % 4);
    const char* from = la_row(a.x, b, t, h, sizeof(T)) + (int64_t)v * sizeof(T);
    const int64_t xs = a.x.st * (int64_t)sizeof(T);
    float sum[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float y = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (t + 8 * i + z < len && v + 8 * u < a.dv)
            y = fmaf(o[u / 2][4 * i + 2 * (u % 2) + z],
                     to_f32(reinterpret_cast<const T*>(from + (8 * i + z) * xs)[8 * u]), y);
        sum[2 * i + z] = y;
      }
    // the lanes with the same tokens are 4, 8 and 16 apart
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int m = 4; m <= 16; m *= 2) sum[s] += __shfl_xor_sync(kFullMask, sum[s], m);
    if (lane < 4) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int tt = t + 8 * (s / 2) + s % 2;
        if (tt < len) a.dots[(bh * a.seqlen + tt) * 4 + quad] = sum[s];
      }
    }
  }
}

// The products of planes pa < PA of one operand and pb < PB of the other whose
// weight counts, the smaller ones first: they add up while the sum is small.  STEPS
// MMAs each, given the planes' places (in descriptor units: blocks of a plane, or
// `a_cols` columns).  The loop over planes stays one: the roles together have to fit
// the instruction cache.
template <int PA, int PB, int STEPS, typename F>
__device__ __forceinline__ void la_products(int a_blocks, int b_blocks, F&& mma, int a_cols = 0) {
  constexpr int P = PA > PB ? PA : PB;
  bool add = false;
#pragma unroll 1
  for (int pa = PA - 1; pa >= 0; --pa)
#pragma unroll 1
    for (int pb = (P - pa < PB ? P - pa : PB) - 1; pb >= 0; --pb) {
      const int at_a = pa * (a_blocks * (kLaBlock >> 4) + a_cols), at_b = pb * b_blocks * (kLaBlock >> 4);
#pragma unroll
      for (int i = 0; i < STEPS; ++i) mma(at_a, at_b, i, add || i > 0);
      add = true;
    }
}

// What one CTA works through: pieces of heads, in the order of processing.
struct LaPiece {
  int bh, b, h, len;
  int first, last;   // real chunks [first, last), whichever way they are run
  bool from_carry;   // starts from the previous worker's state
  bool to_carry;     // ends inside its head
};
struct LaWork {
  int worker, n, pieces;   // chunks of a whole head
  int h0, c0, h1, c1;      // from chunk c0 of head h0 to before chunk c1 of head h1
};
__device__ __forceinline__ LaWork la_work(const LaPassArgs& a, int worker) {
  LaWork w;
  w.worker = worker;
  w.n = (a.seqlen + kLaChunk - 1) / kLaChunk;
  if (a.workers > 0) {
    const int64_t total = (int64_t)a.bh * w.n, lo = total * worker / a.workers, hi = total * (worker + 1) / a.workers;
    w.h0 = (int)(lo / w.n), w.c0 = (int)(lo - (int64_t)w.h0 * w.n);
    w.h1 = (int)(hi / w.n), w.c1 = (int)(hi - (int64_t)w.h1 * w.n);
    w.pieces = w.h1 - w.h0 + (w.c1 > 0);  // a range is at least a head long
  } else {
    w.h0 = w.h1 = worker / a.nseg;
    const int step = worker - w.h0 * a.nseg;
    const int64_t p0 = (int64_t)step * a.seg_chunks, p1 = p0 + a.seg_chunks;
    w.c0 = (int)(p0 < w.n ? p0 : w.n);
    w.c1 = (int)(p1 < w.n ? p1 : w.n);
    w.pieces = 1;
  }
  return w;
}
__device__ __forceinline__ LaPiece la_piece(const LaPassArgs& a, const LaWork& w, int i) {
  LaPiece p;
  int p0 = 0, p1 = w.n;  // places in the order of processing, padded
  p.from_carry = p.to_carry = false;
  if (a.workers > 0) {
    // the head that the next worker goes on with comes first, the one that the
    // previous worker began comes last
    const int tail = w.c1 > 0;
    p.bh = w.h0 + (w.c0 > 0) + i - tail;
    if (tail && i == 0) p.bh = w.h1, p1 = w.c1, p.to_carry = true;
    else if (p.bh >= w.h1) p.bh = w.h0, p0 = w.c0, p.from_carry = true;
  } else {
    p.bh = w.h0, p0 = w.c0, p1 = w.c1;
  }
  p.b = p.bh / a.heads;
  p.h = p.bh - p.b * a.heads;
  p.len = la_length(a, p.b);
  const int all = (p.len + kLaChunk - 1) / kLaChunk;
  const int f = a.reverse ? w.n - p1 : p0, l = a.reverse ? w.n - p0 : p1;
  p.first = f < all ? f : all;
  p.last = l < all ? l : all;
  return p;
}

// STATES: only the states (the sequence's segments, each from zero, all at once).
template <typename T, int KD, int VD, bool STATES>
__global__ void __launch_bounds__(LaCfg<T, KD, VD>::kThreads, 1)
linattn_pass_kernel(const __grid_constant__ LaPassArgs a, const __grid_constant__ LaMaps maps) {
  using CF = LaCfg<T, KD, VD>;
  constexpr int NPI = CF::NPI, NPX = CF::NPX, NPW = CF::NPW;
  extern __shared__ __align__(1024) char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + CF::kBars);
  // a ring's barriers: CF::kRing slots each, whatever its length
  uint64_t *full_k = bars, *empty_k = full_k + CF::kRing, *full_v = empty_k + CF::kRing, *empty_v = full_v + CF::kRing,
           *full_q = empty_v + CF::kRing, *empty_q = full_q + CF::kRing, *full_f = empty_q + CF::kRing,
           *empty_f = full_f + CF::kRing, *single = empty_f + CF::kRing;
  uint64_t *b_qk = single + 6;    // scores are there, one for each place
  uint64_t *b_pk = single + 1;    // P and the weighted keys are there
  uint64_t *b_ds = single + 2;    // increment and P V are there
  uint64_t *b_o = single + 3;     // S Q too: the chunk's products are done
  uint64_t *b_free = single + 4;  // the back warps have read them
  uint64_t *b_s = single + 5;     // the state's planes are there
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(single + 8);
  int* worker_at = reinterpret_cast<int*>(tmem_at + 1);
  volatile int* dead = worker_at + 1;

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    for (int i = 0; i < CF::RK; ++i) mbar_init(&full_k[i], 1), mbar_init(&empty_k[i], 1);
    for (int i = 0; i < CF::RV; ++i) mbar_init(&full_v[i], 1), mbar_init(&empty_v[i], 1);
    for (int i = 0; i < CF::RQ; ++i) mbar_init(&full_q[i], 1), mbar_init(&empty_q[i], 1);
    for (int i = 0; i < CF::RF; ++i) mbar_init(&full_f[i], 1), mbar_init(&empty_f[i], kLaFrontWarps + CF::kHolders);
    for (int i = 0; i < 2; ++i) mbar_init(&b_qk[i], 1);
    mbar_init(single, 1);
    mbar_init(b_pk, kLaFrontWarps);
    mbar_init(b_ds, 1);
    mbar_init(b_o, 1);
    mbar_init(b_free, CF::kHolders);
    mbar_init(b_s, CF::kHolders);
    fence_mbar_init();
    *dead = 0;
    // workers are numbered in the order in which they start, so that the one a
    // worker may wait for is running
    *worker_at = a.workers > 0 ? (int)atomicAdd(a.flags, 1u) : (int)blockIdx.x;
  }
  if (warp == kLaMmaWarp) tmem_alloc(tmem_at, CF::kCols);
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  const uint32_t tmem = *tmem_at;
  const LaWork work = la_work(a, *worker_at);
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp >= kLaMmaWarp) {
    regs_give<kLaAuxRegs>();
    if (warp == kLaMmaWarp) {
      // ---- MMA issue, by one thread of the warp
      const uint32_t base = smem_u32(smem);
      const bool leader = elect_one();
      auto scores = [&](int n) {
        la_wait(&full_k[n % CF::RK], (uint32_t)((n / CF::RK) & 1), dead);
        la_wait(&full_q[n % CF::RQ], (uint32_t)((n / CF::RQ) & 1), dead);
        tc5_fence_after();
        if (leader) {
          const uint64_t q = tile_desc(base + CF::kQ + (n % CF::RQ) * CF::kTileK, 0);
          const uint64_t k = tile_desc(base + CF::kK + (n % CF::RK) * CF::kTileK, 0);
          la_products<NPI, NPI, KD / 16>(CF::KB, CF::KB, [&](int pa, int pb, int i, bool add) {
            const int off = (i / 4) * (kLaBlock >> 4) + (i % 4) * 2;
            mma_ss(tmem + CF::cQK + (n % CF::kAhead) * 64, q + pa + off, k + pb + off, mma_idesc(64, 64, false, false), add);
          });
          mma_commit(&b_qk[n % CF::kAhead]);
        }
        __syncwarp();
      };
      int total = 0, scored = 0;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        total += p.last - p.first;
      }
      if (!STATES)
        while (scored < CF::kAhead && scored < total) scores(scored++);
      for (int n = 0; n < total; ++n) {
        const uint64_t v = tile_desc(base + CF::kV + (n % CF::RV) * CF::kTileV, kLaBlock);
        // planes of the weighted keys: in the key tile's place, then in a ring of their own
        const uint64_t w0 = tile_desc(base + CF::kK + (n % CF::RK) * CF::kTileK, kLaBlock);
        const uint64_t w1 = tile_desc(base + CF::kW + (n % CF::RW) * CF::kTileW, kLaBlock) -
                            (uint64_t)(NPI * CF::KB * (kLaBlock >> 4));
        la_wait(b_pk, (uint32_t)(n & 1), dead);
        tc5_fence_after();
        la_wait(&full_v[n % CF::RV], (uint32_t)((n / CF::RV) & 1), dead);
        if (n > 0) la_wait(b_free, (uint32_t)((n - 1) & 1), dead);
        tc5_fence_after();
        if (leader) {
          // dS^T = V^T (w . K)
          la_products<NPI, NPW, kLaChunk / 16>(CF::VB, CF::KB, [&](int pa, int pb, int i, bool add) {
            const int off = i * (16 * kTileRow >> 4);
            mma_ss(tmem + CF::cDS, v + pa + off, (pb < NPI * CF::KB * (kLaBlock >> 4) ? w0 : w1) + pb + off,
                   mma_idesc(128, KD, true, true), add);
          });
          if (!STATES) {
            // O1^T = V^T P^T
            const uint64_t pd = tile_desc(base + CF::kP, 0);
            la_products<NPI, NPX, kLaChunk / 16>(CF::VB, 1, [&](int pa, int pb, int i, bool add) {
              mma_ss(tmem + CF::cO1, v + pa + i * (16 * kTileRow >> 4), pd + pb + i * 2, mma_idesc(128, 64, true, false), add);
            });
          }
          mma_commit(b_ds);
          mma_commit(&empty_v[n % CF::RV]);
          mma_commit(&empty_k[n % CF::RK]);
        }
        __syncwarp();
        if (!STATES) {
          // O2^T = S^T Q^T
          la_wait(b_s, (uint32_t)(n & 1), dead);
          tc5_fence_after();
          if (leader) {
            const uint64_t q = tile_desc(base + CF::kQ + (n % CF::RQ) * CF::kTileK, 0);
            la_products<NPX, NPI, KD / 16>(0, CF::KB, [&](int pa, int pb, int i, bool add) {
              mma_ts(tmem + CF::cO2, tmem + CF::cSP + pa + i * 8, q + pb + (i / 4) * (kLaBlock >> 4) + (i % 4) * 2,
                     mma_idesc(128, 64, false, false), add);
            }, KD / 2);
            mma_commit(b_o);
            mma_commit(&empty_q[n % CF::RQ]);
          }
          __syncwarp();
          // last, so that no tile is waited for while the chunk's own products could run
          if (scored < total) scores(scored++);
        }
      }
    } else if (warp == kLaDecayWarp) {
      // ---- decays
      int n = 0;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        double sum = 0.0;
        auto place = [&](int c) { return (a.reverse ? p.last - 1 - (c - p.first) : c) * kLaChunk; };
        T next[2];
        if (p.first < p.last) la_fetch_decays<T>(next, a, p.b, p.h, place(p.first), p.len, lane);
        for (int c = p.first; c < p.last; ++c, ++n) {
          const int s = (int)(n % CF::RF);
          const float x0 = to_f32(next[0]), x1 = to_f32(next[1]);
          if (c + 1 < p.last) la_fetch_decays<T>(next, a, p.b, p.h, place(c + 1), p.len, lane);
          if (n >= CF::RF) la_wait(&empty_f[s], (uint32_t)((n / CF::RF - 1) & 1), dead);
          const int64_t whole = la_decays(reinterpret_cast<float*>(smem + CF::kFac) + s * CF::kFacFloats, x0, x1,
                                          a.reverse, a.scale_o, a.scale_w, lane);
          if (STATES) sum += (double)whole * 0x1p-32;
          arrive(&full_f[s]);
        }
        if (STATES && lane == 0) a.seg_decay[(int64_t)p.bh * (a.nseg + 1) + work.worker % a.nseg] = sum;
      }
    } else {
      // ---- loaders: one thread by TMA, or all of them
      const int ltid = tid - 32 * kLaLoadWarp;
      int n = 0;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        for (int c = p.first; c < p.last; ++c, ++n) {
          const int t0 = (a.reverse ? p.last - 1 - (c - p.first) : c) * kLaChunk;
          // TMA clips at the tensor's end, not at a row's length
          const bool by_tma = CF::kBf16 && a.tma && (t0 + kLaChunk <= p.len || p.len == a.seqlen);
          auto tile = [&](auto width, const LaTensor& x, const CUtensorMap* map, int ring, int at, int bytes,
                          uint64_t* full, uint64_t* empty, int d) {
            constexpr int DP = decltype(width)::value;
            const int s = n % ring;
            char* to = smem + at + s * bytes;
            if (ltid == 0 && n >= ring) la_wait(&empty[s], (uint32_t)((n / ring - 1) & 1), dead);
            if (by_tma) {
              if (ltid == 0) {
                mbar_arrive_expect_tx(&full[s], DP / 64 * kLaBlock);
#pragma unroll 1
                for (int j = 0; j < DP / 64; ++j)
                  tma_load_block(to + j * kLaBlock, map, &full[s], j * 64, t0, p.h / x.share, p.b);
              }
            } else {
              __syncwarp();
              asm volatile("bar.sync 2, 64;\n" ::: "memory");
              la_load_tile<T, DP>(to, x, p.b, p.h, t0, p.len, d, a.vec, ltid, CF::kLoaders);
              if (CF::kBf16 && a.vec) {
                cp_async_commit();
                cp_async_wait_all();
              }
              fence_proxy_async_smem();
              __syncwarp();
              asm volatile("bar.sync 2, 64;\n" ::: "memory");
              if (ltid == 0) mbar_arrive(&full[s]);
            }
          };
          tile(LaWidth<KD>{}, a.k, &maps.k, CF::RK, CF::kK, CF::kTileK, full_k, empty_k, a.dk);
          if (!STATES) tile(LaWidth<KD>{}, a.q, &maps.q, CF::RQ, CF::kQ, CF::kTileK, full_q, empty_q, a.dk);
          tile(LaWidth<VD>{}, a.v, &maps.v, CF::RV, CF::kV, CF::kTileV, full_v, empty_v, a.dv);
        }
      }
    }
  } else if (warp >= kLaBackWarps) {
    // ---- front: weighted keys and P, a chunk ahead of the back
    regs_give<kLaFrontRegs>();
    // 16 rows of P for each pair of warps, side 0 with every other block of columns
    const int fw = warp % 4, side = (warp - kLaBackWarps) / 4, ftid = tid - 32 * kLaBackWarps;
    int n = 0;
    // Shares of the 32 or 16 steps of a key tile.  A warp's rows of P have none to two
    // blocks of 16 columns under the mask, each about as much work as one and a half
    // steps: where they have fewer, the share of the steps is larger.  Byte i is where
    // the share of the i-th warp begins, in the order of rows (reversed: from the last).
    const int at = 2 * (a.reverse ? 3 - fw : fw) + side;
    const uint64_t begins = STATES ? (CF::KB == 2 ? 0x1c1814100c080400ull : 0x0e0c0a0806040200ull)
                                   : (CF::KB == 2 ? 0x1d1a16130f0a0400ull : 0x0f0e0c0b09060200ull);
    const int w_from = (int)(begins >> (8 * at)) & 0xff;
    const int w_to = at == 7 ? CF::KB * 16 : (int)(begins >> (8 * at + 8)) & 0xff;
    if (!STATES) {
      // what the mask takes away is zero once and for all
      for (int i = ftid; i < NPX * kLaBlock / 16; i += 32 * kLaFrontWarps)
        reinterpret_cast<uint4*>(smem + CF::kP)[i] = make_uint4(0, 0, 0, 0);
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
    }
    for (int i = 0; i < work.pieces; ++i) {
      const LaPiece p = la_piece(a, work, i);
      for (int c = p.first; c < p.last; ++c, ++n) {
        const float* fac = reinterpret_cast<const float*>(smem + CF::kFac) + (int)(n % CF::RF) * CF::kFacFloats;
        la_wait(&full_f[n % CF::RF], (uint32_t)((n / CF::RF) & 1), dead);
        la_wait(&full_k[n % CF::RK], (uint32_t)((n / CF::RK) & 1), dead);
        if (!STATES) la_wait(&b_qk[n % CF::kAhead], (uint32_t)((n / CF::kAhead) & 1), dead);  // the keys as they are were used
        {
          // the keys weighted by their decay to the chunk's end (reversed: start)
          char* k = smem + CF::kK + (n % CF::RK) * CF::kTileK;
          char* w = smem + CF::kW + (n % CF::RW) * CF::kTileW;
#pragma unroll 2
          for (int u = w_from * 32 + lane; u < w_to * 32; u += 32) {
            const int row = (u % 512) / 8;
            const float wj = fac[3 * kLaChunk + row];
            const uint64_t ww = pair(wj, wj);
            const int off = (u / 512) * kLaBlock + row * kTileRow + (u % 8) * 16;
            uint32_t in[NPI][4];
#pragma unroll
            for (int q = 0; q < NPI; ++q) {
              const uint4 y = *reinterpret_cast<const uint4*>(k + q * CF::KB * kLaBlock + off);
              in[q][0] = y.x, in[q][1] = y.y, in[q][2] = y.z, in[q][3] = y.w;
            }
            uint32_t out[NPW][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint64_t y = from_bf16x2(in[NPI - 1][e]);
#pragma unroll
              for (int q = NPI - 2; q >= 0; --q) y = add2(y, from_bf16x2(in[q][e]));  // exact from the smallest
              uint32_t sp[NPW];
              split2<NPW>(mul2(y, ww), sp);
#pragma unroll
              for (int q = 0; q < NPW; ++q) out[q][e] = sp[q];
            }
#pragma unroll
            for (int q = 0; q < NPW; ++q)
              *reinterpret_cast<uint4*>((q < NPI ? k + q * CF::KB * kLaBlock : w + (q - NPI) * CF::KB * kLaBlock) + off) =
                  make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
          }
        }
        // the last chunk's products are done: P may be overwritten, and what is made here
        // is never two chunks ahead
        if (n > 0) la_wait(b_ds, (uint32_t)((n - 1) & 1), dead);
        if (!STATES) {
          // P = (Q K^T) . D: 16 rows a warp, two rows a thread
          tc5_fence_after();
          const int r0 = fw * 16 + lane / 4;
          const float sign = a.reverse ? -1.f : 1.f;
          const float h0 = fac[r0], l0 = fac[kLaChunk + r0], h1 = fac[r0 + 8], l1 = fac[kLaChunk + r0 + 8];
          const uint64_t hh[2] = {pair(h0, h0), pair(h1, h1)}, ll[2] = {pair(l0, l0), pair(l1, l1)};
          const uint64_t minus = pair(-1.f, -1.f), sp2 = pair(a.scale_p, a.scale_p);
          const int c0 = 2 * (lane % 4);
          // this lane's row address for store_blocks: blocks (rows 0-7, 8-15) x two column blocks
          const int srow = fw * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
          // 16 columns at a time, those that the mask leaves (the others stay zero)
          const int from = a.reverse ? fw : 0, to = a.reverse ? 4 : fw + 1;
#pragma unroll 1
          for (int cb = from + side; cb < to; cb += 2) {
            uint32_t x[8];
            tmem_ld_rows16(x, tmem + ((uint32_t)(fw * 32) << 16) + CF::cQK + (n % CF::kAhead) * 64 + cb * 16);
            uint64_t gh[2], gl[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              gh[e] = *reinterpret_cast<const uint64_t*>(fac + cb * 16 + e * 8 + c0);
              gl[e] = *reinterpret_cast<const uint64_t*>(fac + kLaChunk + cb * 16 + e * 8 + c0);
            }
            tmem_wait_ld(x);
            uint32_t o[NPX][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint64_t d = add2(fma2(gh[e], minus, hh[z]), fma2(gl[e], minus, ll[z]));
                const uint64_t f = pair(ex2_approx(pair_lo(d) * sign), ex2_approx(pair_hi(d) * sign));
                uint64_t y = mul2(mul2(pair(x[4 * e + 2 * z], x[4 * e + 2 * z + 1]), sp2), f);
                if (cb == fw) {
                  const int row = lane / 4 + 8 * z, col = 8 * e + c0;
                  y = pair((a.reverse ? col >= row : col <= row) ? pair_lo(y) : 0.f,
                           (a.reverse ? col + 1 >= row : col + 1 <= row) ? pair_hi(y) : 0.f);
                }
                uint32_t sp[NPX];
                split2<NPX>(y, sp);
#pragma unroll
                for (int q = 0; q < NPX; ++q) o[q][e * 2 + z] = sp[q];
              }
#pragma unroll
            for (int q = 0; q < NPX; ++q)
              store_blocks(smem_u32(smem) + CF::kP + q * kLaBlock + tile_unit(srow, cb * 2 + (lane >> 4)), o[q][0], o[q][1],
                           o[q][2], o[q][3]);
          }
          tc5_fence_before();
        }
        fence_proxy_async_smem();
        arrive(b_pk);
        arrive(&empty_f[n % CF::RF]);
      }
    }
  } else {
    // ---- back: the state and the outputs
    regs_take<kLaBackRegs>();
    const int quad = warp % 4, part = warp / 4;  // value lanes; a quarter of the keys and tokens
    if (quad < CF::kQuads) {
      const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
      const int vi = quad * 32 + lane;          // this thread's value index
      constexpr int KH = KD / 4;                // its key indices: part * KH ...
      uint64_t S[KH / 2];                       // in pairs
      auto store_planes = [&]() {
#pragma unroll
        for (int c = 0; c < KH / 2; c += 8) {
          uint32_t w[NPX][8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t s[NPX];
            split2<NPX>(S[c + i], s);
#pragma unroll
            for (int p = 0; p < NPX; ++p) w[p][i] = s[p];
          }
#pragma unroll
          for (int p = 0; p < NPX; ++p) tmem_st(lanes + CF::cSP + p * (KD / 2) + part * (KH / 2) + c, w[p]);
        }
        tmem_wait_st();
      };
      int n = 0;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        const int64_t bh = p.bh;
        const int b = p.b, h = p.h, len = p.len;
        const int all_chunks = (len + kLaChunk - 1) / kLaChunk;
        const int step = a.workers > 0 ? 0 : work.worker % a.nseg;
        if (p.from_carry) {
          const unsigned* flag = a.flags + 1 + (work.worker - 1) * 16 + warp;
          if (lane == 0) {
            unsigned there = 0;
            for (uint32_t spin = 0; spin < kLaCarrySpinLimit && !there && !*dead; ++spin) {
              asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(there) : "l"(flag) : "memory");
              if (!there) __nanosleep(64);
            }
            if (!there && !*dead) {
              atomicOr(&g_error_word, kErrLookback);
              *dead = 1;
            }
          }
          __syncwarp();
          const float4* from = reinterpret_cast<const float4*>(a.carry + ((int64_t)(work.worker - 1) * 16 + warp) * (KH * 32));
#pragma unroll
          for (int c = 0; c < KH; c += 4) {
            const float4 x = __ldcg(from + c / 4 * 32 + lane);
            S[c / 2] = pair(x.x, x.y), S[c / 2 + 1] = pair(x.z, x.w);
          }
        } else {
          const bool in = a.s_in && !STATES && vi < a.dv;
          const float* from = a.s_in + bh * a.s_in_head + step * a.s_in_seg + part * KH * a.sk + vi * a.sv;
#pragma unroll
          for (int c = 0; c < KH; c += 2) {
            const int kk = part * KH + c;
            S[c / 2] = pair(in && kk < a.dk ? from[0] : 0.f, in && kk + 1 < a.dk ? from[a.sk] : 0.f);
            from += 2 * a.sk;
          }
        }
        // every MMA that read the planes before is done (b_o of the last chunk)
        auto give_state = [&]() {
          store_planes();
          tc5_fence_before();
          arrive(b_s);
        };
        if (!STATES && p.first < p.last) give_state();
        for (int cc = p.first; cc < p.last; ++cc, ++n) {
          const int chunk = a.reverse ? p.last - 1 - (cc - p.first) : cc, t0 = chunk * kLaChunk;
          const float* fac = reinterpret_cast<const float*>(smem + CF::kFac) + (int)(n % CF::RF) * CF::kFacFloats;
          const bool anchor_here = a.dump && ((chunk + 1) % a.anchor_chunks == 0 || chunk == all_chunks - 1);
          if (!STATES && a.reverse && anchor_here) {
            // <R, S> behind this chunk: R is the state here, S the forward pass's
            float sum = 0.f;
            const int64_t an = bh * a.anchors + chunk / a.anchor_chunks;
            const float* from = a.dump + (an * 16 + warp) * (KH * 32);
#pragma unroll
            for (int c = 0; c < KH; c += 4) {
              const float4 x = reinterpret_cast<const float4*>(from)[c / 4 * 32 + lane];
              sum += pair_lo(S[c / 2]) * x.x + pair_hi(S[c / 2]) * x.y + pair_lo(S[c / 2 + 1]) * x.z + pair_hi(S[c / 2 + 1]) * x.w;
            }
#pragma unroll
            for (int o = 16; o >= 1; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
            if (lane == 0) a.anchor[an * 16 + warp] = sum;
          }
          la_wait(&full_f[n % CF::RF], (uint32_t)((n / CF::RF) & 1), dead);
          const float decay = fac[4 * kLaChunk];
          la_wait(STATES ? b_ds : b_o, (uint32_t)(n & 1), dead);
          tc5_fence_after();
          float o[2][8];
          uint32_t x[KH];
          if (!STATES) {
            uint32_t x1[2][8], x2[2][8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              tmem_ld_rows16(x1[e], lanes + ((uint32_t)(e * 16) << 16) + CF::cO1 + part * 16);
              tmem_ld_rows16(x2[e], lanes + ((uint32_t)(e * 16) << 16) + CF::cO2 + part * 16);
            }
            tmem_ld(x, lanes + CF::cDS + part * KH);
            float2 f[2];
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2)
              f[i2] = *reinterpret_cast<const float2*>(fac + 2 * kLaChunk + part * 16 + i2 * 8 + 2 * (lane % 4));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              tmem_wait_ld(x1[e]);
              tmem_wait_ld(x2[e]);
#pragma unroll
              for (int i2 = 0; i2 < 8; ++i2)
                o[e][i2] = fmaf(__uint_as_float(x2[e][i2]), i2 % 2 ? f[i2 / 4].y : f[i2 / 4].x, __uint_as_float(x1[e][i2]));
            }
          } else {
            tmem_ld(x, lanes + CF::cDS + part * KH);
          }
          const uint64_t decay2 = pair(decay, decay);
          tmem_wait_ld(x);
#pragma unroll
          for (int e = 0; e < KH / 2; ++e) S[e] = fma2(S[e], decay2, pair(x[2 * e], x[2 * e + 1]));
          tc5_fence_before();
          arrive(b_free);
          arrive(&empty_f[n % CF::RF]);
          if (!STATES && cc + 1 < p.last) give_state();
          if (!STATES)
            la_emit<T>(a, o, smem + CF::kStage + warp * 512, b, bh, h, t0 + part * 16, len, quad * 32, quad, lane);
          if (!STATES && !a.reverse && anchor_here) {
            const int64_t an = bh * a.anchors + chunk / a.anchor_chunks;
            float* to = a.dump + (an * 16 + warp) * (KH * 32);
#pragma unroll
            for (int c = 0; c < KH; c += 4)
              reinterpret_cast<float4*>(to)[c / 4 * 32 + lane] =
                  make_float4(pair_lo(S[c / 2]), pair_hi(S[c / 2]), pair_lo(S[c / 2 + 1]), pair_hi(S[c / 2 + 1]));
          }
        }
        if (p.to_carry) {
          float4* to = reinterpret_cast<float4*>(a.carry + ((int64_t)work.worker * 16 + warp) * (KH * 32));
#pragma unroll
          for (int c = 0; c < KH; c += 4) 
            __stcg(to + c / 4 * 32 + lane,
                   make_float4(pair_lo(S[c / 2]), pair_hi(S[c / 2]), pair_lo(S[c / 2 + 1]), pair_hi(S[c / 2 + 1])));
          __threadfence();
          __syncwarp();
          if (lane == 0)
            asm volatile("st.release.gpu.global.u32 [%0], %1;\n" ::"l"(a.flags + 1 + work.worker * 16 + warp), "r"(1u) : "memory");
        } else if (a.s_out && (STATES || step == a.nseg - 1) && vi < a.dv) {
          float* to = a.s_out + bh * a.s_out_head + step * a.s_out_seg + part * KH * a.sk + vi * a.sv;
#pragma unroll
          for (int c = 0; c < KH; ++c) {
            if (part * KH + c < a.dk) *to = c % 2 ? pair_hi(S[c / 2]) : pair_lo(S[c / 2]);
            to += a.sk;
          }
        }
      }
    }
  }
  // every MMA was waited for (the last chunk's) unless a wait gave up: then this
  // commit, waited for with a limit too, stands between those in flight and the end
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  if (warp == kLaMmaWarp) {
    if (*dead) {
      if (lane == 0) {
        mma_commit(single);  // not used otherwise
        for (int i = 0; i < 4096 && !mbar_try_wait(single, 0); ++i) {}
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
// stretch between two.  One warp a stretch, from its end; sums in fp64.  Keys of at
// most 64 fill two lane quadrants of the partial products, wider ones four.
template <typename T>
__global__ void linattn_decay_grad_kernel(const float* dots_q, const float* dots_k, const float* anchor, T* out,
                                          const int* lengths, int64_t bhs, int heads, int seqlen, int anchors,
                                          int anchor_tokens, bool two_quads) {
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
  for (int i = 0; i < 16; ++i)
    if (!two_quads || i % 4 < 2) carry += anchor[(bh * anchors + an) * 16 + i];
  for (int hi = end; hi > begin; hi -= 32) {
    const int t = hi - 1 - lane;  // lane 0 the latest
    double x = 0.0;
    if (t >= begin) {
      const float4 q = reinterpret_cast<const float4*>(dots_q)[bh * seqlen + t];
      const float4 k = reinterpret_cast<const float4*>(dots_k)[bh * seqlen + t];
      x = ((double)q.x + q.y) - ((double)k.x + k.y);
      if (!two_quads) x += ((double)q.z + q.w) - ((double)k.z + k.w);
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

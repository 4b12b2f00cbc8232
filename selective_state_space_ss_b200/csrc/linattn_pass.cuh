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
// Precision.  The tensor core multiplies bf16 and adds in fp32.  A value that is not bf16
// already is split into bf16 planes.  bf16 inputs stay as they are; scores times decays
// (P) and the state, whose products end in a bf16 output, take two planes, 16 bits; the
// weighted keys, whose products add up in the fp32 state, take four: a product of two
// bf16 is a bf16 and a bf16 that is left over, exactly, so they are formed in bf16
// arithmetic (two planes left the state 2.4e-6 off, four 1e-7).  With P and the state in
// two planes the last place of a bf16 output differs from that of a 32-bit evaluation
// in about one of 400, 9e-5 of the norm next to the rounding's own 1.7e-3; three gave 3e-5
// and took 6% longer with 64 x 64 heads, 34% with 128 x 128 (B4 L8192 H40, 438 -> 587 us:
// tensor memory then has one place for scores).  fp32 inputs and
// everything behind them take three planes, 24 bits, and the six products of planes whose
// weight reaches that far.  Products of smaller planes are added first, while the sum is
// small (in the other order fp32 outputs were 2e-6 off, in this one 2e-7).  The state
// itself stays fp32 in registers.  Running sums of the decays are whole numbers of 2^-44.
//
// Layout.  Scores are Q K^T with tokens in the lanes.  O and S are kept transposed
// (value index in the lanes), so that S^T is the MMA's A operand straight from
// tensor memory: it is written there by the threads that hold it and never goes
// through shared memory.  M is 128 there; where values are 64 wide the other lanes
// hold sums of whatever follows in shared memory and nobody reads them.
//
// Roles.  One thread loads K, V and Q tiles into rings by TMA (a warp or two where TMA
// does not apply), one warp works out the decays, one thread of a warp issues the state's
// increments and one of another the scores and outputs; the front warps (eight) turn
// keys into weighted keys and scores into P a chunk ahead of the back warps (sixteen),
// which hold the state: they add the increment, give the state back as planes, take O
// from tensor memory and write it out while the next chunk's products run.
//
// What bounds it, and what the steps gave (bf16, B4 L8192, 40 heads of 128 x 128: 1.36 GB,
// 207 us at the copy rate of 6.55 TB/s).  Four loader warps and eight that did all the
// rest in turn: 2.32 ms.  The roles apart, TMA: 1.03.  Fewer instructions, code that fits
// the instruction cache (spin loops not unrolled, product loops short): 0.50.  Products
// issued from warp-uniform descriptors, sixteen and eight warps, hand-overs of their own
// for P and the weighted keys: 0.41 to 0.46 (2.9 to 3.3 TB/s, 44 to 51% of the copy
// rate), 2.3 to 2.5 us a chunk and SM of 64 tokens.  ncu: 11 thousand warp instructions a
// chunk, issue slots 60% busy, tensor pipe 43%, DRAM 40%: it is bound by the work around
// the products (splitting, weighting, moving) and its hand-overs, not by a single unit.
// With 64 x 64 heads a chunk takes 1.6 us, half of its data, for the same hand-overs; with
// 128 x 64 2.1 us, tensor pipe 51%, issue slots 50%.  fp32: 7.5 us (64 x 64) to 15
// (128 x 128), issue slots 22% and tensor pipe 22% busy: the warps wait for tiles that two
// loader warps split.
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
// Polls before a wait gives up, a second or so.  A poll of a barrier suspends the thread
// for as long as the hardware likes, 3 to 4 us whatever longer time it is given; a poll of
// the previous worker's flag takes about as many tenths.  (512 polls of the first gave up
// after 2 ms, which a worker may well wait for a state where the rows between are short.)
// As a launch's argument the first limit cost 2 to 4%.
constexpr uint32_t kLaSpinLimit = 1u << 18;
constexpr uint32_t kLaCarrySpinLimit = 1u << 21;

// A [batch, seqlen, heads, d] tensor, last axis contiguous, strides in elements;
// `share` consecutive heads of the pass read one of its heads.
struct LaTensor {
  const void* ptr;
  int64_t sb, st, sh;
  int share;
#ifdef SS_BOUNDS_CHECK
  int64_t lo, n;  // its elements: n of them from offset lo on
#endif
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
  LaTensor x;           // rows to take the inner product of with each output row's part from the state
  float* dots;          // [batch * heads, seqlen, 4] partial products of x, one a lane quadrant
  float* dump;          // the states before each chunk: forward writes them, reversed reads them
  float* flow;          // reversed: [batch * heads, chunks, 16] partial products <R, S>, one a back warp
  int chunks;           // of a whole row
  int heads, seqlen, dk, dv;
  int bh;               // batch * heads
  int nseg, seg_chunks; // segments of a head, or
  int workers;          // > 0: CTAs that share all chunks evenly
  float* carry;         // [workers] states handed to the next worker
  unsigned* flags;      // [0] hands out worker numbers, then [workers][16] one a back warp; zero at launch
  int reverse;
  int vec;              // 16-byte loads apply to q, k and v
  int out_vec, x_vec;   // 16-byte stores to out, loads of x
  int tma;              // so do the tensor maps
  float scale_p, scale_o, scale_w;
  uint32_t carry_spin_limit;  // polls before a wait for another worker's state gives up
  int skip_publish;     // test hooks: a worker that hands nothing on,
  int skip_load;        // a chunk whose values no CTA loads (-1: none)
};

struct LaMaps {
  CUtensorMap q, k, v;
};

// What a launch does: outputs and states; the states alone (the sequence's segments, each
// from zero, all at once); outputs and states with the products that a decay's gradient
// is made of (of x with what each output row has from the state, of the two passes' states
// at every chunk).
enum LaMode { kLaOutputs, kLaStates, kLaProducts };

template <typename T, int KD, int VD, LaMode MODE = kLaOutputs>
struct LaCfg {
  static constexpr bool kBf16 = sizeof(T) == 2;
  static constexpr int NPI = kBf16 ? 1 : 3;  // planes of the inputs
  static constexpr int NPX = kBf16 ? 2 : 3;  // planes of the scores and of the state as operands
  static constexpr int NPW = kBf16 ? 4 : 3;  // planes of the weighted keys
  static constexpr int KB = KD / 64, VB = VD / 64;
  // Tiles in each ring.  A key tile lives until its chunk's increment is formed (the
  // weighted keys' first planes replace it in place), a query tile until S Q is.
  static constexpr int RK = kBf16 ? 3 : 2, RQ = kBf16 ? 3 : 1, RV = kBf16 ? (KB == 2 && VB == 2 ? 2 : 3) : 1;
  static constexpr int RP = kBf16 ? 2 : 1;   // P
  // The weighted keys' further planes: two places, or one that is filled and used in halves.
  // (fp32 has all three planes in the key tile.)
  static constexpr int RW = kBf16 && KB == 2 ? 1 : 2;
  static constexpr int RF = 4;               // decays
  static constexpr int kRing = 4;
  static_assert(RK <= kRing && RV <= kRing && RQ <= kRing && RF <= kRing, "barriers of a ring");
  static constexpr int kTileK = KB * NPI * kLaBlock, kTileV = VB * NPI * kLaBlock, kTileW = KB * (NPW - NPI) * kLaBlock;
  static constexpr int kQ = 0, kK = RQ * kTileK, kV = kK + RK * kTileK, kP = kV + RV * kTileV;
  static constexpr int kW = kP + RP * NPX * kLaBlock;
  static constexpr int kFacFloats = (kBf16 ? 6 : 4) * kLaChunk + 4;
  static constexpr int kFac = kW + RW * kTileW;
  static constexpr int kStage = kFac + (RF * kFacFloats * 4 + 127) / 128 * 128;  // 512 bytes a back warp
  static constexpr int kBars = kStage + (kBf16 ? 16 * 512 : 0);
  static constexpr int kSmem = kBars + 12 * kRing * 8 + 16;
  // tensor memory columns
  // (two increments where there is room: the next one need not wait until the back has
  // read the last)
  static constexpr int ND = KD == 64 || MODE == kLaStates ? 2 : 1;
  static constexpr int cDS = 0, cSP = ND * KD, cO1 = cSP + NPX * KD / 2, cO2 = cO1 + 64, cQK = cO2 + 64;
  static constexpr int kAhead = kBf16 ? 2 : 1;  // chunks that scores run ahead, one place for each
  static constexpr int kUsed = MODE == kLaStates ? ND * KD : cQK + 64 * kAhead;
  static constexpr int kCols = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
  static constexpr int kQuads = VD / 32;        // lane quadrants that hold values
  static constexpr int kHolders = 4 * kQuads;   // back warps at work
  // Two warps issue MMAs: one the state's increments, the other scores and outputs, so
  // that neither chain of hand-overs waits in the other's.  (fp32 has one query tile and
  // one place for scores, so all in one order, and more loading to do: there the second
  // warp loads.)
  static constexpr bool kTwoIssuers = kBf16;
  static constexpr int kLoaders = kTwoIssuers ? 32 : 64;  // loader threads
  static constexpr int kThreads = 896;
  // Registers a thread of the three kinds of warpgroup: 4 x 88 + 2 x 56 + 40 (fp32, with
  // all its loads through registers: 4 x 80 + 2 x 56 + 72, 8% faster with 128 x 128
  // heads) = 7 x 72 at launch.
  static constexpr int kBackRegs = kBf16 ? 88 : 80, kFrontRegs = 56, kAuxRegs = kBf16 ? 40 : 72;
  static_assert(4 * kBackRegs + 2 * kFrontRegs + kAuxRegs == 7 * 72, "registers of a block");
};
constexpr int kLaBackWarps = 16, kLaFrontWarps = 8;
constexpr int kLaMmaWarp = 24, kLaLoadWarp = 25, kLaMmaOrLoadWarp = 26, kLaDecayWarp = 27;

// Waits of one CTA: when one gives up, the others stop waiting too, and the kernel
// runs to its end on whatever is there, inside its buffers.  A poll suspends the
// thread, so that those that wait leave the issue slots to the others.
__device__ __forceinline__ bool la_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(10000000)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool la_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
#pragma unroll 1
  for (uint32_t i = 0; i < kLaSpinLimit; ++i) {
    if (la_poll(bar, parity)) return true;
    if (*dead) return false;
  }
  atomicOr(&g_error_word, kErrTmaWait);
  *dead = 1;
  return false;
}
// Whatever else gave up: for copies and products of one's own that are in flight.
__device__ __forceinline__ void la_wait_own(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kLaSpinLimit; ++i)
    if (la_poll(bar, parity)) return;
  atomicOr(&g_error_word, kErrTmaWait);
}
__device__ __forceinline__ void la_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void la_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void la_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}

// A place in a ring of R and how often it came round: full barriers complete phase
// `turn`, empty ones are waited for from the second turn on.
template <int R>
struct LaRing {
  int i = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next() {
    if (++i == R) i = 0, ++turn;
  }
  __device__ __forceinline__ uint32_t full() const { return turn & 1; }
  __device__ __forceinline__ bool used() const { return turn > 0; }
  __device__ __forceinline__ uint32_t empty() const { return (turn - 1) & 1; }
};

__device__ __forceinline__ int la_length(const LaPassArgs& a, int64_t b) {
  if (!a.lengths) return a.seqlen;
  const int n = a.lengths[b];
  return n < 0 ? 0 : n < a.seqlen ? n : a.seqlen;
}

__device__ __forceinline__ const char* la_row(const LaTensor& x, int64_t b, int64_t t, int h, int es) {
  return static_cast<const char*>(x.ptr) + (b * x.sb + t * x.st + (int64_t)(h / x.share) * x.sh) * es;
}

// Checked builds: whether `count` elements at `from` are the tensor's.
__device__ __forceinline__ bool la_inside(const LaTensor& x, const char* from, int count, int es) {
#ifdef SS_BOUNDS_CHECK
  return in_range((from - static_cast<const char*>(x.ptr)) / es - x.lo, count, x.n);
#else
  return true;
#endif
}

// One tile of 64 tokens into shared memory: rows from `len` on and columns from `d`
// on are zero.  bf16 with 16-byte rows: asynchronous copies (the caller waits);
// everything else through registers, up to four units at a time, the rows `ahead` tokens on
// (the next chunk's) asked for in L2 meanwhile.
template <typename T>
__device__ __forceinline__ void la_fetch_unit(float (&f)[8], const char* from, bool in, int col, int d, bool vec) {
  const T* p = reinterpret_cast<const T*>(from);
  if (sizeof(T) == 4 && vec) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 f0 = in ? reinterpret_cast<const float4*>(p)[0] : z;
    const float4 f1 = in && col + 4 < d ? reinterpret_cast<const float4*>(p)[1] : z;
    f[0] = f0.x, f[1] = f0.y, f[2] = f0.z, f[3] = f0.w, f[4] = f1.x, f[5] = f1.y, f[6] = f1.z, f[7] = f1.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = in && col + i < d ? to_f32(p[i]) : 0.f;
  }
}
template <typename T, int DP>
__device__ __forceinline__ void la_load_tile(char* dst, const LaTensor& x, int64_t b, int h, int t0, int len, int d,
                                             bool vec, int ahead, int tid, int nthreads) {
  constexpr int B = DP / 64, PLANES = sizeof(T) == 2 ? 1 : 3, E = sizeof(T) == 2 ? 1 : 4;
  constexpr int UNITS = kLaChunk * B * 8;
  const char* base = la_row(x, b, 0, h, sizeof(T));
  const int64_t step = x.st * (int64_t)sizeof(T);
  if (sizeof(T) == 2 && vec) {
#pragma unroll 1
    for (int u = tid; u < UNITS; u += nthreads) {
      const int row = u / (B * 8), unit = u % (B * 8), col = unit * 8;
      const bool in = t0 + row < len && col < d && la_inside(x, base + (t0 + row) * step + col * 2, 8, 2);
      const char* from = base + (in ? (t0 + row) * step + col * 2 : 0);
      const uint32_t bytes = in ? 16 : 0;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                       smem_u32(dst + (unit / 8) * kLaBlock + tile_unit(row, unit % 8))),
                   "l"(from), "r"(bytes)
                   : "memory");
    }
    return;
  }
#pragma unroll 1
  for (int u = tid; u < UNITS; u += E * nthreads) {
    float f[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int v = u + e * nthreads, row = v / (B * 8), col = v % (B * 8) * 8;
      const bool in = t0 + row < len && col < d &&
                      la_inside(x, base + (t0 + row) * step + col * (int)sizeof(T), d - col < 8 ? d - col : 8, sizeof(T));
      const char* from = base + (in ? (t0 + row) * step + col * (int)sizeof(T) : 0);
      la_fetch_unit<T>(f[e], from, in, col, d, vec);
      const int next = t0 + row + ahead;
      if (in && next >= 0 && next < len)
        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(from + ahead * step));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int v = u + e * nthreads, row = v / (B * 8), unit = v % (B * 8);
      char* to = dst + (unit / 8) * kLaBlock + tile_unit(row, unit % 8);
      uint32_t w[PLANES][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t s[PLANES];
        split2<PLANES>(pair(f[e][2 * i], f[e][2 * i + 1]), s);
#pragma unroll
        for (int p = 0; p < PLANES; ++p) w[p][i] = s[p];
      }
#pragma unroll
      for (int p = 0; p < PLANES; ++p)
        *reinterpret_cast<uint4*>(to + p * B * kLaBlock) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
  }
}

// A lane's two log decays of a chunk as they are stored, zero behind the row's end.
// Those of `ahead` tokens on are asked for in L2: a chunk may take less than a load.
template <typename T>
__device__ __forceinline__ void la_fetch_decays(T (&x)[2], const LaTensor& g, int b, int h, int t0, int len, int ahead,
                                                int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = t0 + 2 * lane + i;
    x[i] = zero_elem<T>();
    const char* from = la_row(g, b, t, h, sizeof(T));
    if (t < len && la_inside(g, from, 1, sizeof(T))) x[i] = *reinterpret_cast<const T*>(from);
    if (ahead != 0 && t + ahead >= 0 && t + ahead < len)
      asm volatile("prefetch.global.L2 [%0];\n" ::"l"(from + ahead * g.st * (int64_t)sizeof(T)));
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

// Of a sum of decays (below), what la_exp2 takes.
__device__ __forceinline__ int64_t la_fixed32(int64_t x) { return x >> 12; }

// Running sums of a chunk's decays, base 2, two tokens a lane of a warp, and the whole.
// They are whole numbers of 2^-44 (64 tokens of at most 2020 fit 61 bits), so differences of
// large sums lose nothing, nor do the sums of tens of thousands of slow decays.  A log decay
// beyond +-1400 leaves nothing, or too much, in fp32 and is taken as that: minus infinity
// (a reset) is a number like any other here.
constexpr int kLaDecayBits = 44;
__device__ __forceinline__ void la_decay_sums(int64_t (&at)[2], int64_t& total, float x0, float x1, int lane) {
  const float x[2] = {x0, x1};
  int64_t g[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    g[i] = __double2ll_rn((double)fminf(fmaxf(x[i], -1400.f), 1400.f) * (1.4426950408889634 * (double)(INT64_C(1) << kLaDecayBits)));
  int64_t sum = g[0] + g[1];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t up = __shfl_up_sync(kFullMask, sum, o);
    if (lane >= o) sum += up;
  }
  total = __shfl_sync(kFullMask, sum, 31);
  at[0] = sum - g[1], at[1] = sum;
}

// The factor that the state passes a chunk with, from the sum of its decays.  Near 1 what
// rounding leaves out of it, `left` (a natural logarithm), goes into the next chunk's: with
// slow decays the state passes hundreds of equal factors, whose equal roundings would add
// up (to 8e-6 of the state after 256 chunks of log decays of -1e-6).  e^t - 1 by its series,
// |t| < 0.35: the first term left out is 2e-8 of it.
__device__ __forceinline__ float la_exp2_chunk(int64_t x, float& left) {
  if (x <= -(INT64_C(1) << (kLaDecayBits - 1)) || x >= (INT64_C(1) << (kLaDecayBits - 1))) {
    left = 0.f;
    return la_exp2(la_fixed32(x));
  }
  const float t = fmaf((float)x, (float)(0.6931471805599453 / (INT64_C(1) << kLaDecayBits)), left);
  float e = fmaf(t, 1.f / 5040, 1.f / 720);
  e = fmaf(t, e, 1.f / 120);
  e = fmaf(t, e, 1.f / 24);
  e = fmaf(t, e, 1.f / 6);
  e = fmaf(t, e, 0.5f);
  e = fmaf(t * t, e, t);
  const float y = 1.f + e;
  left = (e - (y - 1.f)) * rcp_approx(y);
  return y;
}

// A chunk's decays: running sums, base 2, as integer and fraction (64 floats each), the
// factors of the rows, those of the keys (for bf16 keys as three bf16 planes, each twice
// in a word), and the chunk's whole decay, whose sum is returned.  ROWS false (the states
// alone): the last two.  One warp.
template <bool BF16, bool ROWS>
__device__ __forceinline__ int64_t la_decays(float* fac, float& left, float x0, float x1, bool reverse, float scale_o,
                                             float scale_w, int lane) {
  int64_t at[2], total;
  la_decay_sums(at, total, x0, x1, lane);
  // a NaN among them is not to vanish
  const float bad = __any_sync(kFullMask, x0 != x0 || x1 != x1) ? __int_as_float(0x7fffffff) : 1.f;
  float2* out = reinterpret_cast<float2*>(fac) + lane;
  float keys[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) keys[i] = la_exp2(la_fixed32(reverse ? at[i] : total - at[i])) * scale_w * bad;
  if constexpr (ROWS) {
    float hi[2], lo[2], rows[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t x = la_fixed32(at[i]);
      hi[i] = (float)(int)(x >> 32);
      lo[i] = (float)(uint32_t)x * 0x1p-32f * bad;
      rows[i] = la_exp2(reverse ? la_fixed32(total - at[i]) : x) * scale_o * bad;
    }
    out[0] = make_float2(hi[0], hi[1]);
    out[32] = make_float2(lo[0], lo[1]);
    out[64] = make_float2(rows[0], rows[1]);
  }
  if constexpr (BF16) {
    uint32_t p0[3], p1[3];
    split2<3>(pair(keys[0], keys[0]), p0);
    split2<3>(pair(keys[1], keys[1]), p1);
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<uint2*>(fac)[96 + 32 * i + lane] = make_uint2(p0[i], p1[i]);
  } else {
    out[96] = make_float2(keys[0], keys[1]);
  }
  const float whole = la_exp2_chunk(total, left) * bad;
  if (lane == 0) fac[(BF16 ? 6 : 4) * kLaChunk] = whole;
  return total;
}

template <int N>
struct LaWidth {
  static constexpr int value = N;
};

// 32 values x 16 tokens of a back warp, o[h][4 i + z]: value v0 + 16 h + 8 (z / 2) +
// lane / 4, token t0 + 8 i + 2 (lane % 4) + z % 2.  To the output element by element: fp32
// (32 bytes a token together) and, but for F32_ONLY, rows that are not whole 16-byte
// units.
template <typename T, bool F32_ONLY>
__device__ __forceinline__ void la_emit(const LaPassArgs& a, const float (&o)[2][8], int64_t b, int h, int t0, int len,
                                        int v0, int lane) {
  const int64_t rs = (int64_t)a.heads * a.dv;
  const int v = v0 + lane / 4, t = t0 + 2 * (lane % 4);
  const int64_t mine = ((b * a.seqlen + t) * a.heads + h) * a.dv + v, all = (int64_t)a.bh * a.seqlen * a.dv;
  if ((F32_ONLY || sizeof(T) == 4 || a.out_f32) && t0 + 16 <= len && v0 + 32 <= a.dv) {  // all there
    float* to = static_cast<float*>(a.out) + mine;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float* row = to + (8 * i + z) * rs;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (in_range(row + 8 * u - static_cast<float*>(a.out), all)) row[8 * u] = o[u / 2][4 * i + 2 * (u % 2) + z];
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int64_t row = mine + (8 * i + z) * rs;
      if (t + 8 * i + z < len) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (v + 8 * u < a.dv && in_range(row + 8 * u, all)) {
            const float y = o[u / 2][4 * i + 2 * (u % 2) + z];
            if (F32_ONLY || sizeof(T) == 4 || a.out_f32) static_cast<float*>(a.out)[row + 8 * u] = y;
            else static_cast<__nv_bfloat16*>(a.out)[row + 8 * u] = __float2bfloat16_rn(y);
          }
      }
    }
}

// The same values' products with the rows of x, element by element.
template <typename T>
__device__ __forceinline__ void la_dots(float (&sum)[4], const LaPassArgs& a, const float (&o)[2][8], int64_t b, int h,
                                        int t0, int len, int v0, int lane) {
  const int v = v0 + lane / 4, t = t0 + 2 * (lane % 4);
  const char* from = la_row(a.x, b, t, h, sizeof(T)) + (int64_t)v * sizeof(T);
  const int64_t xs = a.x.st * (int64_t)sizeof(T);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float y = 0.f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t + 8 * i + z < len && v + 8 * u < a.dv &&
            la_inside(a.x, from + (8 * i + z) * xs + 8 * u * (int)sizeof(T), 1, sizeof(T)))
          y = fmaf(o[u / 2][4 * i + 2 * (u % 2) + z], to_f32(reinterpret_cast<const T*>(from + (8 * i + z) * xs)[8 * u]), y);
      sum[2 * i + z] = y;
    }
}

// The products of planes pa < PA of one operand and pb < PB of the other whose
// weight counts, the smaller ones first: they add up while the sum is small.  STEPS MMAs
// each, told the planes, the step and whether they add.
template <int PA, int PB, int STEPS, typename F>
__device__ __forceinline__ void la_products(F&& mma) {
  constexpr int P = PA > PB ? PA : PB;
#pragma unroll
  for (int pa = PA - 1; pa >= 0; --pa)
#pragma unroll
    for (int pb = (P - pa < PB ? P - pa : PB) - 1; pb >= 0; --pb)
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        mma(pa, pb, i, !(pa == PA - 1 && pb == (P - pa < PB ? P - pa : PB) - 1 && i == 0));
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

// FAST: bf16 with 16-byte rows everywhere and no lengths, without the code for the rest
// (720 instructions of plain loads alone; B4 L8192 H40 128 x 128 took 4% longer with it,
// for the instruction cache).
template <typename T, int KD, int VD, LaMode MODE, bool FAST>
__global__ void __launch_bounds__(LaCfg<T, KD, VD, MODE>::kThreads, 1)
linattn_pass_kernel(const __grid_constant__ LaPassArgs a, const __grid_constant__ LaMaps maps) {
  using CF = LaCfg<T, KD, VD, MODE>;
  constexpr int NPI = CF::NPI, NPX = CF::NPX, NPW = CF::NPW;
  constexpr bool STATES = MODE == kLaStates, DOTS = MODE == kLaProducts;
  extern __shared__ __align__(1024) char smem[];
  // barriers: CF::kRing places for each ring, whatever its length
  const uint32_t base = smem_u32(smem), bars = base + CF::kBars;
  const auto ring_bar = [&](int which, int i) { return bars + (uint32_t)(which * CF::kRing + i) * 8; };
  const auto full_k = [&](int i) { return ring_bar(0, i); };
  const auto empty_k = [&](int i) { return ring_bar(1, i); };
  const auto full_v = [&](int i) { return ring_bar(2, i); };
  const auto empty_v = [&](int i) { return ring_bar(3, i); };
  const auto full_q = [&](int i) { return ring_bar(4, i); };
  const auto empty_q = [&](int i) { return ring_bar(5, i); };
  const auto full_f = [&](int i) { return ring_bar(6, i); };
  const auto empty_f = [&](int i) { return ring_bar(7, i); };
  const auto b_qk = [&](int i) { return ring_bar(8, i); };  // scores are there, one for each place
  const auto b_p = [&](int i) { return ring_bar(8, 2 + i); };  // P is there
  const auto b_w = [&](int i) { return ring_bar(11, i); };  // half of the weighted keys is there
  const uint32_t b_half = ring_bar(10, 0); // the first half of them was used
  const auto b_ds = [&](int i) { return ring_bar(11, 2 + i); };  // the state's increment is there
  const auto b_p_free = [&](int i) { return ring_bar(10, 2 + i); };  // P was used
  const uint32_t b_o = ring_bar(9, 0);     // P V and S Q are there
  const auto b_free = [&](int i) { return ring_bar(i ? 10 : 9, 1); };  // the back warps have read the increment
  const uint32_t b_s = ring_bar(9, 2);     // the state's planes are there, and the outputs before were read
  const uint32_t b_end = ring_bar(9, 3);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + CF::kBars + 12 * CF::kRing * 8);
  int* worker_at = reinterpret_cast<int*>(tmem_at + 1);
  volatile int* dead = worker_at + 1;

  // one value for a warp, known as such: what follows from it stays off the vector registers
  const auto same = [](uint32_t x) { return __shfl_sync(kFullMask, x, 0); };
  const int tid = threadIdx.x, warp = (int)same(tid / 32), lane = tid % 32;
  if (tid == 0) {
    for (int i = 0; i < CF::kRing; ++i) {
      for (int w = 0; w < 7; ++w)
        if (STATES || w != 3) la_init(ring_bar(w, i), 1);
      la_init(empty_f(i), kLaFrontWarps + CF::kHolders);
      if (!STATES) la_init(empty_v(i), 2);
    }
    la_init(b_qk(0), 1);
    la_init(b_qk(1), 1);
    la_init(b_p(0), kLaFrontWarps);
    la_init(b_p(1), kLaFrontWarps);
    la_init(b_w(0), kLaFrontWarps);
    la_init(b_w(1), kLaFrontWarps);
    la_init(b_half, 1);
    la_init(b_p_free(0), 1);
    la_init(b_p_free(1), 1);
    for (int i = 0; i < 2; ++i) la_init(b_ds(i), 1), la_init(b_free(i), CF::kHolders);
    la_init(b_o, 1);
    la_init(b_s, CF::kHolders);
    la_init(b_end, CF::kTwoIssuers ? 2 : 1);
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
  const uint32_t tmem = same(*tmem_at);
  const LaWork work = la_work(a, (int)same(*worker_at));
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) la_arrive(bar);
  };

  if (warp >= kLaMmaWarp) {
    regs_give<CF::kAuxRegs>();
    if (warp == kLaMmaWarp || (CF::kTwoIssuers && warp == kLaMmaOrLoadWarp)) {
      // ---- MMA issue, by one thread of a warp
      constexpr int kUnits = kLaBlock >> 4;  // a block in descriptor units
      const bool leader = elect_one();
      const bool states = warp == kLaMmaWarp, outputs = !STATES && (!CF::kTwoIssuers || !states);
      LaRing<CF::RK> rk, sk;  // of the chunk at hand, and of the one whose scores come next
      LaRing<CF::RQ> rq, sq;
      LaRing<CF::RV> rv;
      int total = 0, scored = 0;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        total += p.last - p.first;
      }
      auto scores = [&]() {
        la_wait(full_k(sk.i), sk.full(), dead);
        la_wait(full_q(sq.i), sq.full(), dead);
        tc5_fence_after();
        const int place = scored % CF::kAhead;
        if (leader) {
          const uint32_t q = tile_desc(base + CF::kQ + sq.i * CF::kTileK, 0);
          const uint32_t k = tile_desc(base + CF::kK + sk.i * CF::kTileK, 0);
          la_products<NPI, NPI, KD / 16>([&](int pa, int pb, int i, bool add) {
            const int off = (i / 4) * kUnits + (i % 4) * 2;
            mma_ss(tmem + CF::cQK + place * 64, q + pa * CF::KB * kUnits + off, k + pb * CF::KB * kUnits + off,
                   mma_idesc(64, 64, false, false), add);
          });
          mma_commit(b_qk(place));
        }
        __syncwarp();
        sk.next(), sq.next(), ++scored;
      };
      if (outputs)
        while (scored < CF::kAhead && scored < total) scores();
      for (int n = 0; n < total; ++n) {
        const uint32_t v = tile_desc(base + CF::kV + rv.i * CF::kTileV, kLaBlock);
        la_wait(full_v(rv.i), rv.full(), dead);
        if (states) {
          // planes of the weighted keys: in the key tile's place, then in one of their own
          const uint32_t w0 = tile_desc(base + CF::kK + rk.i * CF::kTileK, kLaBlock);
          const uint32_t w1 = tile_desc(base + CF::kW + (n % CF::RW) * CF::kTileW, kLaBlock);
          const int inc = n % CF::ND;
          if (n >= CF::ND) la_wait(b_free(inc), (n / CF::ND - 1) & 1, dead);
          // dS^T = V^T (w . K), with one place for the keys 32 tokens at a time: the front makes
          // the next chunk's first half while the second is at work
          const auto tokens = [&](auto steps, int first) {
            la_products<NPI, NPW, decltype(steps)::value>([&](int pa, int pb, int i, bool add) {
              const int off = (first + i) * (16 * kTileRow >> 4);
              const uint32_t w = pb < NPI ? w0 + pb * CF::KB * kUnits : w1 + (pb - NPI) * CF::KB * kUnits;
              mma_ss(tmem + CF::cDS + inc * KD, v + pa * CF::VB * kUnits + off, w + off, mma_idesc(128, KD, true, true),
                     add || first > 0);
            });
          };
          la_wait(b_w(CF::RW == 2 ? n % 2 : 0), (CF::RW == 2 ? n / 2 : n) & 1, dead);
          tc5_fence_after();
          if (CF::RW == 1) {
            if (leader) {
              tokens(LaWidth<kLaChunk / 32>{}, 0);
              mma_commit(b_half);
            }
            __syncwarp();
            la_wait(b_w(1), n & 1, dead);
            tc5_fence_after();
          }
          if (leader) {
            if (CF::RW == 1) tokens(LaWidth<kLaChunk / 32>{}, 2);
            else tokens(LaWidth<kLaChunk / 16>{}, 0);
            mma_commit(b_ds(inc));
            mma_commit(empty_v(rv.i));
            mma_commit(empty_k(rk.i));
          }
          __syncwarp();
        }
        if (outputs) {
          const int place = n % CF::RP;
          la_wait(b_p(place), (n / CF::RP) & 1, dead);
          la_wait(b_s, n & 1, dead);  // and the last chunk's outputs were read
          tc5_fence_after();
          if (leader) {
            // O1^T = V^T P^T
            const uint32_t pd = tile_desc(base + CF::kP + place * NPX * kLaBlock, 0);
            la_products<NPI, NPX, kLaChunk / 16>([&](int pa, int pb, int i, bool add) {
              mma_ss(tmem + CF::cO1, v + pa * CF::VB * kUnits + i * (16 * kTileRow >> 4), pd + pb * kUnits + i * 2,
                     mma_idesc(128, 64, true, false), add);
            });
            // O2^T = S^T Q^T
            const uint32_t q = tile_desc(base + CF::kQ + rq.i * CF::kTileK, 0);
            la_products<NPX, NPI, KD / 16>([&](int pa, int pb, int i, bool add) {
              mma_ts(tmem + CF::cO2, tmem + CF::cSP + pa * (KD / 2) + i * 8,
                     q + (pb * CF::KB + i / 4) * kUnits + (i % 4) * 2, mma_idesc(128, 64, false, false), add);
            });
            mma_commit(b_o);
            mma_commit(b_p_free(place));
            mma_commit(empty_v(rv.i));
            mma_commit(empty_q(rq.i));
          }
          __syncwarp();
          // last, so that no tile is waited for while the chunk's own products could run
          if (scored < total) scores();
        }
        rk.next(), rq.next(), rv.next();
      }
      // whoever issued products says when they are done: one waits for it below if a wait gave up
      if (leader) mma_commit(b_end);
      __syncwarp();
    } else if (warp == kLaDecayWarp) {
      // ---- decays
      LaRing<CF::RF> rf;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        double sum = 0.0;
        float left = 0.f;
        auto place = [&](int c) { return (a.reverse ? p.last - 1 - (c - p.first) : c) * kLaChunk; };
        T next[2];
        const int ahead = (a.reverse ? -4 : 4) * kLaChunk;
        if (p.first < p.last) la_fetch_decays<T>(next, a.g, p.b, p.h, place(p.first), p.len, ahead, lane);
        for (int c = p.first; c < p.last; ++c) {
          const float x0 = to_f32(next[0]), x1 = to_f32(next[1]);
          if (c + 1 < p.last) la_fetch_decays<T>(next, a.g, p.b, p.h, place(c + 1), p.len, ahead, lane);
          if (rf.used()) la_wait(empty_f(rf.i), rf.empty(), dead);
          const int64_t whole = la_decays<CF::kBf16, !STATES>(reinterpret_cast<float*>(smem + CF::kFac) + rf.i * CF::kFacFloats,
                                                              left, x0, x1, a.reverse, a.scale_o, a.scale_w, lane);
          if (STATES) sum += (double)whole * (1.0 / (INT64_C(1) << kLaDecayBits));
          arrive(full_f(rf.i));
          rf.next();
        }
        const int64_t at = (int64_t)p.bh * (a.nseg + 1) + work.worker % a.nseg;
        if (STATES && lane == 0 && in_range(at, (int64_t)a.bh * (a.nseg + 1))) a.seg_decay[at] = sum;
      }
    } else {
      // ---- loaders: one thread by TMA, or all of them
      const int ltid = tid - 32 * kLaLoadWarp;
      LaRing<CF::RK> rk;
      LaRing<CF::RQ> rq;
      LaRing<CF::RV> rv;
      bool gone = false;  // (TMA) a place was not free in time: no further copies
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        const int hk = p.h / a.k.share, hq = p.h / a.q.share, hv = p.h / a.v.share;
        for (int c = p.first; c < p.last; ++c) {
          const int t0 = (a.reverse ? p.last - 1 - (c - p.first) : c) * kLaChunk;
          // TMA clips at the tensor's end, not at a row's length
          const bool by_tma = FAST || (CF::kBf16 && a.tma && (t0 + kLaChunk <= p.len || p.len == a.seqlen));
          auto tile = [&](auto width, const LaTensor& x, const CUtensorMap* map, int hx, int at, auto& ring, uint32_t full,
                          uint32_t empty, int d) {
            constexpr int DP = decltype(width)::value;
            if (ltid == 0 && !gone && ring.used()) {
              const bool free = la_wait(empty, ring.empty(), dead);
              if (CF::kBf16) gone = !free;
            }
            if (by_tma) {
              if (ltid == 0 && !gone) {
                la_expect(full, DP / 64 * kLaBlock);
#pragma unroll
                for (int j = 0; j < DP / 64; ++j) tma_load_block(base + at + j * kLaBlock, map, full, j * 64, t0, hx, p.b);
              }
            } else if constexpr (!FAST) {
              __syncwarp();
              if (CF::kLoaders > 32) asm volatile("bar.sync 2, 64;\n" ::: "memory");
              la_load_tile<T, DP>(smem + at, x, p.b, p.h, t0, p.len, d, a.vec, a.reverse ? -kLaChunk : kLaChunk, ltid,
                                  CF::kLoaders);
              if (CF::kBf16 && a.vec) {
                cp_async_commit();
                cp_async_wait_all();
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (CF::kLoaders > 32) asm volatile("bar.sync 2, 64;\n" ::: "memory");
              if (ltid == 0 && !gone) la_arrive(full);
            }
            if (!gone) ring.next();
          };
          tile(LaWidth<KD>{}, a.k, &maps.k, hk, CF::kK + rk.i * CF::kTileK, rk, full_k(rk.i), empty_k(rk.i), a.dk);
          if (!STATES)
            tile(LaWidth<KD>{}, a.q, &maps.q, hq, CF::kQ + rq.i * CF::kTileK, rq, full_q(rq.i), empty_q(rq.i), a.dk);
          if (c != a.skip_load)
            tile(LaWidth<VD>{}, a.v, &maps.v, hv, CF::kV + rv.i * CF::kTileV, rv, full_v(rv.i), empty_v(rv.i), a.dv);
        }
      }
      // the last copies into each place land before the end, also where those that they are
      // for have given up, or give up yet
      if (CF::kBf16 && ltid == 0) {
        const auto land = [&](auto& ring, int count, const auto& full) {
#pragma unroll 1
          for (int i = 0; i < count; ++i) {
            const uint32_t fills = ring.turn + (i < ring.i ? 1 : 0);
            if (fills > 0) la_wait_own(full(i), (fills - 1) & 1);
          }
        };
        land(rk, CF::RK, full_k);
        if (!STATES) land(rq, CF::RQ, full_q);
        land(rv, CF::RV, full_v);
      }
      __syncwarp();
    }
  } else if (warp >= kLaBackWarps) {
    // ---- front: weighted keys and P, a chunk ahead of the back
    regs_give<CF::kFrontRegs>();
    // 16 rows of P for each pair of warps, side 0 with every other block of columns
    const int fw = warp % 4, front = warp - kLaBackWarps, side = front / 4, ftid = tid - 32 * kLaBackWarps;
    int n = 0;
    if (!STATES) {
      // what the mask takes away is zero once and for all
      for (int i = ftid; i < CF::RP * NPX * kLaBlock / 16; i += 32 * kLaFrontWarps)
        reinterpret_cast<uint4*>(smem + CF::kP)[i] = make_uint4(0, 0, 0, 0);
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
    }
    LaRing<CF::RF> rf;
    LaRing<CF::RK> rk;
    for (int i = 0; i < work.pieces; ++i) {
      const LaPiece p = la_piece(a, work, i);
      for (int c = p.first; c < p.last; ++c, ++n) {
        const float* fac = reinterpret_cast<const float*>(smem + CF::kFac) + rf.i * CF::kFacFloats;
        char* k = smem + CF::kK + rk.i * CF::kTileK;
        la_wait(full_f(rf.i), rf.full(), dead);
        la_wait(full_k(rk.i), rk.full(), dead);
        // the keys weighted by their decay to the chunk's end (reversed: start): in the place
        // of the chunk before last, or half by half in that of the last (and when these keys
        // as they are were used: b_qk).  (With one increment a barrier tells only the last
        // chunk's, so that is waited for.)
        if (!STATES) la_wait(b_qk(n % CF::kAhead), (n / CF::kAhead) & 1, dead);
        if (CF::RW == 2 && n >= CF::ND) la_wait(b_ds(n % CF::ND), (n / CF::ND - 1) & 1, dead);
        char* wk = smem + CF::kW + (n % CF::RW) * CF::kTileW;
#pragma unroll CF::RW
        for (int half = 0; half < 2; ++half) {
          if (CF::RW == 1 && n > 0) {
            if (half) la_wait(b_ds((n - 1) % CF::ND), ((n - 1) / CF::ND) & 1, dead);
            else la_wait(b_half, (n - 1) & 1, dead);
          }
#pragma unroll
          for (int st = front; st < CF::KB * 8; st += kLaFrontWarps) {
            const int row = half * 32 + (st % 8) * 4 + lane / 8;
            const int off = (st / 8) * kLaBlock + row * kTileRow + (lane % 8) * 16;
            uint32_t in[NPI][4], out[NPW][4];
#pragma unroll
            for (int q = 0; q < NPI; ++q) {
              const uint4 y = *reinterpret_cast<const uint4*>(k + q * CF::KB * kLaBlock + off);
              in[q][0] = y.x, in[q][1] = y.y, in[q][2] = y.z, in[q][3] = y.w;
            }
            if constexpr (CF::kBf16) {
              // k (w0 + w1 + w2): a product of two bf16 is a bf16 and the bf16 that is left,
              // exactly, so four planes hold 24 bits without leaving bf16 arithmetic
              const uint32_t* w = reinterpret_cast<const uint32_t*>(fac) + 3 * kLaChunk + row;
              const uint32_t w0 = w[0], w1 = w[kLaChunk], w2 = w[2 * kLaChunk];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                out[0][e] = mul_bf16x2(in[0][e], w0);
                out[1][e] = fma_bf16x2(in[0][e], w0, neg_bf16x2(out[0][e]));
                out[2][e] = mul_bf16x2(in[0][e], w1);
                out[3][e] = fma_bf16x2(in[0][e], w2, fma_bf16x2(in[0][e], w1, neg_bf16x2(out[2][e])));
              }
            } else {
              const float wj = fac[3 * kLaChunk + row];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint64_t y = from_bf16x2(in[NPI - 1][e]);
#pragma unroll
                for (int q = NPI - 2; q >= 0; --q) y = add2(y, from_bf16x2(in[q][e]));  // exact from the smallest
                uint32_t sp[NPW];
                split2<NPW>(mul2(y, pair(wj, wj)), sp);
#pragma unroll
                for (int q = 0; q < NPW; ++q) out[q][e] = sp[q];
              }
            }
#pragma unroll
            for (int q = 0; q < NPW; ++q)
              *reinterpret_cast<uint4*>((q < NPI ? k + q * CF::KB * kLaBlock : wk + (q - NPI) * CF::KB * kLaBlock) +
                                        off) = make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
          }
          if (CF::RW == 1) {
            fence_proxy_async_smem();
            arrive(b_w(half));
          }
        }
        if (CF::RW == 2) {
          fence_proxy_async_smem();
          arrive(b_w(n % 2));
        }
        if (!STATES) {
          // P = (Q K^T) . D: 16 rows a warp, two rows a thread
          if (n >= CF::RP) la_wait(b_p_free(n % CF::RP), (n / CF::RP - 1) & 1, dead);
          tc5_fence_after();
          const uint32_t p_to = base + CF::kP + (n % CF::RP) * NPX * kLaBlock;
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
              store_blocks(p_to + q * kLaBlock + tile_unit(srow, cb * 2 + (lane >> 4)), o[q][0], o[q][1],
                           o[q][2], o[q][3]);
          }
          tc5_fence_before();
          fence_proxy_async_smem();
          arrive(b_p(n % CF::RP));
        }
        arrive(empty_f(rf.i));
        rf.next(), rk.next();
      }
    }
  } else {
    // ---- back: the state and the outputs
    regs_take<CF::kBackRegs>();
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
      LaRing<CF::RF> rf;
      int n = 0;
      for (int i = 0; i < work.pieces; ++i) {
        const LaPiece p = la_piece(a, work, i);
        const int bh = p.bh, b = p.b, h = p.h, len = p.len;
        const int step = a.workers > 0 ? 0 : work.worker % a.nseg;
        // 16-byte rows: this lane's part of token lane / 4, in memory and in the stage
        const int tok = lane / 4, c8 = quad * 32 + (lane % 4) * 8;
        char* stage = smem + CF::kStage + warp * 512;
        char* mine = stage + tok * 64 + (((lane % 4) ^ ((tok >> 1) & 3)) << 4);
        const uint32_t blocks = smem_u32(stage) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
        const int rs = a.heads * a.dv * 2;
        const bool fast = FAST && MODE == kLaOutputs ? true : CF::kBf16 && a.out_vec;
        const bool fast_x = DOTS && CF::kBf16 && (FAST || a.x_vec);
        // floats handed on by all workers, elements of the outputs
        const int64_t carried = (int64_t)a.workers * 128 * (a.dk <= 64 && a.dv <= 64 ? 64 : 128);
        const int64_t all = (int64_t)a.bh * a.seqlen * a.dv;
        char* out = static_cast<char*>(a.out) + ((int64_t)b * a.seqlen + tok) * rs + (h * a.dv + c8) * 2;
        if (p.from_carry) {
          const int at = (work.worker - 1) * 16 + warp;  // of the flags, and of the states handed on
          const unsigned* flag = a.flags + 1 + at;
          if (lane == 0 && in_range(at, a.workers * 16)) {
            unsigned there = 0;
            for (uint32_t spin = 0; spin < a.carry_spin_limit && !there && !*dead; ++spin) {
              asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(there) : "l"(flag) : "memory");
              if (!there) __nanosleep(64);
            }
            if (!there && !*dead) {
              atomicOr(&g_error_word, kErrLookback);
              *dead = 1;
            }
          }
          __syncwarp();
          const float4* from = reinterpret_cast<const float4*>(a.carry + (int64_t)at * (KH * 32));
#pragma unroll
          for (int c = 0; c < KH; c += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in_range((int64_t)at * (KH * 32) + (c / 4 * 32 + lane) * 4, 4, carried)) x = __ldcg(from + c / 4 * 32 + lane);
            S[c / 2] = pair(x.x, x.y), S[c / 2 + 1] = pair(x.z, x.w);
          }
        } else {
          const bool in = a.s_in && !STATES && vi < a.dv;
          const float* from = a.s_in + (int64_t)bh * a.s_in_head + step * a.s_in_seg + part * KH * a.sk + vi * a.sv;
#pragma unroll
          for (int c = 0; c < KH; c += 2) {
            const int kk = part * KH + c;
            S[c / 2] = pair(in && kk < a.dk && in_range(from - a.s_in, a.bh * a.s_in_head) ? from[0] : 0.f,
                            in && kk + 1 < a.dk && in_range(from + a.sk - a.s_in, a.bh * a.s_in_head) ? from[a.sk] : 0.f);
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
          const float* fac = reinterpret_cast<const float*>(smem + CF::kFac) + rf.i * CF::kFacFloats;
          const int tw = t0 + part * 16;  // this warp's tokens
          if constexpr (DOTS) {
            // the state before the chunk: S, left by the forward pass, or R, met with it there
            const int64_t at = (int64_t)bh * a.chunks + chunk;
            float4* kept = reinterpret_cast<float4*>(a.dump) + (at * CF::kHolders + part * CF::kQuads + quad) * (KH * 8) + lane;
            const int64_t all_kept = (int64_t)a.bh * a.chunks * CF::kHolders * (KH * 8);
            const auto there = [&](const float4* p) { return in_range(p - reinterpret_cast<float4*>(a.dump), all_kept); };
            if (!a.reverse) {
#pragma unroll
              for (int c = 0; c < KH; c += 4)
                if (there(kept + c / 4 * 32))
                  __stcs(kept + c / 4 * 32,
                         make_float4(pair_lo(S[c / 2]), pair_hi(S[c / 2]), pair_lo(S[c / 2 + 1]), pair_hi(S[c / 2 + 1])));
            } else {
              if (cc + 1 < p.last && lane < KH)  // the next chunk's, 128 bytes a lane
                asm volatile("prefetch.global.L2 [%0];\n" ::"l"(kept - lane - CF::kHolders * (KH * 8) + lane * 8));
              float sum = 0.f;
#pragma unroll
              for (int c = 0; c < KH; c += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (there(kept + c / 4 * 32)) x = __ldcs(kept + c / 4 * 32);
                sum += pair_lo(S[c / 2]) * x.x + pair_hi(S[c / 2]) * x.y + pair_lo(S[c / 2 + 1]) * x.z +
                       pair_hi(S[c / 2 + 1]) * x.w;
              }
#pragma unroll
              for (int o = 16; o >= 1; o /= 2) sum += __shfl_xor_sync(kFullMask, sum, o);
              const int64_t mine_at = at * 16 + part * CF::kQuads + quad;
              if (lane == 0 && in_range(mine_at, (int64_t)a.bh * a.chunks * 16)) a.flow[mine_at] = sum;
            }
          }
          la_wait(full_f(rf.i), rf.full(), dead);
          const float decay = fac[CF::kFacFloats - 4];
          const int inc = n % CF::ND;
          la_wait(b_ds(inc), (n / CF::ND) & 1, dead);
          tc5_fence_after();
          const uint64_t decay2 = pair(decay, decay);
          // 16 key indices at a time: the state, the outputs and more would not fit the registers
#pragma unroll
          for (int c = 0; c < KH; c += 16) {
            uint32_t x[16];
            tmem_ld(x, lanes + CF::cDS + inc * KD + part * KH + c);
            tmem_wait_ld(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) S[c / 2 + e] = fma2(S[c / 2 + e], decay2, pair(x[2 * e], x[2 * e + 1]));
          }
          tc5_fence_before();
          arrive(b_free(inc));
          float o[2][8], sum[4];
          if (!STATES) {
            float2 f[2];
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2)
              f[i2] = *reinterpret_cast<const float2*>(fac + 2 * kLaChunk + part * 16 + i2 * 8 + 2 * (lane % 4));
            const auto read = [&](uint32_t (&y)[2][8], int column) {
#pragma unroll
              for (int e = 0; e < 2; ++e) tmem_ld_rows16(y[e], lanes + ((uint32_t)(e * 16) << 16) + column + part * 16);
            };
            uint32_t x1[2][8], x2[2][8];
            if constexpr (DOTS) {
              // the part from the state first: its products with the rows of x
              uint4 xrow[2];
              const char* xp = la_row(a.x, b, tw + tok, h, sizeof(T)) + c8 * (int)sizeof(T);
              const int64_t xs = 8 * (int64_t)sizeof(T) * a.x.st;
              if (fast_x) {
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                  xrow[i2] = make_uint4(0, 0, 0, 0);
                  if (tw + i2 * 8 + tok < len && c8 < a.dv && la_inside(a.x, xp + i2 * xs, 8, sizeof(T)))
                    xrow[i2] = *reinterpret_cast<const uint4*>(xp + i2 * xs);
                }
                // the next chunk's rows are asked for in L2
                const int ahead = a.reverse ? -8 : 8;  // in steps of 8 tokens
                if (cc + 1 < p.last && c8 < a.dv && tw + ahead * 8 + 8 + tok < len) {
                  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(xp + ahead * xs));
                  asm volatile("prefetch.global.L2 [%0];\n" ::"l"(xp + (ahead + 1) * xs));
                }
              }
              la_wait(b_o, n & 1, dead);
              tc5_fence_after();
              read(x2, CF::cO2);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                tmem_wait_ld(x2[e]);
#pragma unroll
                for (int i2 = 0; i2 < 8; ++i2) o[e][i2] = __uint_as_float(x2[e][i2]) * (i2 % 2 ? f[i2 / 4].y : f[i2 / 4].x);
              }
              if (__builtin_expect(fast_x, CF::kBf16)) {
                // through the stage into the order of o
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                  *reinterpret_cast<uint4*>(mine) = xrow[i2];
                  __syncwarp();
                  uint32_t x4[4];
                  load_blocks_t(blocks, x4);
                  __syncwarp();
                  uint64_t y = 0;
#pragma unroll
                  for (int u = 0; u < 4; ++u)
                    y = fma2(pair(o[u / 2][4 * i2 + 2 * (u % 2)], o[u / 2][4 * i2 + 2 * (u % 2) + 1]), from_bf16x2(x4[u]), y);
                  sum[2 * i2] = pair_lo(y), sum[2 * i2 + 1] = pair_hi(y);
                }
              } else if constexpr (!FAST) {
                la_dots<T>(sum, a, o, b, h, tw, len, quad * 32, lane);
              }
              read(x1, CF::cO1);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                tmem_wait_ld(x1[e]);
#pragma unroll
                for (int i2 = 0; i2 < 8; ++i2) o[e][i2] += __uint_as_float(x1[e][i2]);
              }
            } else {
              la_wait(b_o, n & 1, dead);
              tc5_fence_after();
              read(x1, CF::cO1);
              read(x2, CF::cO2);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                tmem_wait_ld(x1[e]);
                tmem_wait_ld(x2[e]);
#pragma unroll
                for (int i2 = 0; i2 < 8; ++i2)
                  o[e][i2] = fmaf(__uint_as_float(x2[e][i2]), i2 % 2 ? f[i2 / 4].y : f[i2 / 4].x, __uint_as_float(x1[e][i2]));
              }
            }
            if (cc + 1 < p.last) give_state();
          }
          arrive(empty_f(rf.i));
          rf.next();
          if (!STATES && CF::kBf16 && __builtin_expect(fast, 1)) {
            // bf16 rows leave through 512 bytes of shared memory, 8 tokens at a time, as 64
            // bytes of a token together
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              store_blocks_t(blocks, to_bf16x2(o[0][4 * i2], o[0][4 * i2 + 1]), to_bf16x2(o[0][4 * i2 + 2], o[0][4 * i2 + 3]),
                             to_bf16x2(o[1][4 * i2], o[1][4 * i2 + 1]), to_bf16x2(o[1][4 * i2 + 2], o[1][4 * i2 + 3]));
              __syncwarp();
              const uint4 y = *reinterpret_cast<const uint4*>(mine);
              const int t = tw + i2 * 8;
              char* to = out + (int64_t)t * rs;
              if (c8 < a.dv && t + tok < len && in_range((to - static_cast<char*>(a.out)) / 2, 8, all))
                *reinterpret_cast<uint4*>(to) = y;
              __syncwarp();
            }
          } else if constexpr (!STATES && !(FAST && MODE == kLaOutputs)) {
            la_emit<T, FAST>(a, o, b, h, tw, len, quad * 32, lane);
          }
          if (DOTS) {
            // the lanes with the same tokens are 4, 8 and 16 apart
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int m = 4; m <= 16; m *= 2) sum[e] += __shfl_xor_sync(kFullMask, sum[e], m);
            if (lane < 4) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int t = tw + 2 * lane + 8 * (e / 2) + e % 2;
                const int64_t at = ((int64_t)bh * a.seqlen + t) * 4 + quad;
                if (t < len && in_range(at, (int64_t)a.bh * a.seqlen * 4)) a.dots[at] = sum[e];
              }
            }
          }
        }
        if (p.to_carry) {
          const int at = work.worker * 16 + warp;
          float4* to = reinterpret_cast<float4*>(a.carry + (int64_t)at * (KH * 32));
#pragma unroll
          for (int c = 0; c < KH; c += 4)
            if (in_range((int64_t)at * (KH * 32) + (c / 4 * 32 + lane) * 4, 4, carried)) __stcg(to + c / 4 * 32 + lane,
                   make_float4(pair_lo(S[c / 2]), pair_hi(S[c / 2]), pair_lo(S[c / 2 + 1]), pair_hi(S[c / 2 + 1])));
          __threadfence();
          __syncwarp();
          if (lane == 0 && work.worker != a.skip_publish && in_range(at, a.workers * 16))
            asm volatile("st.release.gpu.global.u32 [%0], %1;\n" ::"l"(a.flags + 1 + at), "r"(1u) : "memory");
        } else if (a.s_out && (STATES || step == a.nseg - 1) && vi < a.dv) {
          float* to = a.s_out + (int64_t)bh * a.s_out_head + step * a.s_out_seg + part * KH * a.sk + vi * a.sv;
#pragma unroll
          for (int c = 0; c < KH; ++c) {
            if (part * KH + c < a.dk && in_range(to - a.s_out, a.bh * a.s_out_head))
              *to = c % 2 ? pair_hi(S[c / 2]) : pair_lo(S[c / 2]);
            to += a.sk;
          }
        }
      }
    }
  }
  // every MMA was waited for (the last chunk's) unless a wait gave up: then the issuers'
  // last commits, waited for with a limit too, stand between those in flight and the end
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();
  if (warp == kLaMmaWarp) {
    if (*dead) {
      if (lane == 0) la_wait_own(b_end, 0);
      __syncwarp();
    }
    tmem_free(tmem, CF::kCols);
  }
}

// Segments joined: the state before each segment from the one before the first and
// what each adds, s <- e^{G} s + local, every element on its own.  `states` [bh][nseg]
// of dk x dv holds the local states and gets the starting ones.
__global__ void linattn_join_kernel(float* states, const double* seg_decay, const float* s0, int nseg,
                                    int64_t per_state) {
  const int64_t bh = blockIdx.y;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= per_state) return;
  double s = s0 ? s0[bh * per_state + i] : 0.f;  // equal factors' roundings would add up
  float* at = states + bh * nseg * per_state + i;
  const int64_t all = (int64_t)gridDim.y * nseg;  // states, and decays
  const double* decay = seg_decay + bh * nseg;
  for (int n = 0; n < nseg; n += 8) {
    float local[8];
    double a[8];  // eight segments asked for at once: only the sums are a chain
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool more = n + e + 1 < nseg;
      local[e] = more && in_range(at + (n + e) * per_state - states, all * per_state) ? at[(n + e) * per_state] : 0.f;
      a[e] = more && in_range(decay + n + e - seg_decay, all) ? exp2(decay[n + e]) : 0.0;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < nseg) {
        if (in_range(at + (n + e) * per_state - states, all * per_state)) at[(n + e) * per_state] = (float)s;
        s = fma(s, a[e], (double)local[e]);
      }
  }
}

// Gradients of shared heads: float partials [rows, heads, d] summed over the `share`
// heads that read one, in order.  VEC values a thread, an index of type I.
template <typename T, int VEC, typename I>
__global__ void __launch_bounds__(256)
linattn_share_kernel(const float* part, T* out, const int* lengths, I seqlen, I total, int heads, int share, int d) {
  const I groups = (I)(heads / share), units = (I)(d / VEC);
  const I i = (I)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const I at = i / units, c = i - at * units, row = at / groups, gr = at - row * groups;
  if (lengths) {
    const I b = row / seqlen;
    const int len = lengths[b];
    if ((int64_t)(row - b * seqlen) >= len) return;
  }
  const float* p = part + ((int64_t)row * heads + (int64_t)gr * share) * d + (int64_t)c * VEC;
  T* to = out + ((int64_t)row * groups + gr) * d + (int64_t)c * VEC;
  const int64_t all = (int64_t)(total / units) * d;  // elements of the sums
  if (!in_range(to - out, VEC, all) || !in_range(p - part, (int64_t)(share - 1) * d + VEC, all * share)) return;
  float s[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) s[e] = 0.f;
#pragma unroll 4
  for (int j = 0; j < share; ++j) {
    if constexpr (VEC == 4) {
      const float4 y = __ldcs(reinterpret_cast<const float4*>(p + (int64_t)j * d));
      s[0] += y.x, s[1] += y.y, s[2] += y.z, s[3] += y.w;
    } else {
      s[0] += p[(int64_t)j * d];
    }
  }
  if constexpr (sizeof(T) == 2 && VEC == 4)
    *reinterpret_cast<uint2*>(to) = make_uint2(to_bf16x2(s[0], s[1]), to_bf16x2(s[2], s[3]));
  else if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(to) = make_float4(s[0], s[1], s[2], s[3]);
  else if constexpr (sizeof(T) == 2)
    *to = __float2bfloat16_rn(s[0]);
  else
    *to = s[0];
}

}  // namespace ssscan

// linattn_decay_grad.cuh -- the log decays' gradient of the linear attention.
//
//   dg_t = e^{g_t} <R_t, S_{t-1}>
//
// is what flows from the tokens before t (and the initial state) to the tokens from t on
// (and the last state's gradient).  With C = 64 tokens a chunk, G the running sum of g in
// it, S the state before the chunk and R the gradient of the state behind it, it is the
// sum, for t in the chunk, of
//
//   pairs   sum_{j < t <= i}  scale e^{G_i - G_j} (q_i . k_j) (do_i . v_j)
//   a       sum_{i >= t}      a_i = scale e^{G_i} q_i . (S do_i)
//   b       sum_{j < t}       b_j = e^{G_C - G_j} k_j . (R v_j)
//   all     e^{G_C} <R, S>
//
// a and b come from the passes of dq and dk (the part of their output that goes through
// the state, times q and k), <R, S> from the states that the first leaves at every chunk
// and the second meets.  Every term holds the factor e^{g_t} itself and is only added, so
// a decay that leaves little has a gradient as exact as any other and one that leaves
// nothing a zero.  (As differences of q . dq and k . dk over up to 1024 tokens, which need
// no states at every chunk and no pairs, bf16 gradients were 1.6e-4 of their norm off at
// mean log decays of -1.6 and 1e-2 at -10, fp32 ones 1.2e-6 and 2.7e-5.)
//
// A block takes a chunk of a head: all four tiles by asynchronous copies at once (straight
// from global memory to registers, 32 columns after 32, it took three times as long), the
// products of pairs by the warps' own matrix instructions, 16 rows i a warp.  The order of
// the summed index is free, so a lane takes whole 16-byte units of a row.  The 64 x 64
// results stay in registers, 32 columns at a time, where prefix sums along j and plain
// sums along i >= t give the pairs.  Bound by instructions and latencies (6144 chunks of
// 64 x 64 bf16 heads, 133 MB: 54 us, 2.5 TB/s, issue slots 70% busy; 2080 of 128 x 128,
// 134 MB: 40 us, 3.4 TB/s); with products column after column, each waiting for the one
// before, it was 87 and 52.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "linattn_pass.cuh"

namespace ssscan {

constexpr int kLaGradThreads = 128;  // a warp for 16 rows

struct LaGradArgs {
  LaTensor q, k, v, d, g;  // d: the outputs' gradient
  const int* lengths;
  const float* dots_q;     // [batch * heads, seqlen, 4] partial a
  const float* dots_k;     // likewise b
  const float* flow;       // [batch * heads, chunks, 16] partial <R, S>
  void* out;
  int heads, seqlen, dk, dv, chunks;
  float scale;
};

// A tile of 64 rows as it is, its columns made up to whole 32 with zeros.
__host__ __device__ constexpr int la_grad_row(int d, int es) { return (d + 31) / 32 * 32 * es; }
__host__ __device__ constexpr int la_grad_smem(int dk, int dv, int es) {
  return 2 * kLaChunk * (la_grad_row(dk, es) + la_grad_row(dv, es));
}
// Rows of whole 128 bytes have their halves exchanged in turn, so that four 16-byte units
// of two neighbouring rows are in different banks: the bit of a unit's offset to turn.
__device__ __forceinline__ int la_grad_turn(int row, int bytes) { return bytes % 128 == 0 ? (row & 1) * 64 : 0; }

// The tile at t0; zeros behind the row's end and its last column.  Eight lanes a row.
template <typename T, bool VEC>
__device__ __forceinline__ void la_grad_tile(char* to, const LaTensor& x, int64_t b, int h, int t0, int len, int d) {
  constexpr int N = 16 / sizeof(T), STEP = kLaGradThreads / 8;  // elements of a unit, rows at once
  const int bytes = la_grad_row(d, sizeof(T)), row0 = threadIdx.x / 8;
  const int64_t step = STEP * x.st * (int64_t)sizeof(T);
#pragma unroll 1
  for (int unit = threadIdx.x % 8; unit * 16 < bytes; unit += 8) {
    const char* from = la_row(x, b, t0 + row0, h, sizeof(T)) + unit * 16;
    char* at = to + row0 * bytes + (unit * 16 ^ la_grad_turn(row0, bytes));
    const int col = unit * N;
#pragma unroll
    for (int row = 0; row < kLaChunk; row += STEP, from += step, at += STEP * bytes) {
      const bool in = t0 + row0 + row < len && col < d && la_inside(x, from, d - col < N ? d - col : N, sizeof(T));
      if constexpr (VEC) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(at)),
                     "l"(in ? from : static_cast<const char*>(x.ptr)), "r"(in ? 16 : 0)
                     : "memory");
      } else {
        T e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = in && col + i < d ? reinterpret_cast<const T*>(from)[i] : zero_elem<T>();
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<T*>(at)[i] = e[i];
      }
    }
  }
}

// A lane's eight elements of 32 columns, as bf16 planes: of unit c, and in fp32 of that 64
// bytes further on (`turn`: the other way round).
template <typename T, int PLANES>
__device__ __forceinline__ void la_grad_load(uint32_t (&p)[PLANES][4], const char* from, int turn) {
  if constexpr (sizeof(T) == 2) {
    const uint4 y = *reinterpret_cast<const uint4*>(from);
    p[0][0] = y.x, p[0][1] = y.y, p[0][2] = y.z, p[0][3] = y.w;
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 y = *reinterpret_cast<const float4*>(from + (64 * e ^ turn));
      uint32_t s[2][PLANES];
      split2<PLANES>(pair(y.x, y.y), s[0]);
      split2<PLANES>(pair(y.z, y.w), s[1]);
#pragma unroll
      for (int q = 0; q < PLANES; ++q) p[q][2 * e] = s[0][q], p[q][2 * e + 1] = s[1][q];
    }
  }
}

__device__ __forceinline__ void la_grad_mma(float (&c)[4], const uint32_t (&lo)[4], const uint32_t (&hi)[4],
                                            const uint32_t (&b)[4], int i) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(lo[i]), "r"(hi[i]), "r"(lo[i + 1]), "r"(hi[i + 1]), "r"(b[i]), "r"(b[i + 1]));
}

// Inner products of 16 rows of tile x (this warp's) with 32 rows of y, 8 n0 on: c[n][..] as
// the matrix instruction has them.  A product of each eight columns in turn, so that no
// instruction waits for the one before it.  fp32: three planes, the smaller products added
// on their own.
template <typename T>
__device__ __forceinline__ void la_grad_products(float (&c)[4][4], const char* x, const char* y, int n0, int d, int warp,
                                                 int lane) {
  constexpr int PLANES = sizeof(T) == 2 ? 1 : 3;
  const int r = lane / 4, bytes = la_grad_row(d, sizeof(T)), turn = la_grad_turn(r, bytes);
  const char* xr = x + (warp * 16 + r) * bytes + lane % 4 * 16;
  const char* yr = y + (n0 * 8 + r) * bytes + lane % 4 * 16;
  float small[PLANES > 1 ? 4 : 1][4];
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[n][e] = small[PLANES > 1 ? n : 0][e] = 0.f;
#pragma unroll 1
  for (int k = 0; k < d; k += 32) {
    uint32_t lo[PLANES][4], hi[PLANES][4], z[4][PLANES][4];
    const int at = sizeof(T) == 2 ? k * 2 ^ turn : k * 4;
    la_grad_load<T, PLANES>(lo, xr + at, turn);
    la_grad_load<T, PLANES>(hi, xr + 8 * bytes + at, turn);
#pragma unroll
    for (int n = 0; n < 4; ++n) la_grad_load<T, PLANES>(z[n], yr + n * 8 * bytes + at, turn);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      if constexpr (PLANES > 1) {
#pragma unroll
        for (int p = PLANES - 1; p > 0; --p)
#pragma unroll
          for (int q = p; q >= 0; --q)
#pragma unroll
            for (int n = 0; n < 4; ++n) la_grad_mma(small[n], lo[p - q], hi[p - q], z[n][q], i);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) la_grad_mma(c[n], lo[0], hi[0], z[n][0], i);
    }
  }
  if constexpr (PLANES > 1) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[n][e] += small[n][e];
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kLaGradThreads) linattn_decay_grad_kernel(const __grid_constant__ LaGradArgs a) {
  extern __shared__ __align__(128) char tiles[];
  __shared__ __align__(8) float fac[2 * kLaChunk];  // running sums of the decays, base 2: integers, fractions
  __shared__ float rest[kLaChunk];                  // what goes through the states
  __shared__ __align__(8) float part[4][kLaChunk];  // the pairs, a warp's rows
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // heads fastest: those that share keys and queries, and neighbours in memory, together
  const int h = (int)(blockIdx.x % (unsigned)a.heads);
  const int bc = (int)(blockIdx.x / (unsigned)a.heads), b = bc / a.chunks, chunk = bc % a.chunks;
  int len = a.lengths ? a.lengths[b] : a.seqlen;
  len = len < a.seqlen ? len : a.seqlen;
  const int t0 = chunk * kLaChunk;
  if (t0 >= len) return;
  const int64_t bh = (int64_t)b * a.heads + h;

  char* td = tiles;
  char* tv = td + kLaChunk * la_grad_row(a.dv, sizeof(T));
  char* tq = tv + kLaChunk * la_grad_row(a.dv, sizeof(T));
  char* tk = tq + kLaChunk * la_grad_row(a.dk, sizeof(T));
  la_grad_tile<T, VEC>(td, a.d, b, h, t0, len, a.dv);
  la_grad_tile<T, VEC>(tv, a.v, b, h, t0, len, a.dv);
  la_grad_tile<T, VEC>(tq, a.q, b, h, t0, len, a.dk);
  la_grad_tile<T, VEC>(tk, a.k, b, h, t0, len, a.dk);
  cp_async_commit();

  if (warp == 0) {  // it has the fewest products
    T g[2];
    la_fetch_decays<T>(g, a.g, b, h, t0, len, 0, lane);
    const int64_t rows = (int64_t)gridDim.x / a.chunks, at16 = (bh * a.chunks + chunk) * 16 + lane;  // batch x heads
    float all = lane < (a.dk <= 64 ? 8 : 16) && in_range(at16, rows * a.chunks * 16) ? a.flow[at16] : 0.f;
    float s[2][2];  // a and b of two tokens
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + 2 * lane + i;
      const bool in = t < len && in_range(bh * a.seqlen + t, rows * a.seqlen);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // two quadrants hold keys of at most 64, four wider ones
        const float4 y = in ? reinterpret_cast<const float4*>(e ? a.dots_k : a.dots_q)[bh * a.seqlen + t]
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        s[e][i] = y.x + y.y + (a.dk > 64 ? y.z + y.w : 0.f);
      }
    }
    const float x0 = to_f32(g[0]), x1 = to_f32(g[1]);
    int64_t at[2], total;
    la_decay_sums(at, total, x0, x1, lane);
    const float bad = __any_sync(kFullMask, x0 != x0 || x1 != x1) ? __int_as_float(0x7fffffff) : 1.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t x = la_fixed32(at[i]);
      fac[2 * lane + i] = (float)(int)(x >> 32);
      fac[kLaChunk + 2 * lane + i] = (float)(uint32_t)x * 0x1p-32f * bad;
    }
    // a from its token on, b before its token
    float from = s[0][0] + s[0][1], upto = s[1][0] + s[1][1];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const float down = __shfl_down_sync(kFullMask, from, o), up = __shfl_up_sync(kFullMask, upto, o);
      if (lane + o < 32) from += down;
      if (lane >= o) upto += up;
    }
    const float later = __shfl_down_sync(kFullMask, from, 1);  // a behind this lane's tokens
    const float earlier = __shfl_up_sync(kFullMask, upto, 1);  // b before them
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) all += __shfl_xor_sync(kFullMask, all, o);
    all *= la_exp2(la_fixed32(total)) * bad;
    const float b0 = lane ? earlier : 0.f, a1 = s[0][1] + (lane < 31 ? later : 0.f);
    rest[2 * lane] = all + b0 + (s[0][0] + a1);
    rest[2 * lane + 1] = all + (b0 + s[1][0]) + a1;
  }
  cp_async_wait_all();
  __syncthreads();

  const int c = lane % 4, i = warp * 16 + lane / 4;
  const float hi[2] = {fac[i], fac[i + 8]}, lo[2] = {fac[kLaChunk + i], fac[kLaChunk + i + 8]};
  float before[2] = {0.f, 0.f};  // of rows i and i + 8: the columns passed
  float p[8][2];  // sums over this lane's rows i >= t of A_ij, j < t, for t = 8 n + 2 c and the next
#pragma unroll
  for (int n = 0; n < 8; ++n) p[n][0] = p[n][1] = 0.f;
#pragma unroll
  for (int n0 = 0; n0 < 8; n0 += 4) {
    if (n0 * 8 >= warp * 16 + 16) break;
    float x[4][4], y[4][4];
    la_grad_products<T>(x, td, tv, n0, a.dv, warp, lane);
    la_grad_products<T>(y, tq, tk, n0, a.dk, warp, lane);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int j = (n0 + n) * 8 + c * 2;
      const float2 hj = *reinterpret_cast<const float2*>(fac + j), lj = *reinterpret_cast<const float2*>(fac + kLaChunk + j);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        // A_ij, with what the mask takes away zero
        const int row = i + 8 * z;
        const float d0 = ex2_approx((hi[z] - hj.x) + (lo[z] - lj.x)), d1 = ex2_approx((hi[z] - hj.y) + (lo[z] - lj.y));
        const float a0 = row > j ? x[n][2 * z] * (d0 * a.scale) * y[n][2 * z] : 0.f;
        const float a1 = row > j + 1 ? x[n][2 * z + 1] * (d1 * a.scale) * y[n][2 * z + 1] : 0.f;
        const float own = a0 + a1, next = __shfl_xor_sync(kFullMask, own, 1), two = own + next;
        const float other = __shfl_xor_sync(kFullMask, two, 2);
        const float upto = before[z] + ((c & 2 ? other : 0.f) + (c & 1 ? next : 0.f));
        if (row >= j) p[n0 + n][0] += upto;
        if (row >= j + 1) p[n0 + n][1] += upto + a0;
        before[z] += two + other;
      }
    }
  }
  // over the rows, the columns shared out among the lanes
#pragma unroll
  for (int o = 4; o >= 1; o /= 2)
#pragma unroll
    for (int n = 0; n < o; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool upper = lane & (4 * o);
        const float send = upper ? p[n][e] : p[n + o][e], keep = upper ? p[n + o][e] : p[n][e];
        p[n][e] = keep + __shfl_xor_sync(kFullMask, send, 4 * o);
      }
  // lane bits 4, 3, 2 are the group's 4, 2, 1
  *reinterpret_cast<float2*>(part[warp] + lane / 4 * 8 + c * 2) = make_float2(p[0][0], p[0][1]);
  __syncthreads();
  const int t = t0 + (int)threadIdx.x;
  const int64_t to = ((int64_t)b * a.seqlen + t) * a.heads + h;
  if (threadIdx.x < kLaChunk && t < len && in_range(to, (int64_t)gridDim.x / a.chunks * a.seqlen)) {
    float s = rest[threadIdx.x];
#pragma unroll
    for (int w = 0; w < 4; ++w) s += part[w][threadIdx.x];
    if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(s);
    else static_cast<float*>(a.out)[to] = s;
  }
}

}  // namespace ssscan

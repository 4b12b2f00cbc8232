// winattn_fma.cuh -- the window attention in fp32 arithmetic (ss_winattn_fwd and
// ss_winattn_bwd for float32 operands, and for bfloat16 ones whose rows are not whole
// 16-byte units).
//
// A block takes 64 queries (or, for the keys' gradients, 64 keys) of one head and walks
// the tiles of 64 keys (queries) that they meet; every product is a 64 x 64 x d or
// 64 x d x 64 one in registers, 4 x 4 or 4 x d/16 values a thread, from tiles in shared
// memory, two values at a time (fma.rn.f32x2).  The forward keeps the running maximum and sum of
// the softmax; the backward works the probabilities out again from the saved normaliser.
//
// Bound by shared memory's wavefronts and issue, each about half of what there is, and by the
// last wave of few blocks: ragged B6 L1000, 8 heads of 64 on 4, window 256: 95 us; gradients of B2
// L1024, 8 heads of 64, window 256: 145 us (16 TFLOP/s of fp32).
#pragma once

#include "tc5.cuh"
#include "winattn_common.cuh"

namespace ssscan {

constexpr int kWfTile = 64, kWfThreads = 256;

// Shared memory, in floats: rows of DP + 4 so that a quarter-warp's rows lie in different banks.
template <int DP>
struct WfCfg {
  static constexpr int kRow = DP + 4, kScoreRow = kWfTile + 4;
  static constexpr int kTile = kWfTile * kRow, kScores = kWfTile * kScoreRow;
  static constexpr int kFwd = 2 * kTile + kScores, kDq = 4 * kTile + kScores, kDkv = 4 * kTile + 2 * kScores;
};

// A tile of 64 tokens from t0 on as fp32 rows, first in a thread's registers; what is behind
// `len` or d is zero.
template <typename T, int DP>
struct WfTile {
  float4 y[DP / 16];
  __device__ __forceinline__ void fetch(const LaTensor& x, int64_t b, int h, int t0, int len, int d) {
    const bool vec = sizeof(T) == 4 && d % 4 == 0 && reinterpret_cast<uintptr_t>(x.ptr) % 16 == 0 && x.sb % 4 == 0 &&
                     x.st % 4 == 0 && x.sh % 4 == 0;
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int u = i * kWfThreads + threadIdx.x, row = u / (DP / 4), col = u % (DP / 4) * 4;
      y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t0 + row >= len || col >= d) continue;
      const char* from = la_row(x, b, t0 + row, h, sizeof(T)) + col * sizeof(T);
      if (!la_inside(x, from, d - col < 4 ? d - col : 4, sizeof(T))) continue;
      const T* p = reinterpret_cast<const T*>(from);
      if (vec) {
        y[i] = *reinterpret_cast<const float4*>(from);
      } else {
        y[i].x = to_f32(p[0]);
        if (col + 1 < d) y[i].y = to_f32(p[1]);
        if (col + 2 < d) y[i].z = to_f32(p[2]);
        if (col + 3 < d) y[i].w = to_f32(p[3]);
      }
    }
  }
  __device__ __forceinline__ void put(float* to) const {
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const int u = i * kWfThreads + threadIdx.x;
      *reinterpret_cast<float4*>(to + u / (DP / 4) * WfCfg<DP>::kRow + u % (DP / 4) * 4) = y[i];
    }
  }
};
template <typename T, int DP>
__device__ __forceinline__ void wf_load(float* to, const LaTensor& x, int64_t b, int h, int t0, int len, int d) {
  WfTile<T, DP> tile;
  tile.fetch(x, b, h, t0, len, d);
  tile.put(to);
}

// s[i][j] = <a row 4 ty + i, b row tx + 16 j>, even and odd values summed apart, two at a time
template <int DP>
__device__ __forceinline__ void wf_scores(float (&s)[4][4], const float* a, const float* b, int ty, int tx) {
  constexpr int kRow = WfCfg<DP>::kRow;
  uint64_t sum[4][4] = {};
#pragma unroll 4
  for (int k = 0; k < DP; k += 4) {
    ulonglong2 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(a + (4 * ty + i) * kRow + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(b + (tx + 16 * j) * kRow + k);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[i][j] = fma2(x[i].y, y[j].y, fma2(x[i].x, y[j].x, sum[i][j]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = pair_lo(sum[i][j]) + pair_hi(sum[i][j]);
}

// A thread's sums: rows 4 ty + i, columns 4 tx + 64 c and the three behind, in pairs
template <int DP>
using WfSums = uint64_t[4][DP / 32];

// acc[i] += sum_j w[4 ty + i][j] x row j (TRANSPOSED: w[j][4 ty + i])
template <int DP, bool TRANSPOSED>
__device__ __forceinline__ void wf_accumulate(WfSums<DP>& acc, const float* w, const float* x, int ty, int tx) {
  constexpr int kRow = WfCfg<DP>::kRow, kW = WfCfg<DP>::kScoreRow;
#pragma unroll 2
  for (int j = 0; j < kWfTile; j += 4) {
    float p[4][4];  // [i][j]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 y = *reinterpret_cast<const float4*>(TRANSPOSED ? w + (j + i) * kW + 4 * ty : w + (4 * ty + i) * kW + j);
      if (TRANSPOSED) p[0][i] = y.x, p[1][i] = y.y, p[2][i] = y.z, p[3][i] = y.w;
      else p[i][0] = y.x, p[i][1] = y.y, p[i][2] = y.z, p[i][3] = y.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(x + (j + k) * kRow + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t q = pair(p[i][k], p[i][k]);
          acc[i][2 * c] = fma2(q, y.x, acc[i][2 * c]);
          acc[i][2 * c + 1] = fma2(q, y.y, acc[i][2 * c + 1]);
        }
      }
  }
}

template <typename T>
__device__ __forceinline__ T wf_round(float x);
template <>
__device__ __forceinline__ float wf_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 wf_round<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Row r of [.., heads, d] output from this thread's columns.
template <typename T, int DP>
__device__ __forceinline__ void wf_store(T* row, const uint64_t (&acc)[DP / 32], float by, int d, int tx) {
#pragma unroll
  for (int c = 0; c < DP / 32; ++c) {
    const int at = 4 * tx + 64 * (c / 2) + 2 * (c % 2);
    if (at < d) row[at] = wf_round<T>(pair_lo(acc[c]) * by);
    if (at + 1 < d) row[at + 1] = wf_round<T>(pair_hi(acc[c]) * by);
  }
}

__device__ __forceinline__ float wf_max16(float x) {
#pragma unroll
  for (int o = 1; o < 16; o *= 2) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, o));
  return x;
}
__device__ __forceinline__ float wf_sum16(float x) {
#pragma unroll
  for (int o = 1; o < 16; o *= 2) x += __shfl_xor_sync(kFullMask, x, o);
  return x;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kWfThreads) winattn_fma_fwd_kernel(const __grid_constant__ WaArgs a) {
  using CF = WfCfg<DP>;
  extern __shared__ __align__(16) float wf_smem[];
  float *q = wf_smem, *kv = q + CF::kTile, *p = kv + CF::kTile;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int bh_all = a.batch * a.heads, bh = blockIdx.x % bh_all, b = bh / a.heads, h = bh % a.heads;
  const int tiles = gridDim.x / bh_all, r0 = (tiles - 1 - (int)(blockIdx.x / bh_all)) * kWfTile;  // long rows first
  const int len = wa_length(a.lengths, b, a.seqlen);
  if (r0 >= len) return;
  const int r1 = r0 + kWfTile < len ? r0 + kWfTile : len;
  wf_load<T, DP>(q, a.q, b, h, r0, len, a.d);
  const float by = a.scale * kLog2e;  // exponents are of base 2
  WfSums<DP> acc = {};
  float top[4], sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) top[i] = -CUDART_INF_F, sum[i] = 0.f;
  const WaKeyTiles<kWfTile> keys(r0, r1, a.window, a.sinks);
  WfTile<T, DP> next;  // the values, or the next keys, on their way while the products before them run
  next.fetch(a.k, b, h, keys.at(0) * kWfTile, len, a.d);
  for (int n = 0; n < keys.count; ++n) {
    const int c0 = keys.at(n) * kWfTile;
    __syncthreads();
    next.put(kv);
    __syncthreads();
    next.fetch(a.v, b, h, c0, len, a.d);
    float s[4][4];
    wf_scores<DP>(s, q, kv, ty, tx);
    const bool all = wa_all_seen(r0, r1, c0, c0 + kWfTile, a.window, a.sinks);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float most = -CUDART_INF_F;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = all || wa_sees(r0 + 4 * ty + i, c0 + tx + 16 * j, a.window, a.sinks) ? s[i][j] * by : -CUDART_INF_F;
        most = fmaxf(most, s[i][j]);
      }
      most = fmaxf(top[i], wf_max16(most));
      // a row that has seen nothing yet: exponents from 0, so that nothing is exp(-inf - -inf)
      const float from = most == -CUDART_INF_F ? 0.f : most;
      const float fade = exp2f(top[i] - from);
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - from);
        add += s[i][j];
        p[(4 * ty + i) * CF::kScoreRow + tx + 16 * j] = s[i][j];
      }
      top[i] = most;
      sum[i] = sum[i] * fade + wf_sum16(add);
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) acc[i][c] = mul2(acc[i][c], pair(fade, fade));
    }
    __syncthreads();
    next.put(kv);
    __syncthreads();
    if (n + 1 < keys.count) next.fetch(a.k, b, h, keys.at(n + 1) * kWfTile, len, a.d);
    wf_accumulate<DP, false>(acc, p, kv, ty, tx);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = r0 + 4 * ty + i;
    if (t >= len) continue;
    const int64_t at = (((int64_t)b * a.seqlen + t) * a.heads + h) * a.d, all = (int64_t)bh_all * a.seqlen;
    if (in_range(at, a.d, all * a.d)) wf_store<T, DP>(static_cast<T*>(a.out) + at, acc[i], 1.f / sum[i], a.d, tx);
    const int64_t l = (int64_t)bh * a.seqlen + t;
    if (a.lse && tx == 0 && in_range(l, all)) a.lse[l] = (top[i] + log2f(sum[i])) * kLn2;
  }
}

// p = exp(s - lse) of a tile's scores, and ds = p (dp - delta) (DELTA: p dp); both zero where
// nothing is seen.
template <bool DELTA = false>
__device__ __forceinline__ void wf_probabilities(float (&s)[4][4], float (&dp)[4][4], const WaArgs& a, int64_t bh, int r0,
                                                 int c0, int len, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = r0 + 4 * ty + i;
    const bool real = t < len && in_range(bh * a.seqlen + t, (int64_t)a.batch * a.heads * a.seqlen);
    const float lse = real ? a.lse[bh * a.seqlen + t] * kLog2e : 0.f, delta = real && !DELTA ? a.delta[bh * a.seqlen + t] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool seen = real && wa_sees(t, c0 + tx + 16 * j, a.window, a.sinks);
      s[i][j] = seen ? exp2f(s[i][j] * (a.scale * kLog2e) - lse) : 0.f;
      dp[i][j] = seen ? s[i][j] * (dp[i][j] - delta) : 0.f;
    }
  }
}

template <int DP>
__device__ __forceinline__ void wf_put_scores(float* to, const float (&s)[4][4], int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) to[(4 * ty + i) * WfCfg<DP>::kScoreRow + tx + 16 * j] = s[i][j];
}

// dQ of block `block`'s 64 queries; DELTA: their sums p (do . v) instead, which are do . o with
// an o that is not rounded.
template <typename T, int DP, bool DELTA = false>
__device__ __forceinline__ void wf_dq(const WaArgs& a, int block, int blocks) {
  using CF = WfCfg<DP>;
  extern __shared__ __align__(16) float wf_smem[];
  float *q = wf_smem, *g = q + CF::kTile, *k = g + CF::kTile, *v = k + CF::kTile, *ds = v + CF::kTile;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int bh_all = a.batch * a.heads, bh = block % bh_all, b = bh / a.heads, h = bh % a.heads;
  const int tiles = blocks / bh_all, r0 = (tiles - 1 - block / bh_all) * kWfTile;
  const int len = wa_length(a.lengths, b, a.seqlen);
  if (r0 >= len) return;
  const int r1 = r0 + kWfTile < len ? r0 + kWfTile : len;
  wf_load<T, DP>(q, a.q, b, h, r0, len, a.d);
  wf_load<T, DP>(g, a.g, b, h, r0, len, a.d);
  WfSums<DP> acc = {};
  float delta[4] = {};
  const WaKeyTiles<kWfTile> keys(r0, r1, a.window, a.sinks);
  for (int n = 0; n < keys.count; ++n) {
    const int c0 = keys.at(n) * kWfTile;
    __syncthreads();
    wf_load<T, DP>(k, a.k, b, h, c0, len, a.d);
    wf_load<T, DP>(v, a.v, b, h, c0, len, a.d);
    __syncthreads();
    float s[4][4], dp[4][4];
    wf_scores<DP>(s, q, k, ty, tx);
    wf_scores<DP>(dp, g, v, ty, tx);
    wf_probabilities<DELTA>(s, dp, a, bh, r0, c0, len, ty, tx);
    if constexpr (DELTA) {
#pragma unroll
      for (int i = 0; i < 4; ++i) delta[i] += wf_sum16(dp[i][0] + dp[i][1] + dp[i][2] + dp[i][3]);
    } else {
      wf_put_scores<DP>(ds, dp, ty, tx);
      __syncthreads();
      wf_accumulate<DP, false>(acc, ds, k, ty, tx);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = r0 + 4 * ty + i;
    if constexpr (DELTA) {
      const int64_t l = (int64_t)bh * a.seqlen + t;
      if (tx == 0 && t < len && in_range(l, (int64_t)bh_all * a.seqlen)) a.delta[l] = delta[i];
    } else {
      const int64_t at = (((int64_t)b * a.seqlen + t) * a.heads + h) * a.d;
      if (t < len && in_range(at, a.d, (int64_t)bh_all * a.seqlen * a.d))
        wf_store<T, DP>(static_cast<T*>(a.out) + at, acc[i], a.scale, a.d, tx);
    }
  }
}

// Where a block of the keys' gradients stands: its key tile, the query tiles that it takes,
// and whether it leaves a partial sum.
template <int N>
struct WaKeyBlock {
  int tile, from, to, piece;
  bool partial;
  __device__ __forceinline__ WaKeyBlock(const WaArgs& a, int item, int len) {
    const int pieces = a.sink_tiles * a.pieces;  // the sinks' pieces come first, they are as long as any
    partial = true;
    if (item < pieces) {
      tile = item / a.pieces;
      piece = 1 + item % a.pieces;
    } else {
      tile = item - pieces;
      piece = 0;
      partial = a.pieces > 0 && tile < a.sink_tiles;
    }
    const int c0 = tile * N, c1 = c0 + N < len ? c0 + N : len;
    const WaQueryTiles<N> queries(c0, c1, len, a.window, a.sinks);
    from = queries.first;
    to = a.pieces > 0 ? queries.near : queries.last;
    if (piece > 0) {
      const int64_t at = (int64_t)queries.near + (int64_t)(piece - 1) * a.piece_tiles, end = at + a.piece_tiles;
      from = at < queries.last ? (int)at : queries.last;
      to = end < queries.last ? (int)end : queries.last;
    }
  }
};
// Element offset of a partial sum: dk, then dv, of [N, d] each.
template <int N>
__device__ __forceinline__ int64_t wa_part(const WaArgs& a, int64_t bh_kv, int tile, int piece) {
  return ((bh_kv * a.sink_tiles + tile) * (1 + a.pieces) + piece) * 2 * N * a.d;
}

// dK and dV of block `block`'s 64 keys.
template <typename T, int DP>
__device__ __forceinline__ void wf_dkv(const WaArgs& a, int block) {
  using CF = WfCfg<DP>;
  extern __shared__ __align__(16) float wf_smem[];
  float *k = wf_smem, *v = k + CF::kTile, *q = v + CF::kTile, *g = q + CF::kTile;
  float *p = g + CF::kTile, *ds = p + CF::kScores;
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int kv_heads = a.heads / a.share, bh_all = a.batch * kv_heads;
  const int bh = block % bh_all, b = bh / kv_heads, hk = bh % kv_heads;
  const int len = wa_length(a.lengths, b, a.seqlen);
  const WaKeyBlock<kWfTile> w(a, block / bh_all, len);
  const int c0 = w.tile * kWfTile;
  if (c0 >= len) return;
  wf_load<T, DP>(k, a.k, b, hk * a.share, c0, len, a.d);
  wf_load<T, DP>(v, a.v, b, hk * a.share, c0, len, a.d);
  WfSums<DP> dk = {}, dv = {};
  for (int h = hk * a.share; h < (hk + 1) * a.share; ++h)
    for (int n = w.from; n < w.to; ++n) {
      const int r0 = n * kWfTile;
      __syncthreads();
      wf_load<T, DP>(q, a.q, b, h, r0, len, a.d);
      wf_load<T, DP>(g, a.g, b, h, r0, len, a.d);
      __syncthreads();
      float s[4][4], dp[4][4];
      wf_scores<DP>(s, q, k, ty, tx);
      wf_scores<DP>(dp, g, v, ty, tx);
      wf_probabilities(s, dp, a, (int64_t)b * a.heads + h, r0, c0, len, ty, tx);
      wf_put_scores<DP>(p, s, ty, tx);
      wf_put_scores<DP>(ds, dp, ty, tx);
      __syncthreads();
      wf_accumulate<DP, true>(dv, p, g, ty, tx);
      wf_accumulate<DP, true>(dk, ds, q, ty, tx);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = 4 * ty + i, t = c0 + j;
    if (t >= len) continue;
    if (w.partial) {
      const int64_t at = wa_part<kWfTile>(a, bh, w.tile, w.piece) + (int64_t)j * a.d;
      wf_store<float, DP>(a.part + at, dk[i], a.scale, a.d, tx);
      wf_store<float, DP>(a.part + at + kWfTile * a.d, dv[i], 1.f, a.d, tx);
      continue;
    }
    const int64_t at = (((int64_t)b * a.seqlen + t) * kv_heads + hk) * a.d;
    if (!in_range(at, a.d, (int64_t)bh_all * a.seqlen * a.d)) continue;
    wf_store<T, DP>(static_cast<T*>(a.dk) + at, dk[i], a.scale, a.d, tx);
    wf_store<T, DP>(static_cast<T*>(a.dv) + at, dv[i], 1.f, a.d, tx);
  }
}

// Both in one launch, the keys' blocks first: neither alone fills the last wave (batch 2, 1024
// tokens, 8 heads of 64: 256 blocks each on 148 SMs; two launches took 172 us, one 145).
template <typename T, int DP>
__global__ void __launch_bounds__(kWfThreads) winattn_fma_bwd_kernel(const __grid_constant__ WaArgs a) {
  if ((int)blockIdx.x < a.items) wf_dkv<T, DP>(a, blockIdx.x);
  else wf_dq<T, DP>(a, blockIdx.x - a.items, gridDim.x - a.items);
}

template <typename T, int DP>
__global__ void __launch_bounds__(kWfThreads) winattn_fma_delta_kernel(const __grid_constant__ WaArgs a) {
  wf_dq<T, DP, true>(a, blockIdx.x, gridDim.x);
}

// delta = do . o of every row, a warp each.
template <typename T>
__global__ void __launch_bounds__(256) winattn_delta_kernel(const __grid_constant__ WaArgs a) {
  const int lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32, all = (int64_t)a.batch * a.heads * a.seqlen;
  if (row >= all) return;
  const int h = (int)(row % a.heads);
  const int64_t bt = row / a.heads, t = bt % a.seqlen, b = bt / a.seqlen;
  if (t >= wa_length(a.lengths, b, a.seqlen)) return;
  const char *o = la_row(a.o, b, t, h, sizeof(T)), *g = la_row(a.g, b, t, h, sizeof(T));
  float sum = 0.f;
  if (la_inside(a.o, o, a.d, sizeof(T)) && la_inside(a.g, g, a.d, sizeof(T)))
    for (int i = lane; i < a.d; i += 32)
      sum = fmaf(to_f32(reinterpret_cast<const T*>(o)[i]), to_f32(reinterpret_cast<const T*>(g)[i]), sum);
#pragma unroll
  for (int o2 = 16; o2 > 0; o2 /= 2) sum += __shfl_xor_sync(kFullMask, sum, o2);
  const int64_t at = (b * a.heads + h) * a.seqlen + t;
  if (lane == 0 && in_range(at, all)) a.delta[at] = sum;
}

// The sinks' partial gradients added up, N tokens a tile, VEC values of a row a thread.
template <typename T, int N, int VEC>
__global__ void __launch_bounds__(256) winattn_sinks_kernel(const __grid_constant__ WaArgs a) {
  const int kv_heads = a.heads / a.share;
  const int64_t bh = blockIdx.y, b = bh / kv_heads, hk = bh % kv_heads;
  const unsigned i = (blockIdx.x * 256 + threadIdx.x) * VEC, tile_values = 2 * N * a.d;  // of [sink_tiles, 2, N, d]
  if (i >= a.sink_tiles * tile_values) return;
  const unsigned tile = i / tile_values, rest = i - tile * tile_values, row = rest / (unsigned)a.d;
  const int64_t t = (int64_t)tile * N + row % N;
  if (t >= wa_length(a.lengths, b, a.seqlen)) return;
  const float* part = a.part + wa_part<N>(a, bh, tile, 0) + rest;
  float sum[VEC] = {};
  for (int piece = 0; piece <= a.pieces; ++piece, part += tile_values) {
    if constexpr (VEC == 4) {
      const float4 x = *reinterpret_cast<const float4*>(part);
      sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
    } else {
      sum[0] += *part;
    }
  }
  const int64_t at = ((b * a.seqlen + t) * kv_heads + hk) * a.d + (rest - row * a.d);
  if (!in_range(at, VEC, (int64_t)a.batch * kv_heads * a.seqlen * a.d)) return;
  T* to = static_cast<T*>(row < N ? a.dk : a.dv) + at;
#pragma unroll
  for (int e = 0; e < VEC; ++e) to[e] = wf_round<T>(sum[e]);
}

}  // namespace ssscan

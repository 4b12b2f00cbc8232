// winattn_step.cuh -- the newest tokens of each sequence over its paged cache
// (ss_winattn_step).
//
// A group of `share` heads reads one head of keys and values, so a block takes up to 16
// (query, head) rows of a group and walks that group's visible tokens, 64 at a time: those
// of the sinks that the window does not reach, then the window's, laid end to end, so that
// nothing else of the cache is touched.  A long walk is cut between the blocks of a
// cluster, whose maxima, sums and outputs are joined through their shared memory.
#pragma once

#include <cooperative_groups.h>

#include "rotate.cuh"
#include "winattn_common.cuh"

namespace ssscan {

constexpr int kWsRows = 16, kWsChunk = 64, kWsThreads = 128;

struct WaStepArgs {
  LaTensor q;          // [batch, tokens, heads, d]
  WaPages pages;
  const int* lengths;
  void* out;           // [batch, tokens, heads, d] contiguous
  int64_t window;
  int sinks, tokens, heads, share, d, batch;
  int row_tiles;       // blocks of kWsRows rows of a group
  float scale;
};

// The tokens that the queries at positions p0 .. len - 1 (p0 may be negative) see any of.
struct WaVisible {
  int sink, first, count;
  __device__ __forceinline__ WaVisible(int p0, int len, int64_t window, int sinks) {
    const int64_t from = (int64_t)(p0 > 0 ? p0 : 0) + 1 - window;
    first = from > 0 ? (int)from : 0;
    sink = sinks < first ? sinks : first;
    count = len > 0 ? sink + len - first : 0;
  }
  __device__ __forceinline__ int at(int i) const { return i < sink ? i : first + i - sink; }
};

template <int DP>
struct WsFmaCfg {
  static constexpr int kRow = DP + 4;
  static constexpr int kQ = 0, kKv = kWsRows * DP, kP = kKv + 2 * kWsChunk * kRow, kStat = kP + kWsRows * kWsChunk;
  static constexpr int kAcc = kStat + 3 * kWsRows, kFloats = kAcc + kWsRows * DP;
};

template <typename T, int DP>
__global__ void __launch_bounds__(kWsThreads) winattn_step_fma_kernel(const __grid_constant__ WaStepArgs a) {
  namespace cg = cooperative_groups;
  using CF = WsFmaCfg<DP>;
  extern __shared__ __align__(16) float ws_smem[];
  float *q = ws_smem + CF::kQ, *k = ws_smem + CF::kKv, *v = k + kWsChunk * CF::kRow, *p = ws_smem + CF::kP;
  float *top = ws_smem + CF::kStat, *sum = top + kWsRows, *fade = sum + kWsRows, *acc_out = ws_smem + CF::kAcc;
  __shared__ int at[kWsChunk], page[kWsChunk];  // a chunk's tokens, -1 where there is none, and their pages
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int tid = threadIdx.x, kv_heads = a.heads / a.share;
  const int b = blockIdx.z / kv_heads, hk = blockIdx.z % kv_heads;
  const int row0 = blockIdx.y * kWsRows, all_rows = a.tokens * a.share;
  const int rows = all_rows - row0 < kWsRows ? all_rows - row0 : kWsRows;
  const int len = wa_length(a.lengths, b, a.pages.max_pages * a.pages.page_size);
  // row r of the group: token r / share, head r % share
  const auto token = [&](int r) { return (row0 + r) / a.share; };
  const auto head = [&](int r) { return hk * a.share + (row0 + r) % a.share; };
  const int last = len - a.tokens + token(rows - 1) + 1;  // behind the block's newest query
  const WaVisible seen(len - a.tokens + token(0), last, a.window, a.sinks);
  for (int i = tid; i < kWsRows * DP; i += kWsThreads) {
    const int r = i / DP, c = i % DP;
    float x = 0.f;
    if (r < rows && c < a.d) {
      const char* from = la_row(a.q, b, token(r), head(r), sizeof(T)) + c * sizeof(T);
      if (la_inside(a.q, from, 1, sizeof(T))) x = to_f32(*reinterpret_cast<const T*>(from)) * (a.scale * kLog2e);
    }
    q[i] = x;
  }
  if (tid < kWsRows) top[tid] = -CUDART_INF_F, sum[tid] = 0.f;
  float acc[kWsRows] = {};
  const int chunks = (seen.count + kWsChunk - 1) / kWsChunk, each = (chunks + parts - 1) / parts;
  const int n1 = (part + 1) * each < chunks ? (part + 1) * each : chunks;
  for (int n = part * each; n < n1; ++n) {
    __syncthreads();
    if (tid < kWsChunk) {
      const int i = n * kWsChunk + tid, t = i < seen.count ? seen.at(i) : -1;
      const int64_t of = t >= 0 ? wa_page_of(a.pages, b, t) : -1;
      at[tid] = of >= 0 ? t : -1;
      page[tid] = (int)of;
    }
    __syncthreads();
    for (int u = tid; u < kWsChunk * (DP / 4); u += kWsThreads) {
      const int j = u / (DP / 4), c = u % (DP / 4) * 4;
      float4 x[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const LaTensor& y = w ? a.pages.v : a.pages.k;
        float e[4] = {0.f, 0.f, 0.f, 0.f};
        if (at[j] >= 0 && c < a.d) {
          const char* from = la_row(y, page[j], at[j] % a.pages.page_size, hk, sizeof(T)) + c * sizeof(T);
          const int m = a.d - c < 4 ? a.d - c : 4;
          if (la_inside(y, from, m, sizeof(T)))
            for (int z = 0; z < m; ++z) e[z] = to_f32(reinterpret_cast<const T*>(from)[z]);
        }
        x[w] = make_float4(e[0], e[1], e[2], e[3]);
      }
      *reinterpret_cast<float4*>(k + j * CF::kRow + c) = x[0];
      *reinterpret_cast<float4*>(v + j * CF::kRow + c) = x[1];
    }
    __syncthreads();
    {  // scores: a token and half of the rows a thread
      const int j = tid % kWsChunk, r0 = tid / kWsChunk * (kWsRows / 2);
      float s[kWsRows / 2] = {};
      for (int c = 0; c < DP; c += 4) {
        const float4 y = *reinterpret_cast<const float4*>(k + j * CF::kRow + c);
#pragma unroll
        for (int r = 0; r < kWsRows / 2; ++r) {
          const float4 x = *reinterpret_cast<const float4*>(q + (r0 + r) * DP + c);
          s[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < kWsRows / 2; ++r) {
        const int t = len - a.tokens + token(r0 + r);
        const bool ok = r0 + r < rows && at[j] >= 0 && wa_sees(t, at[j], a.window, a.sinks);
        p[(r0 + r) * kWsChunk + j] = ok ? s[r] : -CUDART_INF_F;
      }
    }
    __syncthreads();
    for (int r = tid / 32; r < kWsRows; r += kWsThreads / 32) {  // softmax: a warp a row
      const int lane = tid % 32;
      float x0 = p[r * kWsChunk + lane], x1 = p[r * kWsChunk + 32 + lane];
      float most = fmaxf(x0, x1);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) most = fmaxf(most, __shfl_xor_sync(kFullMask, most, o));
      most = fmaxf(most, top[r]);
      const float from = most == -CUDART_INF_F ? 0.f : most;
      x0 = exp2f(x0 - from), x1 = exp2f(x1 - from);
      float add = x0 + x1;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) add += __shfl_xor_sync(kFullMask, add, o);
      p[r * kWsChunk + lane] = x0, p[r * kWsChunk + 32 + lane] = x1;
      __syncwarp();
      if (lane == 0) {
        fade[r] = exp2f(top[r] - from);
        sum[r] = sum[r] * fade[r] + add;
        top[r] = most;
      }
    }
    __syncthreads();
    if (tid < DP) {  // outputs: a column a thread
#pragma unroll
      for (int r = 0; r < kWsRows; ++r) acc[r] *= fade[r];
      for (int j = 0; j < kWsChunk; j += 4) {
        float y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] = v[(j + z) * CF::kRow + tid];
#pragma unroll
        for (int r = 0; r < kWsRows; ++r) {
          const float4 x = *reinterpret_cast<const float4*>(p + r * kWsChunk + j);
          acc[r] = fmaf(x.x, y[0], fmaf(x.y, y[1], fmaf(x.z, y[2], fmaf(x.w, y[3], acc[r]))));
        }
      }
    }
  }
  if (tid < DP)
    for (int r = 0; r < kWsRows; ++r) acc_out[r * DP + tid] = acc[r];
  cluster.sync();
  // the blocks' parts joined, each block a share of the values
  for (int i = part * kWsThreads + tid; i < rows * a.d; i += parts * kWsThreads) {
    const int r = i / a.d, c = i % a.d;
    float most = -CUDART_INF_F;
    for (int x = 0; x < parts; ++x) most = fmaxf(most, cluster.map_shared_rank(top, x)[r]);
    float total = 0.f, o = 0.f;
    if (most != -CUDART_INF_F)
      for (int x = 0; x < parts; ++x) {
        const float by = exp2f(cluster.map_shared_rank(top, x)[r] - most);
        total = fmaf(by, cluster.map_shared_rank(sum, x)[r], total);
        o = fmaf(by, cluster.map_shared_rank(acc_out, x)[r * DP + c], o);
      }
    const int64_t to = (((int64_t)b * a.tokens + token(r)) * a.heads + head(r)) * a.d + c;
    if (in_range(to, (int64_t)a.batch * a.tokens * a.heads * a.d))
      rot_set(static_cast<T*>(a.out)[to], total > 0.f ? o / total : 0.f);
  }
  cluster.sync();  // a block's shared memory stays until all have read it
}

}  // namespace ssscan

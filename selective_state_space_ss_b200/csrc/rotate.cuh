// rotate.cuh -- the rotation of positions, by itself (ss_rotate) and on the way into a
// paged cache (ss_kv_append).
//
// Pair i of a head's first 2 * half values is turned by a = position * inv_freq[i],
//
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a).
//
// The angle is a product of a 32-bit integer and a float, exact in a double; it is brought
// into +-pi there (fp32 has lost all of it at a position of 2^24), and its sine and cosine
// are rounded to fp32 once.  A block works them out for a few tokens and then goes over all
// their heads: bound by memory, each value read once and written once.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "heads.cuh"
#include "scan_common.cuh"

namespace ssscan {

constexpr int kRotThreads = 256;

// The cache, as the kernels have it.
struct WaPages {
  LaTensor k, v;  // batch axis: pages; token axis: tokens of a page
  int64_t num_pages;
  const int* table;
  int page_size, max_pages;
};

struct RotArgs {
  LaTensor q, k, v;         // q.ptr or v.ptr null: none
  void *q_out, *k_out;      // contiguous; k_out nullable
  WaPages pages;            // table null: no cache
  const int *starts, *counts;
  const float* inv_freq;
  int half, interleaved, inverse;
  int64_t batch;
  int tokens, heads, kv_heads, d;  // heads 0 without q
  int block_tokens, blocks;        // tokens of a block, blocks of a row
};

// Where token t of row b lies in its cache, in elements of k (or v) before the head; -1: nowhere.
__device__ __forceinline__ int64_t wa_page_of(const WaPages& p, int64_t b, int64_t t) {
  const int64_t page = t / p.page_size;
  if (t < 0 || page >= p.max_pages) return -1;
  const int at = p.table[b * p.max_pages + page];
  return at >= 0 && at < p.num_pages ? at : -1;
}

// VEC values of T as they are stored.
template <typename T, int VEC>
struct RotUnit {
  T x[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ void rot_load(RotUnit<T, VEC>& u, const T* from) {
  if constexpr (VEC * sizeof(T) == 16) *reinterpret_cast<uint4*>(u.x) = *reinterpret_cast<const uint4*>(from);
  else u.x[0] = from[0];
}
template <typename T, int VEC>
__device__ __forceinline__ void rot_store(T* to, const RotUnit<T, VEC>& u) {
  if constexpr (VEC * sizeof(T) == 16) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(u.x);
  else to[0] = u.x[0];
}
__device__ __forceinline__ void rot_set(float& to, float x) { to = x; }
__device__ __forceinline__ void rot_set(__nv_bfloat16& to, float x) { to = __float2bfloat16_rn(x); }

__device__ __forceinline__ void rot_turn(float& x, float& y, float c, float s) {
  const float x0 = x;
  x = fmaf(x0, c, -y * s);
  y = fmaf(x0, s, y * c);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kRotThreads) rotate_kernel(const __grid_constant__ RotArgs a) {
  extern __shared__ float rot_smem[];  // [block_tokens][half] cosines, then sines
  const int64_t b = blockIdx.x / a.blocks;
  const int t0 = (int)(blockIdx.x % a.blocks) * a.block_tokens;
  int end = a.tokens;
  if (a.counts) {
    const int n = a.counts[b];
    end = n < 0 ? 0 : n < end ? n : end;
  }
  const int start = a.starts ? a.starts[b] : 0;
  const int n = end - t0 < a.block_tokens ? end - t0 : a.block_tokens;
  if (n <= 0) return;
  float *cosines = rot_smem, *sines = rot_smem + a.block_tokens * a.half;
  for (int i = threadIdx.x; i < n * a.half; i += kRotThreads) {
    const int t = i / a.half;
    const double x = (double)((int64_t)start + t0 + t) * (double)a.inv_freq[i - t * a.half];
    // x - 2 pi k, 2 pi in two doubles
    const double k = rint(x * 0.15915494309189535);
    double c, s;
    sincos(fma(k, -2.4492935982947064e-16, fma(k, -6.283185307179586, x)), &s, &c);
    cosines[i] = (float)c;
    sines[i] = a.inverse ? -(float)s : (float)s;
  }
  __syncthreads();
  const int units = a.d / VEC, items = (units + 1) / 2;  // an item: two units
  const int half_units = a.interleaved ? 0 : a.half / VEC;
  const int rows = a.heads + (a.v.ptr ? 2 : 1) * a.kv_heads;
  const int64_t bt0 = b * a.tokens + t0;
  for (int e = threadIdx.x; e < n * rows * items; e += kRotThreads) {
    const int r = e / items, i = e - r * items, t = r / rows, h = r - t * rows;
    const bool is_q = h < a.heads, is_v = h >= a.heads + a.kv_heads;
    const int hx = is_q ? h : is_v ? h - a.heads - a.kv_heads : h - a.heads;
    const LaTensor& x = is_q ? a.q : is_v ? a.v : a.k;
    // the units of this item: a pair of the two halves, or neighbours
    const bool halves = !is_v && i < half_units;
    const int first = halves ? i : 2 * i;
    const int c0 = first * VEC, c1 = halves ? c0 + a.half : c0 + VEC;
    const T* from = reinterpret_cast<const T*>(la_row(x, b, t0 + t, hx, sizeof(T)));
    RotUnit<T, VEC> y0, y1;
    const bool two = c1 < a.d;
    if (!la_inside(x, reinterpret_cast<const char*>(from + c0), VEC, sizeof(T)) ||
        (two && !la_inside(x, reinterpret_cast<const char*>(from + c1), VEC, sizeof(T))))
      continue;
    rot_load<T, VEC>(y0, from + c0);
    if (two) rot_load<T, VEC>(y1, from + c1);
    const float *c = cosines + t * a.half, *s = sines + t * a.half;
    if (halves) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float p = to_f32(y0.x[j]), q = to_f32(y1.x[j]);
        rot_turn(p, q, c[c0 + j], s[c0 + j]);
        rot_set(y0.x[j], p), rot_set(y1.x[j], q);
      }
    } else if (a.interleaved && !is_v) {
      if constexpr (VEC == 1) {
        // one value a unit: the two units of the item are the pair
        if (two && c1 < 2 * a.half) {
          float p = to_f32(y0.x[0]), q = to_f32(y1.x[0]);
          rot_turn(p, q, c[c0 / 2], s[c0 / 2]);
          rot_set(y0.x[0], p), rot_set(y1.x[0], q);
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          if (c0 + j < 2 * a.half) {
            float p = to_f32(y0.x[j]), q = to_f32(y0.x[j + 1]);
            rot_turn(p, q, c[(c0 + j) / 2], s[(c0 + j) / 2]);
            rot_set(y0.x[j], p), rot_set(y0.x[j + 1], q);
          }
          if (two && c1 + j < 2 * a.half) {
            float p = to_f32(y1.x[j]), q = to_f32(y1.x[j + 1]);
            rot_turn(p, q, c[(c1 + j) / 2], s[(c1 + j) / 2]);
            rot_set(y1.x[j], p), rot_set(y1.x[j + 1], q);
          }
        }
      }
    }
    const auto put = [&](T* to) {
      rot_store<T, VEC>(to + c0, y0);
      if (two) rot_store<T, VEC>(to + c1, y1);
    };
    const int64_t bt = bt0 + t, all = a.batch * a.tokens;
    if (is_q) {
      const int64_t at = (bt * a.heads + hx) * a.d;
      if (in_range(at, a.d, all * a.heads * a.d)) put(static_cast<T*>(a.q_out) + at);
      continue;
    }
    if (!is_v && a.k_out) {
      const int64_t at = (bt * a.kv_heads + hx) * a.d;
      if (in_range(at, a.d, all * a.kv_heads * a.d)) put(static_cast<T*>(a.k_out) + at);
    }
    if (a.pages.table && start >= 0) {
      const int64_t pos = (int64_t)start + t0 + t, page = wa_page_of(a.pages, b, pos);
      const LaTensor& to = is_v ? a.pages.v : a.pages.k;
      if (page >= 0) {
        const char* at = la_row(to, page, pos % a.pages.page_size, hx, sizeof(T));
        if (la_inside(to, at, a.d, sizeof(T))) put(reinterpret_cast<T*>(const_cast<char*>(at)));
      }
    }
  }
}

}  // namespace ssscan

// state_pool.cuh -- states in 8 bits: each row of `width` values as int8 steps of a
// scale of its own.  Bound by memory: 4 bytes in and 1 out a value, or the other way.
// 64 sequences of 5120 rows of 128, written and read back (422 MB): 72 us, 5.9 TB/s, 90%
// of the copy rate (store 39 us, load 34).  Codes through conversions, with ties looked at
// for every value, kept the store at 63 us and the arithmetic at 72%; a thread's 64 bytes
// of output in a row kept the load at 51.
#pragma once

#include <stdint.h>

#include "scan_common.cuh"

namespace ssscan {

constexpr int kPoolThreads = 256;

struct PoolArgs {
  float* state;
  int8_t* codes;
  float* scales;
  int64_t num_slots;
  const int* slots;
  int64_t batch, rows;
  int width;
};

// x / scale to the nearest integer, ties to even, of the exact quotient, |x / scale| at
// most 127: the low byte of the result (it is 1.5 * 2^23 more than the code, so that its
// last bits are the code's).  The fp32 product lands within one of it; the remainder
// x - n scale is exact (both terms are multiples of the smaller one's last place and it
// has fewer than 24 bits), and where it is not below half a scale it says what is nearer.
__device__ __forceinline__ uint32_t pool_code(float x, float scale, float half, float inv) {
  float t = fmaf(x, inv, 12582912.f);
  const float n = t - 12582912.f, r = fmaf(-n, scale, x);
  if (fabsf(r) >= half) {
    const bool odd = ((int)n & 1) != 0;
    if (r > half || (r == half && odd)) t += 1.f;
    else if (r < -half || (r == -half && odd)) t -= 1.f;
  }
  return __float_as_uint(t);
}

// The row's scale from its largest magnitude's bits (NaN where the row is not finite).
__device__ __forceinline__ float pool_scale(uint32_t top) {
  const float s = __uint_as_float(top) * (1.f / 127.f);
  return top >= 0x7f800000u ? __int_as_float(0x7fffffff) : s < 1.17549435e-38f ? 0.f : s;
}

// The pool slot of sequence b, or -1: outside the pool, or (KEEP_LAST) one that a
// later sequence writes.  By the whole block.
template <bool KEEP_LAST>
__device__ __forceinline__ int64_t pool_slot(const PoolArgs& a, int b) {
  if (!a.slots) return b;
  const int slot = a.slots[b];
  bool skip = slot < 0 || slot >= a.num_slots;
  if constexpr (KEEP_LAST) {
    for (int64_t i = b + 1 + threadIdx.x; i < a.batch; i += blockDim.x) skip |= a.slots[i] == slot;
    skip = __syncthreads_or(skip);
  }
  return skip ? -1 : slot;
}

// LANES lanes a row, VEC values an access, REGS accesses a lane: LANES * VEC * REGS >=
// width.  A block reads its rows before it looks for its slot, so that the two
// latencies pass together.
template <int LANES, int VEC, int REGS>
__global__ void __launch_bounds__(kPoolThreads) state_store8_kernel(const __grid_constant__ PoolArgs a) {
  const int b = blockIdx.y, lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (kPoolThreads / LANES) + threadIdx.x / LANES;
  const bool in = row < a.rows;
  const float* from = a.state + ((int64_t)b * a.rows + (in ? row : 0)) * a.width;
  const int64_t states = a.batch * a.rows * a.width, kept = a.num_slots * a.rows;  // values, and rows of the pool
  float x[REGS][VEC];
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    const int c = (i * LANES + lane) * VEC;
    if constexpr (VEC == 4) {
      const bool there = in && c < a.width && in_range(from + c - a.state, 4, states);
      const float4 y = there ? __ldcs(reinterpret_cast<const float4*>(from + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
    } else {
      x[i][0] = in && c < a.width && in_range(from + c - a.state, states) ? from[c] : 0.f;
    }
  }
  const int64_t slot = pool_slot<true>(a, b);
  if (slot < 0) return;
  uint32_t top = 0;  // magnitudes as bits: those of infinity and NaN are the largest
#pragma unroll
  for (int i = 0; i < REGS; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
#pragma unroll
  for (int o = LANES / 2; o >= 1; o /= 2) top = max(top, __shfl_xor_sync(kFullMask, top, o));
  const float scale = pool_scale(top), half = 0.5f * scale;
  const bool some = scale > 0.f;
  const float inv = some ? __frcp_rn(scale) : 0.f;
  if (!in) return;
  int8_t* to = a.codes + (slot * a.rows + row) * a.width;
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    const int c = (i * LANES + lane) * VEC;
    if (c >= a.width || !in_range(to + c - a.codes, VEC, kept * a.width)) continue;
    uint32_t n[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] = some ? pool_code(x[i][e], scale, half, inv) : 0;
    if constexpr (VEC == 4)
      *reinterpret_cast<uint32_t*>(to + c) = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
    else
      to[c] = (int8_t)n[0];
  }
  if (lane == 0 && in_range(slot * a.rows + row, kept)) a.scales[slot * a.rows + row] = scale;
}

// LANES lanes a row, 4 codes an access, REGS accesses a lane and ROWS rows at once:
// LANES * 4 * REGS >= width.  A warp's stores are 512 bytes together.
template <int LANES, int REGS, int ROWS>
__global__ void __launch_bounds__(kPoolThreads) state_load8_kernel(const __grid_constant__ PoolArgs a) {
  constexpr int PER = kPoolThreads / LANES;
  const int b = blockIdx.y, lane = threadIdx.x % LANES;
  const int64_t slot = pool_slot<false>(a, b);
  const int64_t row0 = (int64_t)blockIdx.x * (PER * ROWS) + threadIdx.x / LANES;
  const int64_t states = a.batch * a.rows * a.width, kept = a.num_slots * a.rows;  // values, and rows of the pool
  uint32_t w[ROWS][REGS];
  float scale[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = row0 + r * PER;
    const bool in = slot >= 0 && row < a.rows && in_range(slot * a.rows + row, kept);
    scale[r] = in ? a.scales[slot * a.rows + row] : 0.f;
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      const int c = (i * LANES + lane) * 4;
      const int64_t at = (slot * a.rows + row) * a.width + c;
      const bool there = in && c < a.width && in_range(at, 4, kept * a.width);
      w[r][i] = there ? __ldcs(reinterpret_cast<const uint32_t*>(a.codes + at)) : 0;
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = row0 + r * PER;
    if (row >= a.rows) continue;
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      const int c = (i * LANES + lane) * 4;
      if (c >= a.width || !in_range(((int64_t)b * a.rows + row) * a.width + c, 4, states)) continue;
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = (float)(int8_t)(w[r][i] >> (8 * e)) * scale[r];
      __stcs(reinterpret_cast<float4*>(a.state + ((int64_t)b * a.rows + row) * a.width + c), make_float4(f[0], f[1], f[2], f[3]));
    }
  }
}

// Any width and alignment, code by code.
__global__ void __launch_bounds__(kPoolThreads) state_load8_plain_kernel(const __grid_constant__ PoolArgs a) {
  const int b = blockIdx.y;
  const int64_t slot = pool_slot<false>(a, b);
  const uint32_t n = (uint32_t)(a.rows * a.width), i = blockIdx.x * kPoolThreads + threadIdx.x;
  if (i >= n) return;
  float y = 0.f;
  const int64_t code = slot * a.rows * a.width + i, row = slot * a.rows + i / (uint32_t)a.width;
  const int64_t to = (int64_t)b * a.rows * a.width + i;
  if (slot >= 0 && in_range(code, a.num_slots * a.rows * a.width) && in_range(row, a.num_slots * a.rows))
    y = (float)a.codes[code] * a.scales[row];
  if (in_range(to, a.batch * a.rows * a.width)) a.state[to] = y;
}

}  // namespace ssscan

// state_pool.cuh -- states in 8 bits: each row of `width` values as int8 steps of a
// scale of its own.  Bound by memory: 4 bytes in and 1 out a value, or the other way.
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

// x / scale to the nearest integer, ties to even, of the exact quotient.  The fp32
// product lands within one of it; the remainder x - n scale is exact (both terms
// are multiples of the smaller one's last place and it has fewer than 24 bits), so
// comparing it with half a scale corrects the step.
__device__ __forceinline__ int pool_code(float x, float scale, float inv) {
  float n = rintf(x * inv);
  const float r = fmaf(-n, scale, x), half = 0.5f * scale;
  const bool odd = ((int)n & 1) != 0;
  if (r > half || (r == half && odd)) n += 1.f;
  else if (r < -half || (r == -half && odd)) n -= 1.f;
  return (int)n;
}

// The row's scale from its largest magnitude (NaN where the row is not finite).
__device__ __forceinline__ float pool_scale(float top, bool finite) {
  const float s = top * (1.f / 127.f);
  return !finite ? __int_as_float(0x7fffffff) : s < 1.17549435e-38f ? 0.f : s;
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
  float x[REGS][VEC], top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    const int c = (i * LANES + lane) * VEC;
    if constexpr (VEC == 4) {
      const float4 y = in && c < a.width ? __ldcs(reinterpret_cast<const float4*>(from + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
    } else {
      x[i][0] = in && c < a.width ? from[c] : 0.f;
    }
  }
  const int64_t slot = pool_slot<true>(a, b);
  if (slot < 0) return;
#pragma unroll
  for (int i = 0; i < REGS; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float m = fabsf(x[i][e]);
      finite = finite && m <= 3.402823466e38f;
      top = fmaxf(top, m);
    }
#pragma unroll
  for (int o = LANES / 2; o >= 1; o /= 2) {
    top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    finite = __shfl_xor_sync(kFullMask, (int)finite, o) && finite;
  }
  const float scale = pool_scale(top, finite);
  const bool some = scale > 0.f;
  const float inv = some ? __frcp_rn(scale) : 0.f;
  if (!in) return;
  int8_t* to = a.codes + (slot * a.rows + row) * a.width;
#pragma unroll
  for (int i = 0; i < REGS; ++i) {
    const int c = (i * LANES + lane) * VEC;
    if (c >= a.width) continue;
    int n[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) n[e] = some ? pool_code(x[i][e], scale, inv) : 0;
    if constexpr (VEC == 4)
      *reinterpret_cast<char4*>(to + c) = make_char4((signed char)n[0], (signed char)n[1], (signed char)n[2], (signed char)n[3]);
    else
      to[c] = (int8_t)n[0];
  }
  if (lane == 0) a.scales[slot * a.rows + row] = scale;
}

// VEC codes an access (16, 4 or 1; width a multiple of it), four accesses a thread at
// once: the pool's latency comes twice, slot and codes, so more is kept in flight.
template <int VEC>
__global__ void __launch_bounds__(kPoolThreads) state_load8_kernel(const __grid_constant__ PoolArgs a) {
  constexpr int W = VEC == 1 ? 1 : VEC / 4, E = 4;
  const int b = blockIdx.y;
  const int64_t slot = pool_slot<false>(a, b);
  const uint32_t n = (uint32_t)(a.rows * a.width / VEC), per_row = (uint32_t)(a.width / VEC);
  const int8_t* codes = a.codes + slot * a.rows * a.width;
  const float* scales = a.scales + slot * a.rows;
  float* out = a.state + (int64_t)b * a.rows * a.width;
  const uint32_t i0 = blockIdx.x * (kPoolThreads * E) + threadIdx.x;
  uint32_t w[E][W];
  float scale[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t i = i0 + e * kPoolThreads;
#pragma unroll
    for (int j = 0; j < W; ++j) w[e][j] = 0;
    scale[e] = 0.f;
    if (slot >= 0 && i < n) {
      scale[e] = scales[i / per_row];
      if constexpr (VEC == 16) {
        const uint4 y = __ldcs(reinterpret_cast<const uint4*>(codes) + i);
        w[e][0] = y.x, w[e][1] = y.y, w[e][2] = y.z, w[e][3] = y.w;
      } else if constexpr (VEC == 4) {
        w[e][0] = reinterpret_cast<const uint32_t*>(codes)[i];
      } else {
        w[e][0] = (uint8_t)codes[i];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t i = i0 + e * kPoolThreads;
    if (i >= n) continue;
    if constexpr (VEC == 1) {
      out[i] = (float)(int8_t)w[e][0] * scale[e];
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float f[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = (float)(int8_t)(w[e][j] >> (8 * c)) * scale[e];
        __stcs(reinterpret_cast<float4*>(out) + (int64_t)i * W + j, make_float4(f[0], f[1], f[2], f[3]));
      }
    }
  }
}

}  // namespace ssscan

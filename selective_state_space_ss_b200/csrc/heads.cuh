// heads.cuh -- strided [batch, seqlen, heads, d] operands as the kernels have them.
#pragma once

#include <stdint.h>

#include "scan_common.cuh"

namespace ssscan {

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

}  // namespace ssscan

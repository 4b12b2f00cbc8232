// waits.cuh -- bounded waits on a block's barriers, and rings of places that they guard.
#pragma once

#include <stdint.h>

#include "scan_common.cuh"

namespace ssscan {

// Polls before a wait gives up, a second or so.  A poll of a barrier suspends the thread
// for as long as the hardware likes, 3 to 4 us whatever longer time it is given; a poll of
// the previous worker's flag takes about as many tenths.  (512 polls of the first gave up
// after 2 ms, which a worker may well wait for a state where the rows between are short.)
// As a launch's argument the first limit cost 2 to 4%.
constexpr uint32_t kLaSpinLimit = 1u << 18;

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

}  // namespace ssscan

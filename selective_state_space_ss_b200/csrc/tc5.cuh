// tc5.cuh -- the fifth-generation tensor core: shared-memory and instruction
// descriptors, tensor memory, the MMA itself and its completion.
//
// Every operand tile here is kept as blocks of 64 columns: a block's rows are 128
// bytes (64 bf16), in 8-row groups of 1024 bytes, the 16-byte units of a row
// permuted by XOR with the row's number modulo 8 (the 128-byte swizzle).  One such
// block serves two ways: with its columns as the summed index ("K-major") or with
// its rows as the summed index ("MN-major").
#pragma once

#include <stdint.h>

#include "scan_common.cuh"

namespace ssscan {

constexpr uint32_t kTileRow = 128;           // bytes of a block's row (64 bf16)
constexpr uint32_t kTileGroup = 8 * kTileRow;  // the swizzle's 8-row group

// Byte offset of 16-byte unit `unit` (0..7) of row `row` in a block.
__device__ __forceinline__ uint32_t tile_unit(uint32_t row, uint32_t unit) {
  return row * kTileRow + ((unit ^ (row & 7u)) << 4);
}

// Shared-memory descriptor, 128-byte swizzle: the low word has the address and, for
// MN-major operands, the bytes between blocks of 64 columns (both in 16 bytes); the high
// word the bytes between 8-row groups, the version and the swizzle, always the same.
__device__ __forceinline__ uint32_t tile_desc(uint32_t smem_addr, uint32_t lbo) { return (smem_addr >> 4) | (lbo >> 4) << 16; }
constexpr uint32_t kTileDescHigh = (kTileGroup >> 4) | (1u << 14) | (2u << 29);

// Instruction descriptor of a bf16 x bf16 -> fp32 MMA.
__host__ __device__ constexpr uint32_t mma_idesc(int m, int n, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn_major ? 1u << 15 : 0u) |
         (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A[shared] B[shared]; issued by one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"((uint32_t)add), "n"(kTileDescHigh)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[shared]: A's row is the lane, two summed values per 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n mov.b64 y, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"((uint32_t)add), "n"(kTileDescHigh)
      : "memory");
}

// One arrival on `bar` when every MMA that this thread issued before is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}

// Tensor memory, by a whole warp: `cols` a power of two from 32.
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_result, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                   smem_u32(smem_result)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(cols) : "memory");
}

__device__ __forceinline__ void tc5_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc5_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 16 consecutive columns of this warp's 32 lanes; tmem_wait_ld(r) before use.
__device__ __forceinline__ void tmem_ld(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// 16 lanes, 16 columns in two blocks of 8: of block i a thread holds the columns
// 2 (lane % 4) and the next, of row lane / 4 in r[4 i], r[4 i + 1] and of the row 8
// further down in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_rows16(uint32_t (&r)[8], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(addr));
}
// Waits for this warp's loads; the values pass through, so that no use of them moves before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0],"
               " {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// Two floats in a register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return pair(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ float pair_lo(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float pair_hi(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// bf16 of two floats, the first in the low half.
__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
  return h;
}
// Two bf16 as floats.
__device__ __forceinline__ uint64_t from_bf16x2(uint32_t h) { return pair(h << 16, h & 0xffff0000u); }

// Arithmetic on two bf16 at once, each result rounded once.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t neg_bf16x2(uint32_t a) { return a ^ 0x80008000u; }

// Two floats as bf16 planes: plane 0 the nearest bf16, each further plane the
// nearest bf16 of what is left, so that p planes hold 8 p bits of the value.
// Packed as the MMA wants them: the first value in the low half.
template <int PLANES>
__device__ __forceinline__ void split2(uint64_t x, uint32_t (&out)[PLANES]) {
  const uint64_t minus = pair(-1.f, -1.f);
#pragma unroll
  for (int p = 0; p < PLANES; ++p) {
    out[p] = to_bf16x2(pair_lo(x), pair_hi(x));
    if (p + 1 < PLANES) x = fma2(from_bf16x2(out[p]), minus, x);
  }
}

// Four 8 x 8 blocks of bf16 to shared memory: lane i gives the address of row i % 8
// (16 bytes) of block i / 8; a thread holds two neighbours of row lane / 4 of each.
__device__ __forceinline__ void store_blocks(uint32_t row_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(row_addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// Four 8 x 8 blocks from shared memory, each transposed: a thread gets two neighbours
// of column lane / 4 of each.
__device__ __forceinline__ void load_blocks_t(uint32_t row_addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(row_addr)
               : "memory");
}

// The same, each block transposed on its way.
__device__ __forceinline__ void store_blocks_t(uint32_t row_addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};\n" ::"r"(row_addr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

// Registers of a warpgroup: given back to the block, or taken from what others gave.
template <int N>
__device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N)); }

// One 64 x 64 block of a [batch, seqlen, heads, d] tensor by TMA (no multicast).
__device__ __forceinline__ void tma_load_block(uint32_t smem_dst, const void* tmap, uint32_t bar, int32_t d, int32_t t,
                                               int32_t h, int32_t b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];\n" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(d), "r"(t), "r"(h), "r"(b)
      : "memory");
}

}  // namespace ssscan

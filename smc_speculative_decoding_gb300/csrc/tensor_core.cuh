// 5th-generation tensor cores, tensor memory, TMA copies and bounded waits.
#pragma once

#include <cuda.h>

#include "cache_common.cuh"

namespace smcsd {

constexpr uint32_t kWaitPolls = 1u << 17;  // each may suspend up to 20 us

// ---------------------------------------------------------------------------
// Tensor-core and tensor-memory primitives (PTX for sm_103a).
// ---------------------------------------------------------------------------
template <int kColumns>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)),
               "n"(kColumns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int kColumns>
__device__ __forceinline__ void tmem_free(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(kColumns)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
// Shared-memory operand in 128-byte-swizzled rows of 64 elements: `lbo` bytes
// between 64-element panels (of the contiguous axis, MN-major operands only),
// 1024 bytes between groups of eight rows.  Only the low word of a descriptor
// varies.  The products take it as 32 bits and are issued by an elected
// thread: with 64-bit descriptors in an unrolled `lane == 0` branch the
// compiled code used wrong addresses for all but the first step.
constexpr uint32_t kDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;  // version, swizzle
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t lbo) {  // low word
  return (addr & 0x3ffffu) >> 4 | (lbo >> 4) << 16;
}
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem] of 8-bit numbers; `b_high`, the high word of B's descriptor.
__device__ __forceinline__ void mma8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(b_high), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
#define SMC_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                     "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SMC_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                     "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of the calling warp's 32 lanes: thread = lane, register = column.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SMC_R8(r, 0), SMC_R8(r, 8), SMC_R8(r, 16), SMC_R8(r, 24)
      : "r"(addr));
}
// 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : SMC_R8(r, 0), SMC_R8(r, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
          SMC_I8(r, 0),
      SMC_I8(r, 8), SMC_I8(r, 16), SMC_I8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::SMC_I8(r, 0),
      SMC_I8(r, 8), "r"(addr)
      : "memory");
}
// Waits for the warp's loads.  The registers of a load count as written only
// here, so that no use of them moves ahead of the wait.
#define SMC_T8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), \
                     "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : SMC_T8(r, 0), SMC_T8(r, 8), SMC_T8(r, 16), SMC_T8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_wait_all() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_tie16(uint32_t *r) {
  asm volatile("" : SMC_T8(r, 0), SMC_T8(r, 8));
}
__device__ __forceinline__ void tmem_tie(uint32_t *r) {
  asm volatile("" : SMC_T8(r, 0), SMC_T8(r, 8), SMC_T8(r, 16), SMC_T8(r, 24));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The same as pairs, two times 16 columns, there when it returns.
#define SMC_L8(r) "=l"(r[0]), "=l"(r[1]), "=l"(r[2]), "=l"(r[3]), "=l"(r[4]), "=l"(r[5]), "=l"(r[6]), "=l"(r[7])
__device__ __forceinline__ void tmem_get16x2(uint32_t a, uint32_t b, unsigned long long *x, unsigned long long *y) {
  asm volatile(
      "{\n\t.reg .b32 a<16>, b<16>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {b0, b1, b2, b3, b4, b5, b6, b7, b8, b9, b10, b11, b12, b13, b14, b15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {a0, a1};\n\tmov.b64 %1, {a2, a3};\n\tmov.b64 %2, {a4, a5};\n\tmov.b64 %3, {a6, a7};\n\t"
      "mov.b64 %4, {a8, a9};\n\tmov.b64 %5, {a10, a11};\n\tmov.b64 %6, {a12, a13};\n\tmov.b64 %7, {a14, a15};\n\t"
      "mov.b64 %8, {b0, b1};\n\tmov.b64 %9, {b2, b3};\n\tmov.b64 %10, {b4, b5};\n\tmov.b64 %11, {b6, b7};\n\t"
      "mov.b64 %12, {b8, b9};\n\tmov.b64 %13, {b10, b11};\n\tmov.b64 %14, {b12, b13};\n\tmov.b64 %15, {b14, b15};\n\t}"
      : SMC_L8(x), SMC_L8(y)
      : "r"(a), "r"(b)
      : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t addr, const unsigned long long *x) {
  asm volatile(
      "{\n\t.reg .b32 a<16>;\n\t"
      "mov.b64 {a0, a1}, %1;\n\tmov.b64 {a2, a3}, %2;\n\tmov.b64 {a4, a5}, %3;\n\tmov.b64 {a6, a7}, %4;\n\t"
      "mov.b64 {a8, a9}, %5;\n\tmov.b64 {a10, a11}, %6;\n\tmov.b64 {a12, a13}, %7;\n\tmov.b64 {a14, a15}, %8;\n\t"
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {a0, a1, a2, a3, a4, a5, a6, a7, a8, a9, a10, a11, a12, a13, a14, a15};\n\t}" ::"r"(addr),
      "l"(x[0]), "l"(x[1]), "l"(x[2]), "l"(x[3]), "l"(x[4]), "l"(x[5]), "l"(x[6]), "l"(x[7])
      : "memory");
}
// kind::f16 with 128 rows, n columns, fp32 accumulators; b_mn: B is stored
// with its n axis contiguous.
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, int n, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}
// kind::f8f6f4 with 128 rows, n columns, fp32 accumulators; A in e4m3, B in e4m3
// or e5m2; *_mn: the operand is stored with its m or n axis contiguous.
__host__ __device__ constexpr uint32_t instr_desc8(int n, bool a_mn, bool b_mn, bool b_e5m2) {
  return 1u << 4 | (b_e5m2 ? 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int d, int token,
                                            int head, int block, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(d), "r"(token), "r"(head), "r"(block)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int d, int head,
                                            int row, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(d), "r"(head), "r"(row)
      : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}

// Eight words to a 32-byte boundary, one whole sector a thread.
__device__ __forceinline__ void store_32_bytes(void *dst, const uint32_t *x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// Waits.  Every one is bounded, and gives up for the whole CTA: the one that
// ran out raises the status bit and the abort flag, at which the others end.
// What is done when a barrier has already completed is kept to a few
// instructions: each role's code runs once a tile, after other roles' code has
// displaced it from the instruction cache, and is paid for by its length.
// `Tail` is a kernel's shared state, with the flag `abort`.
template <typename Tail>
__device__ __noinline__ bool wait_slowly(Tail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (s->abort) return false;
  }
  s->abort = 1;
  raise_status(status, SMC_DEV_TIMEOUT);
  return false;
}
template <typename Tail>
__device__ __forceinline__ bool guarded_wait(Tail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  return mbar_try_wait(bar, parity) || wait_slowly(s, bar, parity, status);
}
// The same for a whole warp, in step: every lane polls and takes the same
// branch, so that the warp is converged for the .aligned instructions that
// follow.
template <typename Tail>
__device__ __noinline__ bool warp_wait_slowly(Tail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, s->abort)) return false;
  }
  s->abort = 1;
  raise_status(status, SMC_DEV_TIMEOUT);
  return false;
}
template <typename Tail>
__device__ __forceinline__ bool warp_wait(Tail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait_slowly(s, bar, parity, status);
}
// One arrival for a warp (lane 0's), by predicate and not by a branch, for
// the same reason.  What the other lanes did before is ordered by __syncwarp.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(lane)
      : "memory");
}

}  // namespace smcsd

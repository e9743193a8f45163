// Fifth-generation tensor cores: descriptors, tcgen05 instructions and tensor memory for sm_103a.
#pragma once
#include <stdint.h>

#include "mk_device.cuh"

namespace mk {

// ------------------------------------------------------------------------- descriptors
// A shared-memory operand of 16-bit elements in rows of 128 bytes, 128-byte swizzled (eight rows to an
// atom of 1024 bytes, 1024-byte aligned).
//   K-major (rows are M or N): `stride` bytes from eight rows to the next eight, `lead` is not used.
//   MN-major (rows are K): `stride` bytes from eight rows to the next eight, `lead` from 64 elements of M or N
//     to the next 64.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}
// kind::f16 with 32-bit accumulators: a and b 0 fp16 or 1 bf16; b_mn: B is MN-major
__device__ __forceinline__ constexpr uint32_t mma_desc(int type, bool b_mn, int m, int n) {
  return 1u << 4 | (uint32_t)type << 7 | (uint32_t)type << 10 | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(m >> 4) << 24;
}

// --------------------------------------------------------------------------- operations
// D (tensor memory) (+)= A (shared memory) B (shared memory); one thread issues
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
               "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
               : "memory");
}
// the same with A in tensor memory, two 16-bit elements of a row to a column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
               "r"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
               : "memory");
}
// an arrival on the barrier once everything this thread has issued is done
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// this thread's shared memory accesses before what it then starts in the async proxy (products, copies)
__device__ __forceinline__ void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// true in one lane of a converged warp, the same one each time
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// all 512 columns, by one warp; the address goes to *where (shared memory)
__device__ __forceinline__ void tmem_alloc_all(uint32_t* where) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(where)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_all(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base));
}

#define MK_R8(a, i) a(i), a(i + 1), a(i + 2), a(i + 3), a(i + 4), a(i + 5), a(i + 6), a(i + 7)
#define MK_O(i) "=r"(r[i])
#define MK_I(i) "r"(r[i])
// 32, 16 or 8 columns of the warp's 32 lanes (a lane a row), to and from registers; the reads are there after
// tmem_wait_ld
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : MK_R8(MK_O, 0), MK_R8(MK_O, 8), MK_R8(MK_O, 16), MK_R8(MK_O, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : MK_R8(MK_O, 0), MK_R8(MK_O, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::MK_R8(MK_I, 0),
      MK_R8(MK_I, 8), MK_R8(MK_I, 16), MK_R8(MK_I, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::MK_R8(
          MK_I, 0),
      MK_R8(MK_I, 8), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::MK_R8(MK_I, 0), "r"(addr)
               : "memory");
}
#undef MK_I
#undef MK_O
#undef MK_R8
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t addr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(addr) : "memory");
  return r;
}

// global -> shared copy of one box of a 4D tensor map that is a kernel parameter
__device__ __forceinline__ void tma_box_4d(uint32_t dst, const void* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}

}  // namespace mk

// tcgen05.cuh -- wrappers of the fifth-generation tensor core instructions: tensor memory, descriptors, products.
#pragma once

#include "srkv_internal.cuh"

namespace srkv {

// ---- tensor memory: 128 lanes x 512 columns of 32 bits; an address is lane << 16 | column.  Warp w of a
// warpgroup reaches lanes [32 (w % 4), 32 (w % 4) + 32).

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t columns) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define SRKV_R8(f, b) f(b), f(b + 1), f(b + 2), f(b + 3), f(b + 4), f(b + 5), f(b + 6), f(b + 7)
#define SRKV_R32(f) SRKV_R8(f, 0), SRKV_R8(f, 8), SRKV_R8(f, 16), SRKV_R8(f, 24)

// 32 columns of the lane's row; valid after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
#define SRKV_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SRKV_R32(SRKV_OUT)
      : "r"(addr));
#undef SRKV_OUT
}
#define SRKV_R16(f) SRKV_R8(f, 0), SRKV_R8(f, 8)
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
#define SRKV_OUT(i) "=r"(r[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : SRKV_R16(SRKV_OUT)
      : "r"(addr));
#undef SRKV_OUT
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
#define SRKV_IN(i) "r"(r[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
          SRKV_R16(SRKV_IN),
      "r"(addr)
      : "memory");
#undef SRKV_IN
}
__device__ __forceinline__ void tmem_use16(uint32_t* r) {
#define SRKV_IO(i) "+r"(r[i])
  asm volatile("" : SRKV_R16(SRKV_IO));
#undef SRKV_IO
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Keeps uses of loaded registers behind the wait in front of it.
__device__ __forceinline__ void tmem_use32(uint32_t* r) {
#define SRKV_IO(i) "+r"(r[i])
  asm volatile("" : SRKV_R32(SRKV_IO));
#undef SRKV_IO
}

// ---- shared-memory operands: rows of 128 bytes with the 128-byte swizzle, groups of eight rows 1024 bytes apart.

// A descriptor's low word: address, and bytes between one block of 64 columns and the next for an operand whose
// columns are its M or N extent (unused, 0, where they are its K extent).  Steps along the operand add to it.
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t block) {
  return addr >> 4 | (block ? block >> 4 : 1u) << 16;
}
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;  // its high word: eight rows, version, swizzle

// bf16 x bf16 -> fp32, M x N; `b_rows_are_k`: B's rows run along K (its columns along N).
constexpr uint32_t mma_desc(int m, int n, bool b_rows_are_k) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_rows_are_k ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
         (uint32_t)(m >> 4) << 24;
}

// One K step of 16: D (+)= A B with A in shared memory, and with A in tensor memory.  One thread issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHigh)
      : "memory");
}
// The mbarrier gets one arrival once every product that this thread issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// Ordinary writes to shared memory become visible to the tensor cores and copy engine.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace srkv

// The tensor core instructions with accumulators in tensor memory (tcgen05), the barriers in
// shared memory that go with them, and the descriptors of the operand layouts used here.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "serving/wait_clock.h"

namespace rope {
namespace tc {

__device__ __forceinline__ unsigned smem_at(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

// ---------------------------------------------------------------------------
// Barriers in shared memory.  Every wait has a time limit: one that runs out marks the CTA
// as dead, every other wait of the CTA then gives up, and the kernel ends with an error bit.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(bar)) : "memory");
}

__device__ __forceinline__ bool bar_try(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_at(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint32_t now_ns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
  return t;
}

// Waits until the phase of the given parity has completed; false when the CTA is dead.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, unsigned parity, int* dead) {
  if (bar_try(bar, parity)) return true;
  WaitClock clock(now_ns());
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_try(bar, parity)) return true;
    if (*(volatile int*)dead) return false;
    if (clock.expired(now_ns())) {
      *(volatile int*)dead = 1;
      return false;
    }
  }
}

// The barrier gets one arrival when all cp.async copies of this thread so far are there.
__device__ __forceinline__ void bar_arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
}

// Shared memory written by ordinary stores or cp.async copies, this thread's or others' that it
// has waited for, is visible to the products that this thread issues from here on.
__device__ __forceinline__ void fence_to_tensor() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Tensor memory: 512 columns of 128 lanes of 32 bits.  A warp reads and writes the 32 lanes
// (warp % 4) * 32 and up; an address is lane << 16 | column.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* where, int columns) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(where)), "r"(columns)
               : "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_done_allocating() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define ROPE_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define ROPE_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 columns of the thread's lane.
__device__ __forceinline__ void tmem_load32(uint32_t (&v)[32], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : ROPE_R8(v, 0), ROPE_R8(v, 8), ROPE_R8(v, 16), ROPE_R8(v, 24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t (&v)[16], uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : ROPE_R8(v, 0), ROPE_R8(v, 8)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      ROPE_I8(v, 0), ROPE_I8(v, 8)
      : "memory");
}
#undef ROPE_R8
#undef ROPE_I8

// ---------------------------------------------------------------------------
// Products.  16-bit operands of one type, binary32 accumulators; issued by one thread, the one
// that elect() picks of a whole converged warp.  The instruction takes its operands from the
// warp's uniform registers: the values it is given pass through uniform() once, so that no
// product waits for moves of its own.
//
// Operands in shared memory are panels of 64 columns: row r of a panel is 128 bytes at
// r * 128, its 16-byte piece i at place i ^ (r & 7) (the 128-byte swizzle; panels start on
// 1024-byte boundaries).
// ---------------------------------------------------------------------------
template <typename T>
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool b_transposed) {
  const uint32_t type = sizeof(T) == 2 && __is_same(T, __half) ? 0u : 1u;
  return (1u << 4) | (type << 7) | (type << 10) | (b_transposed ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// A value that is the same in all lanes of a converged warp, as the compiler's to know.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Descriptors of operands in shared memory: the upper half says how 8-row groups follow each
// other (1024 bytes) and the swizzle, the lower half holds the address in 16 bytes (an offset
// may be added to it) and, where K runs down the rows (a transposed operand), how 64-column
// panels follow each other.
constexpr uint32_t kLayout = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t operand(uint32_t low) { return (uint64_t)kLayout << 32 | low; }
__device__ __forceinline__ uint32_t k_major(unsigned at) { return ((at & 0x3ffff) >> 4) | 1u << 16; }
__device__ __forceinline__ uint32_t mn_major(unsigned at, unsigned panel) {
  return ((at & 0x3ffff) >> 4) | (panel >> 4) << 16;
}

__device__ __forceinline__ bool elect() {
  uint32_t leader;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(leader)::"memory");
  return leader != 0;
}

// d (+)= a b, a and b in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t inst, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(inst), "r"((uint32_t)add)
      : "memory");
}
// d (+)= a b, a in tensor memory (two 16-bit values a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t inst, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(inst), "r"((uint32_t)add)
      : "memory");
}
// The barrier gets one arrival when the products issued so far by this thread are done.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(bar))
               : "memory");
}

}  // namespace tc
}  // namespace rope

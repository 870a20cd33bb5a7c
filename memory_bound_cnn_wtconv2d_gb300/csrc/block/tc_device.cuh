// Thin wrappers of the sm_103a instructions that the matrix kernels use:
// mbarriers, bulk copies, tcgen05.  Those with an aligned instruction bring the
// warp together first: lanes may have parted before (a lane that leads, one
// that sees its wait end later).
#pragma once

#include <stdint.h>

namespace wtb {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// One lane of a converged warp.  The loops that issue copies and MMAs run on
// whole warps with only the issue itself elected: what they compute is then
// uniform and stays in uniform registers, where these instructions want it (in
// code of a single thread each operand is moved there first, 60 cycles an MMA).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

// Global -> shared, completing on an mbarrier; sizes and addresses are multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// Shared -> global, tracked by the issuing thread's bulk groups.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Orders this thread's generic accesses against bulk copies.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <int THREADS>
__device__ __forceinline__ void named_sync(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

// The same barrier, and whether any of its threads has `p`.
template <int THREADS>
__device__ __forceinline__ bool named_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r) : "r"((uint32_t)p), "r"(id), "n"(THREADS) : "memory");
  return r != 0;
}

__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns) {
  __syncwarp();
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  __syncwarp();
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D[tmem] (+)= A B for one K = 16 step, float16 operands, float32 accumulator.
// Descriptors come as their low words and one high word.
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 x, y;\n"
      "mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3}; setp.ne.b32 p, %5, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p; }" ::"r"(d), "r"(a), "r"(b), "r"(high), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
// The barrier completes when every MMA issued so far has.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// 8 consecutive columns of this warp's 32 lanes; valid after tmem_wait_load().
__device__ __forceinline__ void tmem_load8(uint32_t addr, float (&v)[8]) {
  __syncwarp();
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load() {
  __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Keeps uses of v behind the wait.
__device__ __forceinline__ void tmem_loaded(float (&v)[8]) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}

// Shared-memory descriptor of a 128-byte-swizzled operand tile made of 64 x 64
// sub-blocks of 16-bit values (64 rows of 128 bytes, 8 KB, 1024-aligned).
//   along K:  rows are the operand's M or N index; 8-row groups lie 1024 bytes apart
//   along MN: rows are the K index; 8-row groups 1024 bytes apart, and the
//             next 64 of M or N mn_stride bytes on
// The descriptor's low word: the address and the MN stride; its high word: the
// 8-row stride, the version and the swizzle, the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, bool k_major, uint32_t mn_stride = 8192) {
  // in a cluster the address also holds the CTA's rank, above these bits
  return ((addr & 0x3FFFF) >> 4) | ((k_major ? 1u : mn_stride >> 4) << 16);
}
// What a K = 16 step adds to it: 32 bytes along K, or 16 rows of 128 bytes.
__device__ __forceinline__ uint32_t desc_step(bool k_major) { return k_major ? 32u >> 4 : 2048u >> 4; }
// M = 128, N columns, float16 operands, float32 accumulator.
__device__ __forceinline__ uint32_t instr_desc(int n, bool a_k_major, bool b_k_major) {
  return (1u << 4) | ((a_k_major ? 0u : 1u) << 15) | ((b_k_major ? 0u : 1u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

}  // namespace wtb

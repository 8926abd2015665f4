// Wrappers of the fifth-generation tensor-core instructions (tcgen05) that the
// fp8b prefill uses.  Tensor memory (TMEM) is 128 lanes x 512 columns of 32 bits
// per SM; an address is (lane << 16) | column, and a warp reaches only the 32
// lanes 32 (warp % 4) .. 32 (warp % 4) + 31.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// Allocate ncols columns (a power of two >= 32) for this CTA; the whole warp
// executes it and the base address lands in *dst (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Order tcgen05 operations against thread synchronisation (barriers, mbarriers):
// "before" on the signalling side, "after" on the waiting side.
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrive once on bar when every tcgen05.mma this thread issued so far is complete.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Generic-proxy writes to shared memory before this become visible to the tensor
// core's and the copies' reads after the synchronisation that follows.
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory descriptor of a K-major operand with a swizzle: 8-row atoms sbo
// bytes apart; layout 2 = 128-byte swizzle (rows of 128 bytes), 4 = 64-byte.
__device__ __forceinline__ uint64_t umma_desc(uint32_t saddr, uint32_t sbo, uint32_t layout) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           ((uint64_t)layout << 61);
}
// Instruction descriptor of kind::f8f6f4: fp32 accumulator, K-major operands; type 0 = E4M3, 1 = E5M2.
__host__ __device__ constexpr uint32_t umma_idesc_f8(int M, int N, int a_type, int b_type) {
    return (1u << 4) | ((uint32_t)a_type << 7) | ((uint32_t)b_type << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A B^T, A and B in shared memory / A in tensor memory.
__device__ __forceinline__ void umma_f8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)acc)
                 : "memory");
}
__device__ __forceinline__ void umma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)acc)
                 : "memory");
}

#define KVQ_R8(a, o) "r"(a[o]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])
#define KVQ_W8(a, o) "=r"(a[o]), "=r"(a[o + 1]), "=r"(a[o + 2]), "=r"(a[o + 3]), "=r"(a[o + 4]), "=r"(a[o + 5]), "=r"(a[o + 6]), "=r"(a[o + 7])
// Each lane moves 32 (16) consecutive columns of its own TMEM lane; r[AT] is the first register.
template <int AT, int N> __device__ __forceinline__ void tmem_ld32(uint32_t ta, uint32_t (&r)[N]) {
    static_assert(AT + 32 <= N, "registers");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
                 "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : KVQ_W8(r, AT), KVQ_W8(r, AT + 8), KVQ_W8(r, AT + 16), KVQ_W8(r, AT + 24)
                 : "r"(ta)
                 : "memory");
}
template <int AT, int N> __device__ __forceinline__ void tmem_st32(uint32_t ta, const uint32_t (&r)[N]) {
    static_assert(AT + 32 <= N, "registers");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(ta),
                 KVQ_R8(r, AT), KVQ_R8(r, AT + 8), KVQ_R8(r, AT + 16), KVQ_R8(r, AT + 24)
                 : "memory");
}
template <int AT, int N> __device__ __forceinline__ void tmem_st16(uint32_t ta, const uint32_t (&r)[N]) {
    static_assert(AT + 16 <= N, "registers");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(ta),
                 KVQ_R8(r, AT), KVQ_R8(r, AT + 8)
                 : "memory");
}
#undef KVQ_R8
#undef KVQ_W8

}  // namespace kvq

// tcgen05.cuh -- inline-PTX building blocks for the tcgen05 tensor cores: tensor
// memory (TMEM), its loads and stores, the matrix instruction with its
// descriptors, and tiled TMA loads.
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "ptx.cuh"

namespace skinny {
namespace ptx {

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// PAIR: the instruction works on both CTAs of a cluster of two (cta_group::2).
// One kernel uses one form throughout.

// All 512 columns of the SM's tensor memory; the address lands in *slot
// (shared memory).  One warp allocates, and the same warp frees; with PAIR a
// warp of each CTA does.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc_all(uint32_t* slot)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_free_all(uint32_t base)
{
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base));
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive on `bar` (PAIR: on the barrier at this address in both CTAs) when every
// tcgen05 operation this thread has issued is done.
template <bool PAIR>
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}

// Clusters of two.
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The cluster address of the same variable in the CTA of rank 0.
__device__ __forceinline__ uint32_t leader_addr(const void* p)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
    return a;
}
// An arrival on the leader's barrier.  What it announces lies in tensor memory
// and is ordered by the tcgen05 fences; a release at cluster scope, which would
// order other memory too, takes ~2000 clocks here.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
// Shared-memory operand descriptor: K-major rows of 128 bytes in the 128-byte
// swizzle that a tiled TMA load writes (8-row groups 1024 bytes apart).  The
// high word is constant; the low word holds the address in units of 16 bytes,
// so 32 bytes further along K is + 2.
constexpr uint32_t kSmemDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t smem_desc_low(uint32_t addr) { return (addr & 0x3FFFF) >> 4 | (1u << 16); }

// Instruction descriptor of an m x n matrix instruction, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n)   // f16 x f16 -> f32
{
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_s8(int m, int n)    // s8 x s8 -> s32
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A[tmem, 128 x 16 f16] . B[smem, n x 16 f16]^T; b is the low
// word of B's descriptor.  PAIR: each CTA has 128 of the 256 rows of A and D
// in its own tensor memory, and half the rows of B in its own shared memory.  `add` is a constant wherever it can be.
template <bool PAIR>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add)
{
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "mov.b64 bd, {%2, %5};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], bd, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kSmemDescHigh)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "mov.b64 bd, {%2, %5};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kSmemDescHigh)
            : "memory");
    }
}

// D[tmem] (+)= A[smem, 128 x 32 s8] . B[smem, n x 32 s8]^T
template <bool PAIR>
__device__ __forceinline__ void mma_s8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add)
{
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "mov.b64 ad, {%1, %5};\n\t"
            "mov.b64 bd, {%2, %5};\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], ad, bd, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kSmemDescHigh)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "mov.b64 ad, {%1, %5};\n\t"
            "mov.b64 bd, {%2, %5};\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], ad, bd, %3, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kSmemDescHigh)
            : "memory");
    }
}

__device__ __forceinline__ uint64_t policy_evict_normal()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// Tiled TMA load of one box of a 2-D tensor map; x (elements of the inner
// dimension) times the element size must be a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                            uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// Brings a box into L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y) : "memory");
}

// A load of half a pair's data, which reports to the leader's barrier.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t leader_bar,
                                                 uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(leader_bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// The same of a 3-D map: a box of `pieces` 128-byte wide tiles from tile z on.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void lds64(uint32_t addr, uint32_t (&v)[2])
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// A flag that one CTA publishes for another.
__device__ __forceinline__ void st_release_gpu(unsigned* p, unsigned v)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned ld_acquire_gpu(const unsigned* p)
{
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Loads and stores under a predicate.  The compiler makes a branch of a
// condition around a store, ~40 clocks each where the stores are unrolled.
__device__ __forceinline__ uint32_t ld_global_cg_if(const unsigned* p, bool on)
{
    uint32_t v;
    asm volatile("{\n\t.reg .pred on;\n\tsetp.ne.b32 on, %2, 0;\n\tmov.b32 %0, 0;\n\t"
                 "@on ld.global.cg.u32 %0, [%1];\n\t}"
                 : "=&r"(v)
                 : "l"(p), "r"((int)on)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_global_if(unsigned* p, uint32_t v, bool on)
{
    asm volatile("{\n\t.reg .pred on;\n\tsetp.ne.b32 on, %2, 0;\n\t@on st.global.b32 [%0], %1;\n\t}" ::"l"(p), "r"(v),
                 "r"((int)on)
                 : "memory");
}

__device__ __forceinline__ void st_global_if(float* p, float v, bool on)
{
    st_global_if(reinterpret_cast<unsigned*>(p), __float_as_uint(v), on);
}

__device__ __forceinline__ void st_global_if(__half* p, __half v, bool on)
{
    asm volatile("{\n\t.reg .pred on;\n\tsetp.ne.b32 on, %2, 0;\n\t@on st.global.b16 [%0], %1;\n\t}" ::"l"(p),
                 "h"(__half_as_ushort(v)), "r"((int)on)
                 : "memory");
}

// A warp's 32 lanes of tensor memory, n consecutive 32-bit columns per lane.
// A load waits for its own completion inside the one statement, so no use of
// the registers can be moved before the wait.
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
          "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
          "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

}  // namespace ptx
}  // namespace skinny

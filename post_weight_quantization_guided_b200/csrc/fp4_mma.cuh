// fp4_mma.cuh -- device helpers of the block-scaled 4-bit product: the pair MMA with its
// descriptors, the scales' way to TMEM, and TMEM loads that are waited for together. Inline PTX
// from the public PTX ISA for sm_100a.
#pragma once

#include "common.cuh"

namespace lnq {

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0u;
}

// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0u;
}

// Arrivals on an mbarrier of a CTA of the cluster, given by its shared::cluster address. Neither is
// a plain release at cluster scope, which would also wait for all other writes of this SM (the
// epilogue's stores to global memory): 777 x 11008 -> 4096 with its quantising takes 43 us with that
// and 37 with these, 16384 x 4096 -> 14336 takes 576 and 527.
//   smem_written: releases this CTA's shared memory, as this thread has it, to the cluster.
__device__ __forceinline__ void mbar_arrive_smem_written(uint32_t bar_cluster_addr)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr)
                 : "memory");
}
//   tmem_read: behind this thread's (finished) reads of TMEM; hands over no memory.
__device__ __forceinline__ void mbar_arrive_tmem_read(uint32_t bar_cluster_addr)
{
    asm volatile("tcgen05.fence::before_thread_sync;\n\t"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster_addr)
                 : "memory");
}

// A word of this CTA's shared memory that another CTA of the cluster waits for: the store, and the
// wait until it is not zero (for at most `limit` SM cycles; 0 if it gave up).
__device__ __forceinline__ void st_release_cluster(uint64_t *p, uint64_t v)
{
    asm volatile("st.release.cluster.shared::cta.u64 [%0], %1;" ::"r"(smem_u32(p)), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t wait_nonzero_cluster(uint32_t cluster_address, long long limit)
{
    const long long t0 = clock64();
    uint64_t v;
    do {
        asm volatile("ld.acquire.cluster.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_address) : "memory");
    } while (v == 0u && clock64() - t0 < limit);
    return v;
}

// N (1 or 2) consecutive words of global memory.
template <int N>
__device__ __forceinline__ void ldg_words(uint32_t *v, const uint8_t *src)
{
    if constexpr (N == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src));
        v[0] = u.x, v[1] = u.y;
    } else {
        v[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
    }
}
__device__ __forceinline__ void sts_word(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Four consecutive words of shared memory.
__device__ __forceinline__ void lds_words4(uint32_t *v, uint32_t addr)
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void sts_words4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// Mask of a word's first n bytes (n <= 0: none, n >= 4: all).
__device__ __forceinline__ uint32_t first_bytes(int n)
{
    return n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
}

// Block-scaled product of a pair, kind::mxf4nvf4 (E2M1 operands, two 4-bit elements a byte, K = 64
// per instruction): D (+)= (A sA) x (B sB) with the block scales read from both CTAs' TMEM.
// kBlock16: four scales per row and instruction (blocks of 16), else two (blocks of 32).
template <bool kBlock16>
__device__ __forceinline__ void umma_f4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t sa_tmem, uint32_t sb_tmem,
                                             uint32_t accumulate)
{
    if constexpr (kBlock16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate)
            : "memory");
}

// 32 rows of 16 bytes of each CTA's shared memory (512 consecutive bytes) into four columns of its
// TMEM, row i in lane i of all four lane quarters. Ordered before MMAs issued later by the thread.
__device__ __forceinline__ void tmem_cp_32x128b_pair(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
}

// Shared-memory descriptor of 512 consecutive bytes (8-row groups of 128 bytes, no swizzle), the
// source of tmem_cp_32x128b_pair.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t start)
{
    return static_cast<uint64_t>((start & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46);
}

// Instruction descriptor for kind::mxf4nvf4: E2M1 operands, both K-major; power-of-two (E8M0) or
// E4M3 scales; `sf` the byte of a scale word where the instruction's scales begin.
__host__ __device__ constexpr uint32_t umma_idesc_f4(int M, int N, bool e8m0, uint32_t sf)
{
    return (sf << 4)                                  // B scales' byte
           | (1u << 7) | (1u << 10)                   // A, B: E2M1
           | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
           | ((e8m0 ? 1u : 0u) << 23)                 // scale type
           | (static_cast<uint32_t>(M >> 4) << 24)    // M / 16 (a multiple of 8)
           | (sf << 29);                              // A scales' byte
}

// 32 lanes x 32 columns of 32-bit values: thread t of the warp gets lane (base + t), columns
// [col, col + 32). The registers may be read after tmem_ld_wait and tmem_ld_fence.
__device__ __forceinline__ void tmem_ld_32x32b_x32_nowait(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps the compiler from reading r before the wait that precedes this.
__device__ __forceinline__ void tmem_ld_fence(uint32_t (&r)[32])
{
#pragma unroll
    for (int k = 0; k < 32; ++k)
        asm volatile("" : "+r"(r[k]));
}

}  // namespace lnq

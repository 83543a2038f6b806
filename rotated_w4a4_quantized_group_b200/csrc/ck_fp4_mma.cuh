// ck_fp4_mma.cuh -- tcgen05 operations of the block-scaled fp4 products, for one CTA (CG = 1) or a
// pair (CG = 2), and the mbarrier operations across a cluster that a pair needs.
#pragma once

#include <stdint.h>

#include "ck_device.cuh"
#include "ck_gemm_common.cuh"

namespace ck {

// ------------------------------------------------------------------ mbarriers across a cluster

__device__ __forceinline__ bool mbar_test_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool mbar_try_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// mbar_wait for a barrier on which another CTA of the cluster arrives.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                  int* dev_status) {
    const long long limit = abort ? kRoleWaitLimitCycles : kWaitLimitCycles;
    if (limit <= 0) {
        if (mbar_test_cluster(bar, parity)) return true;
        if (abort) *abort = 1;
        record_timeout(dev_status);
        return false;
    }
    if (mbar_try_cluster(bar, parity)) return true;
    const long long t0 = clock64();
    while (true) {
        if (mbar_try_cluster(bar, parity)) return true;
        if (abort && *abort) return false;
        if (clock64() - t0 > limit) {
            if (abort) *abort = 1;
            record_timeout(dev_status);
            return false;
        }
    }
}

// The cluster address of CTA `rank`'s copy of `local`.
__device__ __forceinline__ uint32_t cluster_address(const void* local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
    return remote;
}

// A word of CTA `rank`'s shared memory at the address of `local` in this CTA.
__device__ __forceinline__ void dsmem_store_u32(void* local, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_address(local, rank)), "r"(v) : "memory");
}

// Orders this thread's writes before the cluster's later reads, past a relaxed barrier too.
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

// Every thread of the cluster's CTAs arrives; orders no writes but those fenced before it.
__device__ __forceinline__ void cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Account for bytes that no copy will bring.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

// Arrive on CTA `rank`'s barrier at the address of `local` in this CTA.
__device__ __forceinline__ void mbar_arrive_remote(uint64_t* local, uint32_t rank) {
    const uint32_t remote = cluster_address(local, rank);
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// ------------------------------------------------------------------ tensor memory

template <int CG> __device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst_smem, uint32_t ncols) {
    if (CG == 1) {
        tmem_alloc(dst_smem, ncols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(dst_smem)),
                     "r"(ncols)
                     : "memory");
    }
}

template <int CG> __device__ __forceinline__ void tmem_relinquish_cg() {
    if (CG == 1) tmem_relinquish();
    else asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

template <int CG> __device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols) {
    if (CG == 1) {
        tmem_dealloc(taddr, ncols);
    } else {
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                     : "memory");
    }
}

// ------------------------------------------------------------------ loads

// A TMA box into this CTA's shared memory that completes on the barrier at cluster address `bar`,
// this CTA's own or (CG = 2) the other's of the pair.
template <int CG>
__device__ __forceinline__ void tma_load_2d_cg(void* dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                               int32_t c1) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_load_3d_cg(void* dst, const CUtensorMap* map, uint32_t bar, int32_t c0,
                                               int32_t c1, int32_t c2) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// 16 lanes x 32 consecutive 32-bit columns as four 16 x 8 fragments: registers 4 i, 4 i + 1 of
// thread t hold lane t / 4, columns 8 i + 2 (t % 4) and the next, 4 i + 2 and 4 i + 3 lane t / 4 + 8.
__device__ __forceinline__ void tc_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// ------------------------------------------------------------------ commits

// Arrive on the barrier (of both CTAs of the pair, at the same address) once every tcgen05
// operation this thread issued so far completes.
template <int CG> __device__ __forceinline__ void tc_commit_cg(uint64_t* bar) {
    if (CG == 1) {
        tc_commit(bar);
    } else {
        const uint16_t both = 3;
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
            " [%0], %1;" ::"r"(smem_u32(bar)),
            "h"(both)
            : "memory");
    }
}

// The same on this CTA's barrier alone.
template <int CG> __device__ __forceinline__ void tc_commit_local(uint64_t* bar) {
    if (CG == 1) {
        tc_commit(bar);
    } else {
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(bar))
                     : "memory");
    }
}

// ------------------------------------------------------------------ scales and MMA

// Shared-memory descriptor of one 512-byte scale tile: 32 rows of 16 bytes without swizzle, 8-row
// groups 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)(128 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    return d;
}

// One scale tile into four tensor-memory columns: word 4 i + j of the tile goes to lane i, column j
// of each of the four lane quarters (of both CTAs, each from its own shared memory, for CG = 2).
template <int CG>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t desc_lo, uint32_t desc_hi) {
#define CK_FP4_CP(group)                                                             \
    asm volatile(                                                                    \
        "{\n\t.reg .b64 s;\n\t"                                                     \
        "mov.b64 s, {%1, %2};\n\t"                                                   \
        "tcgen05.cp.cta_group::" group ".32x128b.warpx4 [%0], s;\n\t}" ::"r"(taddr), \
        "r"(desc_lo), "r"(desc_hi)                                                   \
        : "memory")
    if (CG == 1) CK_FP4_CP("1");
    else CK_FP4_CP("2");
#undef CK_FP4_CP
}

// Instruction descriptor of tcgen05.mma kind::mxf4nvf4: E2M1 A and B, both K-major, M x N (M over
// both CTAs of a pair).  Bits: [4,6) B's scale byte, [7,10) A format (1 = E2M1), [10,12) B format,
// [17,23) N >> 3, [23] scale type (0 = E4M3, 1 = E8M0), [24,29) M >> 4, [29,31) A's scale byte.
__host__ __device__ constexpr uint32_t idesc_fp4(int M, int N, bool nv) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((nv ? 0u : 1u) << 23) |
           ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T over 64 k, each product times A's and B's block scales in
// tensor memory: one scale byte per 16 k (NV, four to a word) or 32 k (MX, two to a word).
// The descriptors of A and B share their high word.
template <bool NV, int CG>
__device__ __forceinline__ void tc_mma_fp4(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t ab_hi,
                                           uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate) {
#define CK_FP4_MMA(group, vec)                                                                     \
    asm volatile(                                                                                  \
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"                                               \
        "setp.ne.b32 p, %7, 0;\n\t"                                                                \
        "mov.b64 a, {%1, %3};\n\t"                                                                 \
        "mov.b64 b, {%2, %3};\n\t"                                                                 \
        "tcgen05.mma.cta_group::" group ".kind::mxf4nvf4.block_scale.scale_vec::" vec              \
        " [%0], a, b, %4, [%5], [%6], p;\n\t}" ::"r"(d_tmem),                                      \
        "r"(a_lo), "r"(b_lo), "r"(ab_hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)          \
        : "memory")
    if (NV) {
        if (CG == 1) CK_FP4_MMA("1", "4X");
        else CK_FP4_MMA("2", "4X");
    } else {
        if (CG == 1) CK_FP4_MMA("1", "2X");
        else CK_FP4_MMA("2", "2X");
    }
#undef CK_FP4_MMA
}

// ------------------------------------------------------------------ outputs

// Two outputs of a 16-bit type in one word, the first in its low half.
template <typename OutT> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return 0u;   // fp32 outputs are not packed
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A bias of any of the three types.
__device__ __forceinline__ float load_any(const void* p, ck_dtype dt, int64_t i) {
    if (dt == CK_F32) return load_scale<float>(p, i);
    if (dt == CK_F16) return load_scale<__half>(p, i);
    return load_scale<__nv_bfloat16>(p, i);
}

}  // namespace ck

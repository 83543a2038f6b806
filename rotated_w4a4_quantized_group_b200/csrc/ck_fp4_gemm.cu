// ck_fp4_gemm.cu -- the product of microscaled fp4 activations and weights:
//   out[m, n] = cvt(fl(acc[m, n] * alpha) + bias[n]),   alpha = x_tensor_scale * w_tensor_scale
//   acc[m, n] = sum over blocks of sx[m, block] * sw[n, block] * (sum over the block of x * w)
// for one weight matrix, or with the rows sorted by expert and a matrix per expert.
//
// Bound: 2 M N K operations on the tensor cores (tcgen05.mma kind::mxf4nvf4, which multiplies the
// block scales in) when there are many rows, the weights' bytes from HBM when there are few.
//
// Persistent; a tile is 128 channels per CTA times BN rows, transposed (D[n, m], channels on the
// tensor-memory lanes), so that a tile of few rows, an expert's, wastes columns of the MMA and not
// its 128 lanes.  CG = 2: two CTAs of a cluster form one 256 x BN tile with
// tcgen05.mma.cta_group::2; each holds its own 128 channels and half of the rows' codes, so a
// byte of shared memory feeds twice the math.  Per stage of 256 k (four MMAs):
//   warps 0, 2, 3  TMA of the weights' codes, of the rows' codes (128-byte rows, 128-byte swizzle)
//            and of both scale tiles; the weights' codes of the first stages before the wait for the
//            kernel before this one (the quantizer)
//   warp 1   copies the scale tiles from shared to tensor memory (tcgen05.cp, in order with the
//            MMAs that read them) and issues the MMAs: the CTA of rank 0 for both CTAs
//   warps 4-11  the epilogue: two warps per lane quarter on alternate 32-row chunks, from one of
//            two accumulators while the MMAs fill the other
// Measured (graph-replayed, the product alone, by box): 8192 x 3840 x 3840 NV 54 to 56 us (4.3 to 4.5
// PFLOP/s; tensor pipe 60% of active cycles, 1.63 GHz at the power cap), 8192 x 10240 x 3840 MX 116 to 120
// us (5.4 to 5.5 PFLOP/s); a stage takes 547 (NV) or 476 (MX) cycles where its MMAs alone need 384.  What
// holds it there is not settled: no change to how a stage is issued shortened it, and both formats, as the
// one-CTA tile of 128 rows, come to 64 to 67 bytes a cycle into an SM's shared memory, a bound that no
// measurement with fewer bytes has tested.
// Every wait is bounded; a CTA leaves only after its own copies have landed, the MMAs that read
// its memory have completed and the arrivals that were sent to it have come.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ck_device.cuh"
#include "ck_fp4.cuh"
#include "ck_fp4_mma.cuh"
#include "ck_gemm_common.cuh"
#include "ck_internal.h"

namespace ck {

namespace fp4g {
constexpr int BW = 128;                 // channels per CTA
constexpr int BK = 256;                 // k per stage: 128 bytes of codes
constexpr int BN_MAX = 192;
constexpr int WARP_TMA_W = 0, WARP_MMA = 1, WARP_TMA_X = 2, WARP_TMA_S = 3, EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int STAGES_MAX = 8;
constexpr uint32_t A_BYTES = BW * BK / 2;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SF_COL = 2 * BN_MAX;   // two accumulators, then two sets of scale columns
constexpr uint32_t SF_SET = 48;
constexpr int EPI_STAGE_BYTES = 32 * 32 * 2;
constexpr size_t SMEM_MAX = 227 * 1024 - 1024;   // less the static shared memory
static_assert(SF_COL + 2 * SF_SET <= TMEM_COLS, "accumulators and scales fit");
}  // namespace fp4g

struct Fp4GemmParams {
    int64_t M, N;
    int num_kb;           // stages per tile: ceil(K / 256)
    int k64;              // MMA steps per tile: ceil(K / 64)
    int BN;               // rows per tile
    int tiles_n;          // tiles along the channels
    int stages;
    uint32_t b_bytes;     // a CTA's codes of the rows per stage
    uint32_t stage_bytes;
    uint32_t idesc;
    int n_experts;        // 1 without offsets
    int n_sf_blocks;      // scale blocks of one weight matrix
    const int32_t* offsets;
    const float* x_ts;
    const float* w_ts;    // one per expert
    const void* bias;     // (n_experts, N)
    ck_dtype bias_dt;
    void* out;
    int64_t ldo;
    int* dev_status;
};

// One tile: expert, first row, rows, first channel of the CTA's 128, and where its rows' scales are.
struct Fp4Tile {
    int e;
    int64_t m0;        // first row
    int rows;          // rows of the expert from m0 on, at most BN
    int64_t n0;        // first channel of the tile
    int sf_block;      // 128-row scale block of m0
    int sf_shift;      // 32-row groups of that block before m0
};

template <int CG>
__device__ __forceinline__ Fp4Tile fp4_tile(const Fp4GemmParams& p, const int* cum, int t) {
    // the last expert whose first tile is not after t
    int lo = 0, hi = p.n_experts - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    Fp4Tile r;
    r.e = lo;
    int64_t first = 0, last = p.M, block = 0;
    if (p.offsets) {
        const RowRange rr = expert_rows(p.offsets, lo, p.M);
        first = rr.lo;
        last = rr.hi;
        block = expert_scale_block(first, lo);
    }
    const int u = t - cum[lo];
    const int i = u / p.tiles_n;
    const int64_t off = (int64_t)i * p.BN;
    r.n0 = (int64_t)(u % p.tiles_n) * (fp4g::BW * CG);
    r.m0 = first + off;
    const int64_t left = last - r.m0;
    r.rows = (int)(left < p.BN ? left : p.BN);
    r.sf_block = (int)(block + off / kFp4TileRows);
    r.sf_shift = (int)(off % kFp4TileRows) / 32;
    return r;
}

// 32 rows (tensor-memory columns from taddr on) x 32 channels (lanes) of 16-bit outputs: loaded as
// 8 x 8 fragments, whose pairs of neighbouring rows pack into one register, and stored transposed
// (stmatrix) into the staging buffer, whose rows then leave in 16-byte pieces.  64-byte staging rows;
// piece c of row m sits at c ^ (m / 2 % 4), so that neither side meets a bank twice.  b: the biases
// of channels lane / 4 + 8 i.
template <typename OutT>
__device__ __forceinline__ void epilogue_vec(uint32_t taddr, float alpha, const float (&b)[4], bool bias,
                                             unsigned char* stage, int lane, OutT* out, int64_t ldo,
                                             int rows) {
    uint32_t r[2][16];
    tc_ld_16x256b_x4(taddr, r[0]);
    tc_ld_16x256b_x4(taddr + (16u << 16), r[1]);
    tc_wait_ld();
    const uint32_t base = smem_u32(stage);
    const int mat = lane >> 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t u[8];   // [4 row groups of 8][channels 16 h.., 16 h + 8..]
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = __fmul_rn(__uint_as_float(r[h][2 * i]), alpha);
            float y = __fmul_rn(__uint_as_float(r[h][2 * i + 1]), alpha);
            if (bias) {
                x = __fadd_rn(x, b[2 * h + (i & 1)]);
                y = __fadd_rn(y, b[2 * h + (i & 1)]);
            }
            u[i] = pack2<OutT>(x, y);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const int m = 8 * (i + (mat >> 1)) + (lane & 7);
            const int c = (2 * h + (mat & 1)) ^ ((m >> 1) & 3);
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             base + (uint32_t)(m * 64 + c * 16)),
                         "r"(u[2 * i]), "r"(u[2 * i + 1]), "r"(u[2 * i + 2]), "r"(u[2 * i + 3])
                         : "memory");
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 8 * i + (lane >> 2), c = lane & 3;
        if (m < rows)
            *reinterpret_cast<uint4*>(out + m * ldo + c * 8) =
                *reinterpret_cast<const uint4*>(stage + m * 64 + ((c ^ ((m >> 1) & 3)) << 4));
    }
    __syncwarp();
}

// The same for fp32 outputs, whose 32 channels of a row are one 128-byte store of the warp as they
// are, and for 16-bit rows that 16-byte stores do not fit: a lane is a channel.
template <typename OutT>
__device__ __forceinline__ void epilogue_any(uint32_t taddr, float alpha, float b, bool bias, bool n_ok,
                                             OutT* out, int64_t ldo, int rows) {
    uint32_t r[32];
    tc_ld_32x32b_x32(taddr, r);
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        float o = __fmul_rn(__uint_as_float(r[j]), alpha);
        if (bias) o = __fadd_rn(o, b);
        if (n_ok && j < rows) OutStore<OutT>::one(out + j * ldo, o);
    }
}

template <typename OutT, bool NV, int CG>
__global__ void __launch_bounds__(fp4g::THREADS, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ CUtensorMap wmap,
                    const __grid_constant__ CUtensorMap xsmap,
                    const __grid_constant__ CUtensorMap wsmap, Fp4GemmParams p) {
    using namespace fp4g;
    constexpr int SF_TILES = NV ? 4 : 2;     // scale tiles per stage and 128 rows
    constexpr int NBLK = CG;                 // 128-row scale blocks a tile's rows touch: pairs take 192
    constexpr uint32_t SFA_BYTES = SF_TILES * kFp4TileBytes, SFB_BYTES = NBLK * SFA_BYTES;
    extern __shared__ __align__(1024) unsigned char fp4_smem[];
    unsigned char* ring = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(fp4_smem) + 1023) & ~uintptr_t(1023));
    const uint32_t S = (uint32_t)p.stages;
    unsigned char* epi_stage = ring + (size_t)S * p.stage_bytes;
    int* cum = reinterpret_cast<int*>(epi_stage + EPI_WARPS * EPI_STAGE_BYTES);   // [n_experts + 1]

    __shared__ __align__(8) uint64_t full[STAGES_MAX], empty[STAGES_MAX];
    __shared__ __align__(8) uint64_t acc_full[2], acc_empty[2], acc_read[2], drain_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag;
    __shared__ uint32_t commits[2];          // rank 0's count of stage and of accumulator commits
    __shared__ uint32_t loaded[2][3];        // stages whose loads each CTA's producers issued

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
    const int unit = (int)blockIdx.x / CG, units = (int)gridDim.x / CG;

    if (tid == 0) {
        for (int s = 0; s < STAGES_MAX; ++s) {
            mbar_init(&full[s], 3);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], EPI_WARPS + CG - 1);   // and the other CTA's word
            mbar_init(&acc_read[s], EPI_WARPS);
        }
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        commits[0] = commits[1] = 0;
        for (int i = 0; i < 6; ++i) loaded[i / 3][i % 3] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&wmap);
        tma_prefetch_desc(&xsmap);
        tma_prefetch_desc(&wsmap);
    }
    if (warp == WARP_MMA) {
        tmem_alloc_cg<CG>(&tmem_base_sh, TMEM_COLS);
        tmem_relinquish_cg<CG>();
    }
    // tiles before each expert's: a running sum over the experts, 32 at a time
    if (warp == EPI_WARP0) {
        int before = 0;
        for (int e0 = 0; e0 < p.n_experts; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.n_experts) {
                int64_t m = p.M;
                if (p.offsets) {
                    const RowRange r = expert_rows(p.offsets, e, p.M);
                    m = r.hi - r.lo;
                }
                n = (int)((m + p.BN - 1) / p.BN) * p.tiles_n;
            }
            int sum = n;   // this expert's and those before it of the 32
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum = tiles_add(sum, o);
            }
            const int others = __shfl_up_sync(0xffffffffu, sum, 1);
            if (e < p.n_experts) cum[e] = lane ? tiles_add(before, others) : before;
            before = tiles_add(before, __shfl_sync(0xffffffffu, sum, 31));
        }
        if (lane == 0) cum[p.n_experts] = before;
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();   // the peer's barriers are ready for arrivals
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    const int tiles = cum[p.n_experts];
    const uint32_t num_kb = (uint32_t)p.num_kb;
    // bytes of a stage that a producer of one CTA loads
    auto part_bytes = [&](int part) { return part == 0 ? A_BYTES : part == 1 ? p.b_bytes : SFA_BYTES + SFB_BYTES; };
    const uint32_t full0 = CG == 2 ? cluster_address(&full[0], 0) : smem_u32(&full[0]);
    const uint32_t my_tiles = tiles_of_unit(tiles, unit, units);

    if (warp == WARP_TMA_W || warp == WARP_TMA_X || warp == WARP_TMA_S) {
        // ---------------------------------------------------------------- loads
        // Three warps issue a stage's boxes at once: the weights' codes, the rows' codes, and both
        // scales (one warp alone is bound by issuing them: about 170 cycles a box).  Both CTAs'
        // copies of a stage complete on rank 0's barrier, which rank 0 arms for both.
        if (elect_one()) {
            const int part = warp == WARP_TMA_W ? 0 : warp == WARP_TMA_X ? 1 : 2;
            const uint32_t bytes = part_bytes(part);
            // the weights' codes of the first stages do not wait for the kernel before this one
            if (part != 0) grid_dependency_wait();
            uint32_t s = 0, phase = 0, issued = 0;
            bool ok = true;
            for (uint32_t lt = 0; ok && lt < my_tiles; ++lt) {
                const Fp4Tile t = fp4_tile<CG>(p, cum, unit + (int)lt * units);
                const int32_t w_row = (int32_t)t.n0 + (int32_t)rank * BW;
                const int32_t w_sf = t.e * p.n_sf_blocks + (int)(t.n0 / BW) + (int)rank;
                const int32_t x_row = (int32_t)t.m0 + (int32_t)rank * (p.BN / CG);
                for (uint32_t kb = 0; kb < num_kb; ++kb) {
                    if (issued >= S) {
                        // this wait covers MMAs that need the rows: it starts after the kernel before
                        if (part == 0 && issued == S) grid_dependency_wait();
                        if (!mbar_wait(&empty[s], phase ^ 1u, &abort_flag, p.dev_status)) {
                            ok = false;
                            break;
                        }
                    }
                    unsigned char* st = ring + (size_t)s * p.stage_bytes;
                    const uint32_t bar = full0 + s * 8;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * bytes);
                    if (part == 0) {
                        tma_load_3d_cg<CG>(st, &wmap, bar, (int32_t)(kb * (BK / 2)), w_row, t.e);
                    } else if (part == 1) {
                        tma_load_2d_cg<CG>(st + A_BYTES, &xmap, bar, (int32_t)(kb * (BK / 2)), x_row);
                    } else {
                        unsigned char* sf = st + A_BYTES + p.b_bytes;
                        tma_load_3d_cg<CG>(sf, &wsmap, bar, 0, (int32_t)(kb * SF_TILES), w_sf);
                        tma_load_3d_cg<CG>(sf + SFA_BYTES, &xsmap, bar, 0, (int32_t)(kb * SF_TILES), t.sf_block);
                    }
                    ++issued;
                    if (++s == S) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            loaded[rank][part] = issued;
            if (rank != 0) {
                dsmem_store_u32(&loaded[1][part], 0, issued);
                fence_cluster();
            }
        }
        __syncwarp();
    } else if (warp == WARP_MMA && rank == 0) {
        // ---------------------------------------------------------------- MMA issuer
        // One elected thread walks the ring; the loop only adds to the low words of its descriptors
        // (8192 x 3840 x 3840 NV: 60 -> 58 us).
        if (elect_one()) {
            grid_dependency_wait();
            const uint32_t slot_step = p.stage_bytes >> 4;   // descriptors count 16-byte units
            const uint64_t ab = smem_desc_k_sw128(smem_u32(ring));
            const uint64_t sf = smem_desc_scales(smem_u32(ring) + A_BYTES + p.b_bytes);
            const uint32_t ab_hi = (uint32_t)(ab >> 32), sf_hi = (uint32_t)(sf >> 32);
            uint32_t ab_lo = (uint32_t)ab, sf_lo = (uint32_t)sf;
            uint32_t s = 0, phase = 0, n_stage = 0, n_acc = 0;
            bool ok = true;
            for (uint32_t lt = 0; ok && lt < my_tiles; ++lt) {
                const uint32_t shift = (uint32_t)fp4_tile<CG>(p, cum, unit + (int)lt * units).sf_shift;
                const uint32_t acc = lt & 1u;
                if (lt >= 2 && !mbar_wait_cluster(&acc_empty[acc], ((lt >> 1) - 1) & 1u, &abort_flag, p.dev_status))
                    break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * BN_MAX;
#pragma unroll 2
                for (uint32_t kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&full[s], phase, &abort_flag, p.dev_status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sfa = tmem_base + SF_COL + (n_stage & 1u) * SF_SET;
                    const uint32_t sfb = sfa + 16;
#pragma unroll
                    for (int j = 0; j < SF_TILES; ++j) {
                        tc_cp_scales<CG>(sfa + 4 * j, sf_lo + j * (kFp4TileBytes >> 4), sf_hi);
#pragma unroll
                        for (int b = 0; b < NBLK; ++b)
                            tc_cp_scales<CG>(sfb + 4 * (NBLK * j + b),
                                             sf_lo + (SFA_BYTES + (b * SF_TILES + j) * kFp4TileBytes) / 16, sf_hi);
                    }
                    // step j: 32 bytes further in the 128-byte rows.  MX: a scale tile holds two
                    // steps, bytes 0-1 and 2-3 of a word
                    auto step = [&](uint32_t j, uint32_t accumulate) {
                        const uint32_t tile = NV ? j : j >> 1, half = NV ? 0u : (j & 1u) * 2u;
                        tc_mma_fp4<NV, CG>(d, ab_lo + j * 2, ab_lo + j * 2 + (A_BYTES >> 4), ab_hi,
                                           p.idesc | (half << 4) | (half << 29), sfa + 4 * tile,
                                           sfb + 4 * NBLK * tile + shift, accumulate);
                    };
                    const uint32_t left = (uint32_t)p.k64 - kb * 4;
                    step(0, kb != 0 ? 1u : 0u);
                    if (left >= 4) {
                        step(1, 1u);
                        step(2, 1u);
                        step(3, 1u);
                    } else {
                        if (left > 1) step(1, 1u);
                        if (left > 2) step(2, 1u);
                    }
                    tc_commit_cg<CG>(&empty[s]);
                    ++n_stage;
                    ab_lo += slot_step;
                    sf_lo += slot_step;
                    if (++s == S) {
                        s = 0;
                        phase ^= 1u;
                        ab_lo = (uint32_t)ab;
                        sf_lo = (uint32_t)sf;
                    }
                }
                if (ok) {
                    tc_commit_cg<CG>(&acc_full[acc]);
                    ++n_acc;
                }
            }
            // every MMA and copy issued above has completed once drain_bar flips
            tc_commit_local<CG>(&drain_bar);
            mbar_wait(&drain_bar, 0, nullptr, p.dev_status);
            commits[0] = n_stage;
            commits[1] = n_acc;
            if (CG == 2) {
                dsmem_store_u32(&commits[0], 1, n_stage);
                dsmem_store_u32(&commits[1], 1, n_acc);
                fence_cluster();
            }
        }
        __syncwarp();
    } else if (CG == 2 && warp == WARP_MMA) {
        // ---------------------------------------------------------------- the other CTA's epilogue
        // tells rank 0 that this CTA has read an accumulator: an arrival that reaches the other SM
        // waits for its thread's earlier stores, so the epilogue's warps leave it to this one.  Only
        // for the accumulators that rank 0 fills again: it waits for those arrivals, while one of the
        // last two tiles' might reach its shared memory after it has left
        grid_dependency_wait();
        for (uint32_t lt = 0; lt + 2 < my_tiles; ++lt) {
            const uint32_t acc = lt & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_read[acc], (lt >> 1) & 1u, &abort_flag, p.dev_status)))
                break;
            if (lane == 0) mbar_arrive_remote(&acc_empty[acc], 0);
        }
        // after a timeout rank 0 waits for none of them: they have come before the closing barrier
        if (lane == 0) fence_cluster();
        __syncwarp();
    } else if (warp >= EPI_WARP0) {
        // ---------------------------------------------------------------- epilogue
        const int q = warp & 3;                        // TMEM lanes 32q .. 32q + 31
        const int eh = (warp - EPI_WARP0) >> 2;        // 32-row chunks eh, eh + 2, ...
        unsigned char* stage = epi_stage + (size_t)(warp - EPI_WARP0) * EPI_STAGE_BYTES;
        grid_dependency_wait();
        const float xts = p.x_ts ? __ldg(p.x_ts) : 1.0f;
        for (uint32_t lt = 0; lt < my_tiles; ++lt) {
            const Fp4Tile t = fp4_tile<CG>(p, cum, unit + (int)lt * units);
            const uint32_t acc = lt & 1u;
            const int64_t n = t.n0 + (int64_t)rank * BW + q * 32;   // the warp's first channel
            const float alpha = __fmul_rn(xts, p.w_ts ? __ldg(p.w_ts + t.e) : 1.0f);
            OutT* ocol = static_cast<OutT*>(p.out) + t.m0 * p.ldo + n;
            const bool vec = sizeof(OutT) == 2 && n + 32 <= p.N && p.ldo % 8 == 0 &&
                             reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
            float bs[4];   // vec: channels lane / 4 + 8 i, otherwise channel lane in bs[0]
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ch = n + (vec ? lane / 4 + 8 * i : lane);
                bs[i] = p.bias && ch < p.N ? load_any(p.bias, p.bias_dt, (int64_t)t.e * p.N + ch) : 0.0f;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[acc], (lt >> 1) & 1u, &abort_flag, p.dev_status)))
                break;
            tc_fence_after();
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN_MAX;
            for (int c0 = 32 * eh; c0 < t.rows; c0 += 64) {
                if (vec) epilogue_vec<OutT>(tacc + (uint32_t)c0, alpha, bs, p.bias != nullptr, stage, lane,
                                            ocol + c0 * p.ldo, p.ldo, t.rows - c0);
                else epilogue_any<OutT>(tacc + (uint32_t)c0, alpha, bs[0], p.bias != nullptr,
                                        n + lane < p.N, ocol + lane + c0 * p.ldo, p.ldo, t.rows - c0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(rank == 0 ? &acc_empty[acc] : &acc_read[acc]);
        }
    }

    tc_fence_before();
    __syncthreads();
    // rank 0's MMAs have completed, and the counts are there (their writers' fences order them; a
    // releasing barrier would wait for every output store to reach the L2)
    if (CG == 2) cluster_sync_relaxed();
    if (warp == 0) {
        const uint32_t n = commits[0], a = commits[1];   // not larger than what was loaded
        bool short_of = false;
        for (int i = 0; i < 3 * CG; ++i) short_of |= loaded[i / 3][i % 3] != n;
        if (short_of && rank == 0 && lane == 0) {
            // after a timeout copies may still be in flight; what a producer did not issue of a stage
            // that another did, the stage's barrier is told not to expect
            uint32_t most = 0;
            for (int i = 0; i < 3 * CG; ++i) most = max(most, loaded[i / 3][i % 3]);
            for (uint32_t j = most > S ? most - S : 0; j < most; ++j) {
                for (int part = 0; part < 3; ++part) {
                    const bool mine = j < loaded[0][part], other = CG == 2 ? j < loaded[1][part] : mine;
                    if (!mine && other) mbar_arrive_expect_tx(&full[j % S], part_bytes(part));
                    else if (!mine) mbar_arrive(&full[j % S]);
                    else if (!other) mbar_complete_tx(&full[j % S], part_bytes(part));
                }
                mbar_wait(&full[j % S], (j / S) & 1u, nullptr, p.dev_status);
            }
        }
        if (CG == 2) {
            // the arrivals of rank 0's commits at this CTA's barriers have come: a lane per barrier
            const uint32_t slot = (uint32_t)lane;
            if (slot < S && slot < n) mbar_wait(&empty[slot], ((n - 1 - slot) / S) & 1u, nullptr, p.dev_status);
            if (slot < 2 && slot < a) mbar_wait(&acc_full[slot], ((a - 1 - slot) >> 1) & 1u, nullptr, p.dev_status);
            __syncwarp();
        }
    }
    __syncthreads();
    if (CG == 2) cluster_sync_relaxed();
    if (warp == WARP_MMA) {
        tc_fence_after();
        tmem_dealloc_cg<CG>(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host

// CTAs per tile and rows per tile, by the estimated cycles of the busiest unit.  A stage takes its
// MMAs and scale copies (BN / 2 cycles per 64 k, 14 per copy) but never less than about 520, what its
// waits and issues take; a tile a little more; the last tile's epilogue about 30 a row, and a pair
// about 2500 more to start and end.  Measured, us: 413 x 2064 x 1111 NV (one wave each): 13.0, 10.3, 8.3
// with {2, 192}, {1, 128}, {1, 64}; 8192 x 3840 x 3840 NV: 55.5, 66.7, 118; 64 rows over 32 experts,
// 3840 x 3840 MX (HBM-bound): 38, 43, 32.  Pairs of 128 rows were never the best by more than 2%.
// Tiles start at multiples of 64 rows, so that a tile's first scale column is even; 32 rows only where
// one tile holds them all.
Fp4Shape fp4_gemm_shape(int64_t M, int64_t N, int64_t K, int n_experts) {
    const int64_t num_kb = (K + fp4g::BK - 1) / fp4g::BK;
    const int sms = num_sms();
    static const Fp4Shape all[] = {{2, 192}, {1, 128}, {1, 64}, {1, 32}};
    const int64_t m = (M + n_experts - 1) / n_experts;   // rows of an expert, were they even
    Fp4Shape best = all[0];
    double best_cost = -1.0;
    for (const Fp4Shape& s : all) {
        if (s.bn == 32 && M > 32) continue;
        const int64_t units = sms / s.cg;
        const int64_t tiles = (int64_t)n_experts * ((m + s.bn - 1) / s.bn) *
                              ((N + 128 * s.cg - 1) / (128 * s.cg));
        const double stage = 2.0 * s.bn + (s.bn > 128 ? 168.0 : 112.0);
        const double tile = (double)num_kb * (stage > 520.0 ? stage : 520.0) + 600.0;
        const double cost = (double)((tiles + units - 1) / units) * tile + 30.0 * s.bn + (s.cg == 2 ? 2500.0 : 0.0);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return best;
}

template <typename OutT, bool NV, int CG>
static ck_status fp4_launch(const CUtensorMap* maps, const Fp4GemmParams& p, size_t smem, int grid,
                            bool dep, cudaStream_t stream) {
    auto kern = fp4_gemm_kernel<OutT, NV, CG>;
    // the most that any call takes, not this call's: another thread may be about to launch a larger one
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fp4g::SMEM_MAX) != cudaSuccess)
        return cuda_error();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (CG == 2) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (dep) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(fp4g::THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)n;
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], p) == cudaSuccess ? CK_OK : cuda_error();
}

template <typename OutT>
static ck_status fp4_launch_out(const CUtensorMap* maps, const Fp4GemmParams& p, size_t smem, int grid,
                                bool nv, int cg, bool dep, cudaStream_t stream) {
    if (nv)
        return cg == 2 ? fp4_launch<OutT, true, 2>(maps, p, smem, grid, dep, stream)
                       : fp4_launch<OutT, true, 1>(maps, p, smem, grid, dep, stream);
    return cg == 2 ? fp4_launch<OutT, false, 2>(maps, p, smem, grid, dep, stream)
                   : fp4_launch<OutT, false, 1>(maps, p, smem, grid, dep, stream);
}

ck_status launch_fp4_gemm(const Fp4Product& a, cudaStream_t stream) {
    using namespace fp4g;
    const int E = a.offsets ? a.n_experts : 1;
    const int64_t num_kb = (a.K + BK - 1) / BK;
    const int64_t k_tiles = fp4_k_tiles(a.K, a.nv);
    const Fp4Shape shape = fp4_gemm_shape(a.M, a.N, a.K, E);
    Fp4GemmParams p;
    p.M = a.M;
    p.N = a.N;
    p.num_kb = (int)num_kb;
    p.k64 = (int)((a.K + 63) / 64);
    p.BN = shape.bn;
    p.tiles_n = (int)((a.N + BW * shape.cg - 1) / (BW * shape.cg));
    // the tile count stays an int: rows split over experts give at most one more tile each (and one
    // expert's alone, for offsets that decrease: see tiles_add)
    if ((double)p.tiles_n * ((double)a.M / p.BN + E + 1) >= 2147483647.0) return CK_ERR_UNSUPPORTED;
    p.b_bytes = (uint32_t)(shape.bn / shape.cg) * (BK / 2);
    const uint32_t sf_bytes = (a.nv ? 4 : 2) * kFp4TileBytes * (1 + shape.cg);
    p.stage_bytes = (A_BYTES + p.b_bytes + sf_bytes + 1023) & ~1023u;
    const size_t fixed = 1024 + EPI_WARPS * EPI_STAGE_BYTES + (size_t)(E + 1) * sizeof(int);
    p.stages = (int)((SMEM_MAX - fixed) / p.stage_bytes);
    if (p.stages > STAGES_MAX) p.stages = STAGES_MAX;
    const size_t smem = fixed + (size_t)p.stages * p.stage_bytes;
    p.idesc = idesc_fp4(BW * shape.cg, shape.bn, a.nv);
    p.n_experts = E;
    p.n_sf_blocks = (int)((a.N + kFp4TileRows - 1) / kFp4TileRows);
    p.offsets = a.offsets;
    p.x_ts = a.x_ts;
    p.w_ts = a.w_ts;
    p.bias = a.bias;
    p.bias_dt = a.bias_dt;
    p.out = a.out;
    p.ldo = a.ldo;
    p.dev_status = a.dev_status;

    CUtensorMap maps[4];   // rows, weights, rows' scales, weights' scales
    const uint64_t half = (uint64_t)(a.K / 2);
    const uint64_t sf_blocks = (uint64_t)(a.offsets ? a.M / kFp4TileRows + E
                                                    : (a.M + kFp4TileRows - 1) / kFp4TileRows);
    const uint64_t tile_words = kFp4TileBytes / 4;
    const uint32_t sf_tiles = a.nv ? 4 : 2;
    {
        const uint64_t dims[2] = {half, (uint64_t)a.M}, strides[1] = {(uint64_t)a.ldq};
        const uint32_t box[2] = {BK / 2, (uint32_t)(shape.bn / shape.cg)};
        const ck_status st = encode_tma(&maps[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, dims, strides,
                                        box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != CK_OK) return st;
    }
    {
        const uint64_t dims[3] = {half, (uint64_t)a.N, (uint64_t)E};
        const uint64_t strides[2] = {(uint64_t)a.w_ld, (uint64_t)(E > 1 ? a.w_stride : a.w_ld * a.N)};
        const uint32_t box[3] = {BK / 2, BW, 1};
        const ck_status st = encode_tma(&maps[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.w, dims, strides, box,
                                        CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != CK_OK) return st;
    }
    {
        const uint64_t dims[3] = {tile_words, (uint64_t)k_tiles, sf_blocks};
        const uint64_t strides[2] = {kFp4TileBytes, (uint64_t)k_tiles * kFp4TileBytes};
        const uint32_t box[3] = {(uint32_t)tile_words, sf_tiles, (uint32_t)shape.cg};
        const ck_status st = encode_tma(&maps[2], CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, a.scales, dims, strides,
                                        box, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (st != CK_OK) return st;
    }
    {
        const uint64_t dims[3] = {tile_words, (uint64_t)k_tiles, (uint64_t)p.n_sf_blocks * (uint64_t)E};
        const uint64_t strides[2] = {kFp4TileBytes, (uint64_t)k_tiles * kFp4TileBytes};
        const uint32_t box[3] = {(uint32_t)tile_words, sf_tiles, 1};
        const ck_status st = encode_tma(&maps[3], CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, a.w_scales, dims,
                                        strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (st != CK_OK) return st;
    }
    // tiles of one matrix are known here; the experts' only on the device
    int64_t units = num_sms() / shape.cg;
    if (!a.offsets) {
        const int64_t tiles = (int64_t)p.tiles_n * ((a.M + p.BN - 1) / p.BN);
        if (tiles < units) units = tiles;
    }
    const int grid = (int)units * shape.cg;
    switch (a.out_dt) {
        case CK_F32: return fp4_launch_out<float>(maps, p, smem, grid, a.nv, shape.cg, a.dependent, stream);
        case CK_F16: return fp4_launch_out<__half>(maps, p, smem, grid, a.nv, shape.cg, a.dependent, stream);
        case CK_BF16:
            return fp4_launch_out<__nv_bfloat16>(maps, p, smem, grid, a.nv, shape.cg, a.dependent, stream);
        default: return CK_ERR_INVALID_ARG;
    }
}

}  // namespace ck

// ck_fp4_few.cu -- the fp4 linear for few rows or few tiles: a read of the weights, and for the smallest
// calls a chain of latencies.
//
//   out[m, n] = cvt(fl(acc[m, n] * alpha) + bias[n]),   alpha = x_tensor_scale * w_tensor_scale
//
// Tiles of 128 channels x up to 64 rows alone would be a CTA on a few SMs, so each tile's K is split over
// a cluster of S CTAs (about one per SM in all), each of which
//   - asks for its share of the weights, as many steps of 256 k at once as shared memory holds (one
//     box of codes and one of scale tiles a step, on the step's mbarrier), for the others as MMAs
//     free their slots,
//   - meanwhile, FUSED, quantizes the rows' share of K straight into the shared-memory layouts that
//     the MMA and the scale copies read (one launch, no workspace; every tile repeats the
//     quantizing, so this is for few values: see fp4_few_fuses), or else loads codes and scales that
//     the quantizer before it wrote,
//   - multiplies on the tensor cores, 128 channels x BN rows, as the weights arrive,
//   - writes its partial sums to shared memory; after a cluster barrier each CTA adds its share of
//     the tile over the S partials in rank order (no atomics) and stores it.
// Measured, 3840 x 3840: one bf16 row to NV 6.9 us replayed back to back (10.2 with the quantizer and
// the persistent kernel), 32 rows to MX with the quantizer before it 7.6 (10.1); the weights alone are
// 1.3 us of HBM.
// Every CTA takes both cluster barriers whatever happened before them; every mbarrier wait is bounded.
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

namespace fp4f {
constexpr int BW = 128;                  // channels per tile
constexpr int BK = 256;                  // k per step of the ring: 128 bytes of codes
constexpr int THREADS = 256;
constexpr int SLOTS_MAX = 8;             // steps of weights in flight
constexpr int MAX_CLUSTER = 8;
constexpr uint32_t A_BYTES = BW * BK / 2;
constexpr uint32_t TMEM_COLS = 128;
constexpr uint32_t SF_COL = 64;          // accumulator [0, 64), then two sets of 16 + 16 scale columns
constexpr size_t SMEM_BUDGET = 220 * 1024;
}  // namespace fp4f

struct Fp4FewParams {
    int M, BN;               // rows, and rows of a tile: the MMA's N
    int64_t N, K;
    int num_kb, kb_per;      // steps of K, and of one CTA
    int slots;               // steps of weights (FUSED), or of both operands, held at a time
    uint32_t b_bytes;        // BN * 128
    uint32_t idesc;
    const void* x;           // FUSED: the activations
    int64_t sm, sk;
    bool x_vec;              // 16-byte loads
    const float* x_ts;
    const float* w_ts;
    const void* bias;
    ck_dtype bias_dt;
    void* out;
    ck_dtype out_dt;
    int64_t ldo;
    bool out_vec;            // four outputs in one aligned store
    int* dev_status;
};

// T: the activations' type (FUSED), otherwise ignored.  RING: a CTA has more steps than slots (the short
// form saves the smallest calls half a microsecond of 6.5).
template <typename T, bool NV, bool HAS_T, bool FUSED, bool RING>
__global__ void __launch_bounds__(fp4f::THREADS)
    fp4_few_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                   const __grid_constant__ CUtensorMap xsmap, const __grid_constant__ CUtensorMap wsmap,
                   Fp4FewParams p) {
    using namespace fp4f;
    constexpr int SF_TILES = NV ? 4 : 2;
    constexpr uint32_t SF_BYTES = SF_TILES * kFp4TileBytes;   // scale tiles of 128 rows x 256 k
    extern __shared__ __align__(1024) unsigned char few_smem[];
    unsigned char* abuf = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(few_smem) + 1023) & ~uintptr_t(1023));
    const int R = RING ? p.slots : p.kb_per, b_steps = FUSED ? p.kb_per : R;   // the rows' steps held
    unsigned char* bbuf = abuf + (size_t)R * A_BYTES;
    unsigned char* sfa_buf = bbuf + (size_t)b_steps * p.b_bytes;
    unsigned char* sfb_buf = sfa_buf + (size_t)R * SF_BYTES;
    float* partial = reinterpret_cast<float*>(sfb_buf + (size_t)b_steps * SF_BYTES);   // [BN][128]

    __shared__ __align__(8) uint64_t full[SLOTS_MAX], empty[SLOTS_MAX], acc_full, drain_bar;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_flag, loaded;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank(), ncta = cluster_nctarank();
    const int kb_lo = (int)rank * p.kb_per;
    const int n_kb = min(p.num_kb - kb_lo, p.kb_per);
    const int n0 = (int)blockIdx.y * BW;
    const int m0 = FUSED ? 0 : (int)blockIdx.z * p.BN;      // the tile's first row, and its rows
    const int rows = min(p.M - m0, p.BN);

    auto load_w = [&](int i, int slot) {
        mbar_arrive_expect_tx(&full[slot], A_BYTES + SF_BYTES);
        tma_load_2d(abuf + (size_t)slot * A_BYTES, &wmap, &full[slot], (kb_lo + i) * (BK / 2), n0);
        tma_load_3d(sfa_buf + (size_t)slot * SF_BYTES, &wsmap, &full[slot], 0, (kb_lo + i) * SF_TILES,
                    (int)blockIdx.y);
    };
    auto load_x = [&](int i, int slot) {
        mbar_arrive_expect_tx(&full[slot], p.b_bytes + SF_BYTES);
        tma_load_2d(bbuf + (size_t)slot * p.b_bytes, &xmap, &full[slot], (kb_lo + i) * (BK / 2), m0);
        tma_load_3d(sfb_buf + (size_t)slot * SF_BYTES, &xsmap, &full[slot], 0, (kb_lo + i) * SF_TILES,
                    m0 / kFp4TileRows);
    };
    const int head = RING ? min(n_kb, R) : n_kb;   // steps asked for at once
    if (tid == 0) {
        for (int i = 0; i < SLOTS_MAX; ++i) {
            mbar_init(&full[i], FUSED ? 1 : 2);
            if (RING) mbar_init(&empty[i], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        loaded = head;
        fence_mbar_init();
        // the weights first: nothing else is as far away
        for (int i = 0; i < head; ++i) load_w(i, i);
        if (!FUSED) {
            grid_dependency_wait();
            for (int i = 0; i < head; ++i) load_x(i, i);
        }
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, TMEM_COLS);
        tmem_relinquish();
    }
    if (FUSED) {
        // scale bytes past K are zero: what they multiply is, too, and must not meet a NaN
        for (uint32_t i = tid; i < b_steps * SF_BYTES / 16; i += THREADS)
            reinterpret_cast<uint4*>(sfb_buf)[i] = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;

    if (FUSED) {
        // ---------------------------------------------------------------- quantize the rows' share of K
        const int64_t k0 = (int64_t)kb_lo * BK;
        const int64_t left = p.K - k0;
        const int groups = (int)min(left, (int64_t)n_kb * BK) / 16;   // of sixteen k; even for MX
        const int total = rows * groups;
        Fp4Tensor t = fp4_tensor(HAS_T ? p.x_ts : nullptr);
        if (HAS_T && GridBits<T>::value > 0) {
            const uint2 m = fp4_moves<T>(t.t);
            t.moves = m.x;
            t.ups = m.y;
        }
        const T* x = static_cast<const T*>(p.x);
        for (int base = 0; base < total; base += THREADS) {
            const int i = base + tid;
            const bool ok = i < total;
            const int r = ok ? i / groups : 0, g = ok ? i % groups : 0;
            const T* src = x + r * p.sm + (k0 + g * 16) * p.sk;
            float v[16];
            if (p.x_vec) {
                uint4 u[sizeof(T)];
#pragma unroll
                for (int j = 0; j < (int)sizeof(T); ++j)
                    u[j] = ok ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0, 0, 0, 0);
                const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = Elem<T>::to_f(e[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = ok ? Elem<T>::to_f(src[j * p.sk]) : 0.0f;
            }
            uint32_t amax = absmax16(v);
            if (!NV) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const Fp4Scale b = fp4_scale<T, NV, HAS_T>(amax, t);
            uint32_t c[2];
            fp4_codes<T, NV, HAS_T>(v, b, c);
            if (ok) {
                // 128-byte rows, 16-byte piece j of row r at j ^ (r % 8)
                const int kb = g >> 4, gk = g & 15;
                *reinterpret_cast<uint2*>(bbuf + (size_t)kb * p.b_bytes + r * 128 +
                                          (((gk >> 1) ^ (r & 7)) << 4) + (gk & 1) * 8) =
                    make_uint2(c[0], c[1]);
                const int blk = NV ? gk : gk >> 1;
                if (NV || !(gk & 1))
                    sfb_buf[(size_t)kb * SF_BYTES + (blk >> 2) * kFp4TileBytes + fp4_tile_byte(r, blk & 3)] =
                        (uint8_t)b.byte;
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
    }

    if (RING && warp == 0) {
        // ---------------------------------------------------------------- the steps that did not fit
        if (elect_one()) {
            if (!FUSED) grid_dependency_wait();   // its waits need the kernel before this one
            int i = R;
            for (; i < n_kb; ++i) {
                const int slot = i % R;
                if (!mbar_wait(&empty[slot], (uint32_t)(i / R - 1) & 1u, &abort_flag, p.dev_status)) break;
                load_w(i, slot);
                if (!FUSED) load_x(i, slot);
            }
            loaded = i;
        }
        __syncwarp();
    }
    if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        if (elect_one()) {
            if (!FUSED) grid_dependency_wait();   // its waits need the kernel before this one
            const uint64_t ad = smem_desc_k_sw128(smem_u32(abuf)), bd = smem_desc_k_sw128(smem_u32(bbuf));
            const uint64_t fa = smem_desc_scales(smem_u32(sfa_buf)), fb = smem_desc_scales(smem_u32(sfb_buf));
            const uint32_t ab_hi = (uint32_t)(ad >> 32), sf_hi = (uint32_t)(fa >> 32);
            bool ok = true;
            const uint32_t shift = (uint32_t)(m0 % kFp4TileRows) / 32;   // the rows' first scale column
            int slot = 0;
            uint32_t phase = 0;
            for (int i = 0; i < n_kb; ++i) {
                if (!mbar_wait(&full[slot], phase, &abort_flag, p.dev_status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int b = FUSED ? i : slot;
                const uint32_t a_lo = (uint32_t)ad + slot * (A_BYTES >> 4), b_lo = (uint32_t)bd + b * (p.b_bytes >> 4);
                const uint32_t sfa = tmem_base + SF_COL + (i & 1) * 32, sfb = sfa + 16;
#pragma unroll
                for (int j = 0; j < SF_TILES; ++j) {
                    tc_cp_scales<1>(sfa + 4 * j, (uint32_t)fa + ((slot * SF_BYTES + j * kFp4TileBytes) >> 4), sf_hi);
                    tc_cp_scales<1>(sfb + 4 * j, (uint32_t)fb + ((b * SF_BYTES + j * kFp4TileBytes) >> 4), sf_hi);
                }
                const int steps = min(4, (int)((p.K - (int64_t)(kb_lo + i) * BK + 63) / 64));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < steps) {
                        const uint32_t tile = NV ? j : j >> 1, half = NV ? 0u : (j & 1u) * 2u;
                        tc_mma_fp4<NV, 1>(tmem_base, a_lo + j * 2, b_lo + j * 2, ab_hi,
                                          p.idesc | (half << 4) | (half << 29), sfa + 4 * tile,
                                          sfb + 4 * tile + shift, (i | j) != 0 ? 1u : 0u);
                    }
                }
                if (RING) tc_commit(&empty[slot]);
                if (++slot == R) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            if (ok) tc_commit(&acc_full);
            // every MMA and copy issued above has completed once drain_bar flips
            tc_commit(&drain_bar);
            mbar_wait(&drain_bar, 0, nullptr, p.dev_status);
        }
        __syncwarp();
    }
    if (warp >= 4) {
        // the partial sums, transposed into shared memory as [row][channel]
        const int q = warp & 3;
        if (!FUSED) grid_dependency_wait();
        if (__all_sync(0xffffffffu, mbar_wait(&acc_full, 0, &abort_flag, p.dev_status))) {
            tc_fence_after();
            const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16);
            for (int c = 0; c < rows; c += 16) {
                uint32_t a[16];
                tc_ld_32x32b_x16(tacc + (uint32_t)c, a);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < rows) partial[(c + j) * BW + q * 32 + lane] = __uint_as_float(a[j]);
            }
        }
        tc_fence_before();
    }

    // ---------------------------------------------------------------- sum over the cluster
    __syncthreads();
    if (warp == 1) {
        // before the cluster's barrier: a CTA that held tensor memory there could wait for a peer that
        // waits for tensor memory of its own, which such a CTA of another cluster holds
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
    cluster_sync_all();
    if (!FUSED) grid_dependency_wait();   // also what this kernel writes waits for the one before
    if (!abort_flag) {
        const float alpha = __fmul_rn(p.x_ts ? __ldg(p.x_ts) : 1.0f, p.w_ts ? __ldg(p.w_ts) : 1.0f);
        const int nvec = rows * (BW / 4);
        const int lo = (int)((int64_t)nvec * rank / ncta), hi = (int)((int64_t)nvec * (rank + 1) / ncta);
        for (int vi = lo + tid; vi < hi; vi += THREADS) {
            const int m = vi / (BW / 4), c4 = (vi % (BW / 4)) * 4;
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint4 u[MAX_CLUSTER];
#pragma unroll
            for (uint32_t q = 0; q < MAX_CLUSTER; ++q)
                if (q < ncta) u[q] = dsmem_load_v4(partial + m * BW + c4, q);
#pragma unroll
            for (uint32_t q = 0; q < MAX_CLUSTER; ++q)
                if (q < ncta) {
                    s[0] = __fadd_rn(s[0], __uint_as_float(u[q].x));
                    s[1] = __fadd_rn(s[1], __uint_as_float(u[q].y));
                    s[2] = __fadd_rn(s[2], __uint_as_float(u[q].z));
                    s[3] = __fadd_rn(s[3], __uint_as_float(u[q].w));
                }
            const int64_t n = (int64_t)n0 + c4, at = (int64_t)(m0 + m) * p.ldo + n;
            const int have = (int)min(p.N - n, (int64_t)4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[e] = __fmul_rn(s[e], alpha);
                if (p.bias && e < have) s[e] = __fadd_rn(s[e], load_any(p.bias, p.bias_dt, n + e));
            }
            if (p.out_vec && have == 4) {   // four channels in one store
                if (p.out_dt == CK_F32) {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(s[0], s[1], s[2], s[3]);
                } else {
                    const uint2 u = p.out_dt == CK_F16 ? make_uint2(pack2<__half>(s[0], s[1]), pack2<__half>(s[2], s[3]))
                                                       : make_uint2(pack2<__nv_bfloat16>(s[0], s[1]),
                                                                    pack2<__nv_bfloat16>(s[2], s[3]));
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = u;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= have) break;
                    if (p.out_dt == CK_F32) static_cast<float*>(p.out)[at + e] = s[e];
                    else if (p.out_dt == CK_F16) static_cast<__half*>(p.out)[at + e] = __float2half_rn(s[e]);
                    else static_cast<__nv_bfloat16*>(p.out)[at + e] = __float2bfloat16_rn(s[e]);
                }
            }
        }
    }
    // no CTA leaves while a peer may still read its partial sums, nor with a copy still landing
    cluster_sync_all();
    if (tid == 0 && abort_flag)
        for (int i = max(loaded - R, 0); i < loaded; ++i)
            mbar_wait(&full[i % R], (uint32_t)(i / R) & 1u, nullptr, nullptr);
}

// Shared memory of a CTA: `slots` steps of weights, `b_steps` steps of BN rows, the partial sums.
static size_t few_smem_bytes(int slots, int b_steps, int bn, bool nv) {
    using namespace fp4f;
    const size_t sf = (nv ? 4 : 2) * kFp4TileBytes;
    return 1024 + slots * (A_BYTES + sf) + b_steps * ((size_t)bn * (BK / 2) + sf) + (size_t)bn * BW * 4;
}

static int few_bn(int64_t M) { return M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : 64; }

// How a call is split: S CTAs a tile, kb_per steps a CTA, `slots` of them in flight, shared memory.
struct FewPlan {
    int S, kb_per, slots;
    size_t smem;
};

// The largest split whose clusters all run at once: a second round costs more than any split gains (16
// tiles of 10240 k in clusters of eight took 13 us, 12 tiles 7.8).  The room is what a B200 holds of
// clusters of S (they do not cross GPCs) with one CTA an SM and with two, where shared memory fits twice.
static FewPlan few_plan(int64_t tiles, int64_t num_kb, int bn, bool nv, bool fused) {
    using namespace fp4f;
    static const struct {
        int S, room[2];
    } splits[] = {{8, {15, 33}}, {6, {22, 45}}, {5, {26, 56}}, {4, {33, 71}}, {3, {45, 93}}, {2, {74, 148}}, {1, {148, 296}}};
    FewPlan r = {};
    for (const auto& c : splits) {
        FewPlan p;
        p.kb_per = (int)((num_kb + c.S - 1) / c.S);
        p.S = (int)((num_kb + p.kb_per - 1) / p.kb_per);   // every rank has a step
        // fused, half of shared memory stays for weights: otherwise the larger split, in several rounds
        if (fused && r.S && few_smem_bytes(0, p.kb_per, bn, nv) > SMEM_BUDGET / 2) break;
        p.slots = p.kb_per < SLOTS_MAX ? p.kb_per : SLOTS_MAX;
        while (p.slots > 1 && few_smem_bytes(p.slots, fused ? p.kb_per : p.slots, bn, nv) > SMEM_BUDGET) --p.slots;
        p.smem = few_smem_bytes(p.slots, fused ? p.kb_per : p.slots, bn, nv);
        r = p;
        // (large clusters of more than 16 rows lose that way: 64 rows of 3840x3840 in sixes 9.2 us, in fours 8.85)
        const bool twice = 2 * (p.smem + 2048) <= 228 * 1024 && (c.S <= 4 || bn <= 16);
        if (tiles <= c.room[twice]) break;
    }
    return r;
}

static int64_t few_tiles(int64_t M, int64_t N) {
    const int bn = few_bn(M);
    return ((N + fp4f::BW - 1) / fp4f::BW) * ((M + bn - 1) / bn);
}

// From codes: whether the split takes less than the persistent kernel.  Both measured on 17 to 600 rows,
// 64 to 3840 channels and 256 to 10240 k, us: the split 4.3, 0.02 a row of the tile, 0.5 a further step
// and 1.1 where CTAs share SMs; the persistent kernel, while its tiles are one round, 3.9, 0.26 a step,
// and 1.1 where 16-bit rows do not take 16-byte stores (`ragged`).  100 x 907 x 10240: 8.8 against 15.1.
bool fp4_few_takes(int64_t M, int64_t N, int64_t K, bool nv, bool ragged) {
    const int64_t tiles = few_tiles(M, N), num_kb = (K + fp4f::BK - 1) / fp4f::BK;
    if (M < 1 || 2 * tiles > num_sms()) return false;
    const int bn = few_bn(M);
    const FewPlan r = few_plan(tiles, num_kb, bn, nv, false);
    const double shared = tiles * r.S > num_sms() ? 1.1 : 0.0;
    return 4.3 + 0.02 * bn + 0.5 * (r.kb_per - 1) + shared < 3.9 + 0.26 * (double)num_kb + (ragged ? 1.1 : 0.0);
}

// Rows x steps of 256 k up to which the tiles quantize for themselves.  Measured (3840 channels, replayed,
// bf16): K = 3840, 8 rows: MX 6.5 us and NV 7.3 against 7.3 and 7.9 with the quantizer in a launch of its
// own; 16 rows: 8.1 and 9.7 against 7.3 and 7.9; but that launch also costs the host 3 us.  The channels do
// not count, though every tile quantizes the rows again: with more tiles than run at once, 4096 k to MX, 1
// row takes 21 us for 28672 channels (the weights alone 9.7) and 80 for 151936 (51), 8 rows 28 and 116, where
// 16 rows, quantized by a launch of their own, take 16 for 28672.
bool fp4_few_fuses(int64_t M, int64_t K) {
    return M >= 1 && M <= 16 && M * ((K + fp4f::BK - 1) / fp4f::BK) <= 180;
}

template <typename T, bool NV, bool HAS_T, bool FUSED, bool RING>
static ck_status few_launch_ring(const CUtensorMap* maps, const Fp4FewParams& p, int S, int tiles_n, size_t smem,
                            bool dep, cudaStream_t stream) {
    auto kern = fp4_few_kernel<T, NV, HAS_T, FUSED, RING>;
    // the most that any call takes, not this call's: another thread may be about to launch a larger one
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fp4f::SMEM_BUDGET) != cudaSuccess)
        return cuda_error();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)S, (unsigned)tiles_n, (unsigned)((p.M + p.BN - 1) / p.BN));
    cfg.blockDim = dim3(fp4f::THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = dep ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], p) == cudaSuccess ? CK_OK : cuda_error();
}

template <typename T, bool NV, bool HAS_T, bool FUSED>
static ck_status few_launch(const CUtensorMap* maps, const Fp4FewParams& p, int S, int tiles_n, size_t smem,
                            bool dep, cudaStream_t stream) {
    return p.kb_per > p.slots
               ? few_launch_ring<T, NV, HAS_T, FUSED, true>(maps, p, S, tiles_n, smem, dep, stream)
               : few_launch_ring<T, NV, HAS_T, FUSED, false>(maps, p, S, tiles_n, smem, dep, stream);
}

template <typename T>
static ck_status few_fused(const CUtensorMap* maps, const Fp4FewParams& p, bool nv, int S, int tiles_n,
                           size_t smem, cudaStream_t stream) {
    if (!nv) return few_launch<T, false, false, true>(maps, p, S, tiles_n, smem, false, stream);
    return p.x_ts ? few_launch<T, true, true, true>(maps, p, S, tiles_n, smem, false, stream)
                  : few_launch<T, true, false, true>(maps, p, S, tiles_n, smem, false, stream);
}

// a.codes NULL: fused, from the activations x.
ck_status launch_fp4_few(const Fp4Product& a, const void* x, ck_dtype x_dt, int64_t sm, int64_t sk,
                         cudaStream_t stream) {
    using namespace fp4f;
    const bool fused = a.codes == nullptr;
    Fp4FewParams p;
    p.M = (int)a.M;
    p.BN = few_bn(a.M);
    p.N = a.N;
    p.K = a.K;
    p.num_kb = (int)((a.K + BK - 1) / BK);
    const int64_t tiles_n = (a.N + BW - 1) / BW, tiles_m = (a.M + p.BN - 1) / p.BN;
    if (tiles_n >= 65536 || tiles_m >= 65536) return CK_ERR_UNSUPPORTED;
    const FewPlan plan = few_plan(tiles_n * tiles_m, p.num_kb, p.BN, a.nv, fused);
    const int S = plan.S;
    const size_t smem = plan.smem;
    if (smem > SMEM_BUDGET) return CK_ERR_UNSUPPORTED;
    p.kb_per = plan.kb_per;
    p.slots = plan.slots;
    p.b_bytes = (uint32_t)p.BN * (BK / 2);
    p.idesc = idesc_fp4(BW, p.BN, a.nv);
    p.x = x;
    p.sm = sm;
    p.sk = sk;
    const int64_t eb = x_dt == CK_F32 ? 4 : 2;
    p.x_vec = fused && sk == 1 && aligned(x, 16) && sm * eb % 16 == 0;
    p.x_ts = a.x_ts;
    p.w_ts = a.w_ts;
    p.bias = a.bias;
    p.bias_dt = a.bias_dt;
    p.out = a.out;
    p.out_dt = a.out_dt;
    p.ldo = a.ldo;
    p.out_vec = a.ldo % 4 == 0 && aligned(a.out, a.out_dt == CK_F32 ? 16 : 8);
    p.dev_status = a.dev_status;

    CUtensorMap maps[4];
    const uint64_t half = (uint64_t)(a.K / 2), k_tiles = (uint64_t)fp4_k_tiles(a.K, a.nv);
    const uint64_t words = kFp4TileBytes / 4;
    const uint32_t sf_tiles = a.nv ? 4 : 2;
    {
        const uint64_t dims[2] = {half, (uint64_t)a.N}, strides[1] = {(uint64_t)a.w_ld};
        const uint32_t box[2] = {BK / 2, BW};
        const ck_status st = encode_tma(&maps[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.w, dims, strides, box,
                                        CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != CK_OK) return st;
    }
    {
        const uint64_t dims[3] = {words, k_tiles, (uint64_t)tiles_n};
        const uint64_t strides[2] = {kFp4TileBytes, k_tiles * kFp4TileBytes};
        const uint32_t box[3] = {(uint32_t)words, sf_tiles, 1};
        const ck_status st = encode_tma(&maps[3], CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, a.w_scales, dims, strides,
                                        box, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (st != CK_OK) return st;
    }
    maps[0] = maps[1];   // not read when fused
    maps[2] = maps[3];
    if (!fused) {
        const uint64_t dims[2] = {half, (uint64_t)a.M}, strides[1] = {(uint64_t)a.ldq};
        const uint32_t box[2] = {BK / 2, (uint32_t)p.BN};
        ck_status st = encode_tma(&maps[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, a.codes, dims, strides, box,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != CK_OK) return st;
        const uint64_t sdims[3] = {words, k_tiles, (uint64_t)((a.M + kFp4TileRows - 1) / kFp4TileRows)};
        const uint64_t sstrides[2] = {kFp4TileBytes, k_tiles * kFp4TileBytes};
        const uint32_t sbox[3] = {(uint32_t)words, sf_tiles, 1};
        st = encode_tma(&maps[2], CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, a.scales, sdims, sstrides, sbox,
                        CU_TENSOR_MAP_SWIZZLE_NONE);
        if (st != CK_OK) return st;
    }
    if (!fused)
        return a.nv ? few_launch<float, true, false, false>(maps, p, S, (int)tiles_n, smem, a.dependent, stream)
                    : few_launch<float, false, false, false>(maps, p, S, (int)tiles_n, smem, a.dependent, stream);
    switch (x_dt) {
        case CK_F32: return few_fused<float>(maps, p, a.nv, S, (int)tiles_n, smem, stream);
        case CK_F16: return few_fused<__half>(maps, p, a.nv, S, (int)tiles_n, smem, stream);
        case CK_BF16: return few_fused<__nv_bfloat16>(maps, p, a.nv, S, (int)tiles_n, smem, stream);
        default: return CK_ERR_INVALID_ARG;
    }
}

}  // namespace ck

// ck_fp4_few.cu -- the fp4 linear for few rows (M <= 64): a read of the weights, and for the
// smallest calls a chain of latencies.
//
//   out[m, n] = cvt(fl(acc[m, n] * alpha) + bias[n]),   alpha = x_tensor_scale * w_tensor_scale
//
// 128-channel tiles alone would be N / 128 CTAs, so each tile's K is split over a cluster of S CTAs
// (S * N / 128 about one per SM), each of which
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
// Measured, 3840 x 3840: one bf16 row to NV 7.0 us replayed back to back (10.2 with the quantizer and
// the persistent kernel), 32 rows with the quantizer before it 7.5 (10.1); the weights alone are 1.3 us
// of HBM.
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
    int M, BN;               // rows, and the MMA's N
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
    int* dev_status;
};

__device__ __forceinline__ float few_load(const void* p, ck_dtype dt, int64_t i) {
    if (dt == CK_F32) return load_scale<float>(p, i);
    if (dt == CK_F16) return load_scale<__half>(p, i);
    return load_scale<__nv_bfloat16>(p, i);
}

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

    auto load_w = [&](int i, int slot) {
        mbar_arrive_expect_tx(&full[slot], A_BYTES + SF_BYTES);
        tma_load_2d(abuf + (size_t)slot * A_BYTES, &wmap, &full[slot], (kb_lo + i) * (BK / 2), n0);
        tma_load_3d(sfa_buf + (size_t)slot * SF_BYTES, &wsmap, &full[slot], 0, (kb_lo + i) * SF_TILES,
                    (int)blockIdx.y);
    };
    auto load_x = [&](int i, int slot) {
        mbar_arrive_expect_tx(&full[slot], p.b_bytes + SF_BYTES);
        tma_load_2d(bbuf + (size_t)slot * p.b_bytes, &xmap, &full[slot], (kb_lo + i) * (BK / 2), 0);
        tma_load_3d(sfb_buf + (size_t)slot * SF_BYTES, &xsmap, &full[slot], 0, (kb_lo + i) * SF_TILES, 0);
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
        const int total = p.M * groups;
        Fp4Tensor t = fp4_tensor(HAS_T ? p.x_ts : nullptr);
        if (HAS_T && GridBits<T>::value > 0) t.moves = fp4_moves<T>(t.t);
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
                                          p.idesc | (half << 4) | (half << 29), sfa + 4 * tile, sfb + 4 * tile,
                                          (i | j) != 0 ? 1u : 0u);
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
            for (int m0 = 0; m0 < p.M; m0 += 16) {
                uint32_t a[16];
                tc_ld_32x32b_x16(tacc + (uint32_t)m0, a);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (m0 + j < p.M) partial[(m0 + j) * BW + q * 32 + lane] = __uint_as_float(a[j]);
            }
        }
        tc_fence_before();
    }

    // ---------------------------------------------------------------- sum over the cluster
    __syncthreads();
    cluster_sync_all();
    if (!FUSED) grid_dependency_wait();   // also what this kernel writes waits for the one before
    if (!abort_flag) {
        const float alpha = __fmul_rn(p.x_ts ? __ldg(p.x_ts) : 1.0f, p.w_ts ? __ldg(p.w_ts) : 1.0f);
        const int nvec = p.M * (BW / 4);
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
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t n = (int64_t)n0 + c4 + e;
                if (n >= p.N) break;
                float o = __fmul_rn(s[e], alpha);
                if (p.bias) o = __fadd_rn(o, few_load(p.bias, p.bias_dt, n));
                const int64_t at = m * p.ldo + n;
                if (p.out_dt == CK_F32) static_cast<float*>(p.out)[at] = o;
                else if (p.out_dt == CK_F16) static_cast<__half*>(p.out)[at] = __float2half_rn(o);
                else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
            }
        }
    }
    // no CTA leaves while a peer may still read its partial sums, nor with a copy still landing
    cluster_sync_all();
    if (tid == 0 && abort_flag)
        for (int i = max(loaded - R, 0); i < loaded; ++i)
            mbar_wait(&full[i % R], (uint32_t)(i / R) & 1u, nullptr, nullptr);
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// Shared memory of a CTA: `slots` steps of weights, `b_steps` steps of BN rows, the partial sums.
static size_t few_smem_bytes(int slots, int b_steps, int bn, bool nv) {
    using namespace fp4f;
    const size_t sf = (nv ? 4 : 2) * kFp4TileBytes;
    return 1024 + slots * (A_BYTES + sf) + b_steps * ((size_t)bn * (BK / 2) + sf) + (size_t)bn * BW * 4;
}

static int few_bn(int64_t M) { return M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : 64; }

bool fp4_few_takes(int64_t M) { return M >= 1 && M <= 64; }

// Rows x steps of 256 k up to which the tiles quantize for themselves.  Measured (3840 channels, replayed,
// bf16): K = 3840, 8 rows: MX 6.9 us and NV 8.1 against 7.3 and 7.9 with the quantizer in a launch of its
// own; 16 rows: 8.1 and 9.7 against 7.3 and 7.9; but that launch also costs the host 3 us.
bool fp4_few_fuses(int64_t M, int64_t K) {
    return fp4_few_takes(M) && M <= 16 && M * ((K + fp4f::BK - 1) / fp4f::BK) <= 180;
}

template <typename T, bool NV, bool HAS_T, bool FUSED, bool RING>
static ck_status few_launch_ring(const CUtensorMap* maps, const Fp4FewParams& p, int S, int tiles_n, size_t smem,
                            bool dep, cudaStream_t stream) {
    auto kern = fp4_few_kernel<T, NV, HAS_T, FUSED, RING>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return CK_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)S, (unsigned)tiles_n, 1);
    cfg.blockDim = dim3(fp4f::THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = dep ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], p) != cudaSuccess) return CK_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? CK_OK : CK_ERR_CUDA;
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
    const int64_t tiles_n = (a.N + BW - 1) / BW;
    if (tiles_n >= 65536) return CK_ERR_UNSUPPORTED;
    // The smallest split that gives three SMs in four a CTA (3840 x 3840, 32 rows: 4 CTAs a tile 7.45 us,
    // 3 and 5: 8.1 and 7.7), and, fused, leaves half of shared memory for weights.
    const int sms = num_sms();
    int S = 1;
    for (;; ++S) {
        p.kb_per = (p.num_kb + S - 1) / S;
        const bool fits = !fused || few_smem_bytes(0, p.kb_per, p.BN, a.nv) <= SMEM_BUDGET / 2;
        if ((4 * S * tiles_n >= 3 * (int64_t)sms && fits) || S == MAX_CLUSTER || S >= p.num_kb) break;
    }
    S = (p.num_kb + p.kb_per - 1) / p.kb_per;   // every rank has a step
    p.slots = p.kb_per < SLOTS_MAX ? p.kb_per : SLOTS_MAX;
    while (p.slots > 1 && few_smem_bytes(p.slots, fused ? p.kb_per : p.slots, p.BN, a.nv) > SMEM_BUDGET) --p.slots;
    const size_t smem = few_smem_bytes(p.slots, fused ? p.kb_per : p.slots, p.BN, a.nv);
    if (smem > SMEM_BUDGET) return CK_ERR_UNSUPPORTED;
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
        const uint64_t sdims[3] = {words, k_tiles, 1};
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

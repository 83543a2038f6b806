// ck_fp4_quant.cu -- activations or weights to microscaled 4-bit floating point, and back.
//
//   quantize:   per block of 32 (MX) or 16 (NV) along K: scale from the block's absmax, then
//               code = e2m1(x / scale); see ck_fp4.cuh for the arithmetic of one block
//   dequantize: value = cvt(fl(fl(code * scale) * t))
//
// Both are one pass over memory: K * sizeof(x) + K / 2 + K / block bytes a row, 12.5 us for 8192 x 3840
// bf16 at the measured copy rate.  Measured there: MX 15.2 us, NV with a tensor scale 20 to 22 (about 202
// instructions a thread and block, of them 50 for the scale; the integer pipe is 60% busy, issue 64%, and a
// warp waits most for its loads), back 13.9 to 14.3; 4096 x 16384 fp32: NV 49 us (48 at the copy rate),
// column-major 55, back 51.
// A CTA takes 128 rows x 128 channels, so that it owns whole 512-byte scale tiles and writes each
// of them as one contiguous run from shared memory; a thread takes sixteen channels of a row (an
// NV block, or half an MX block whose other half is its neighbour lane's), with the loads of
// several rows in flight.  Column-major input goes through a transposing shared-memory buffer.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ck_device.cuh"
#include "ck_fp4.cuh"
#include "ck_internal.h"

namespace ck {

namespace fp4q {
constexpr int THREADS = 256;
constexpr int ROWS = kFp4TileRows;    // rows of a CTA's tile
constexpr int COLS = 128;             // channels of a CTA's tile
constexpr int LANES = COLS / 16;      // threads across a row
constexpr int STEP = THREADS / LANES; // rows a pass of the CTA covers
constexpr int PASSES = ROWS / STEP;
constexpr int COL_CHUNK = 64;         // channels of a column-major tile that are waited for at a time
enum Layout { VEC = 0, ANY = 1, COL = 2 };
}  // namespace fp4q

struct Fp4QuantParams {
    const void* x;
    int64_t M, K, sm, sk;
    const float* tensor_scale;
    const int32_t* offsets;   // NULL: one matrix
    int n_experts;
    int64_t k_tiles;          // 512-byte scale tiles along K
    int col_ctas;             // CTAs along K
    uint8_t* codes;
    int64_t ldq;
    bool codes_vec;           // 8-byte code stores
    bool x_wide;              // 32-byte loads (VEC, fp32: 59 -> 57 us at 4096 x 16384; bf16 lost 5%)
    uint8_t* scales;
};

// The rows [row0, row0 + n) of scale block rb: 128 rows of the one matrix, or of the expert whose
// scale blocks hold rb (n = 0 where no expert's do).  Every warp looks for itself, 32 experts at a
// time: one load's latency, no barrier.
__device__ __forceinline__ void rows_of_block(const int32_t* offsets, int n_experts, int64_t M,
                                              int64_t rb, int64_t& row0, int& n) {
    using namespace fp4q;
    if (!offsets) {
        row0 = rb * ROWS;
        n = (int)((M - row0) < ROWS ? (M - row0) : ROWS);
        return;
    }
    row0 = 0;
    n = 0;
    for (int e0 = 0; e0 < n_experts; e0 += 32) {
        const int e = e0 + (threadIdx.x & 31);
        int first = 0, rows = 0;
        if (e < n_experts) {
            const RowRange r = expert_rows(offsets, e, M);
            const int64_t at = r.lo + (rb - expert_scale_block(r.lo, e)) * ROWS;
            if (at >= r.lo && at < r.hi) {
                first = (int)at;
                rows = (int)(r.hi - at < ROWS ? r.hi - at : ROWS);
            }
        }
        const uint32_t found = __ballot_sync(0xffffffffu, rows > 0);
        if (found) {
            const int lane = __ffs((int)found) - 1;
            row0 = __shfl_sync(0xffffffffu, first, lane);
            n = __shfl_sync(0xffffffffu, rows, lane);
            return;
        }
    }
}

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {   // all but the last N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sixteen consecutive elements at p as loaded words, and as fp32 values.
template <typename T> struct Raw16 {
    uint32_t w[4 * sizeof(T)];
    // wide: 32-byte loads, otherwise 16-byte ones
    __device__ __forceinline__ void load(const T* p, bool wide) {
        if (sizeof(T) == 4 && wide) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                    : "=r"(w[8 * i]), "=r"(w[8 * i + 1]), "=r"(w[8 * i + 2]), "=r"(w[8 * i + 3]),
                      "=r"(w[8 * i + 4]), "=r"(w[8 * i + 5]), "=r"(w[8 * i + 6]), "=r"(w[8 * i + 7])
                    : "l"(p + 32 / sizeof(T) * i));
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4 * (int)sizeof(T); ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (sizeof(T) == 4) {
                v[i] = __uint_as_float(w[i]);
            } else {
                const uint16_t h = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                v[i] = Elem<T>::to_f(*reinterpret_cast<const T*>(&h));
            }
        }
    }
};

// The scale byte of the block of channel group g in row r of the CTA's tile, into its place in the
// shared scale tiles (an MX block's from its first half's lane).
template <bool NV>
__device__ __forceinline__ void put_scale(uint8_t* sf, int r, int g, uint32_t byte) {
    const int c = NV ? g : g >> 1;
    if (NV || !(g & 1)) sf[(c >> 2) * kFp4TileBytes + fp4_tile_byte(r, c & 3)] = (uint8_t)byte;
}

__device__ __forceinline__ void store_codes(uint8_t* dst, const uint32_t (&c)[2], bool vec) {
    if (vec) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
    }
}

template <typename T, bool NV, bool HAS_T, int LAYOUT>
__global__ void __launch_bounds__(fp4q::THREADS, 4)
    fp4_quant_kernel(Fp4QuantParams p) {
    using namespace fp4q;
    constexpr int TILES = COLS / 4 / fp4_block(NV);   // scale tiles across the CTA's columns
    __shared__ __align__(16) uint8_t sf[TILES * kFp4TileBytes];
    extern __shared__ __align__(16) unsigned char q_smem[];
    const int tid = threadIdx.x;
    grid_dependents_launch();
    for (int i = tid; i < TILES * kFp4TileBytes / 16; i += THREADS)
        reinterpret_cast<uint4*>(sf)[i] = make_uint4(0, 0, 0, 0);

    const int64_t rb = blockIdx.x / p.col_ctas;
    const int cc = (int)(blockIdx.x % p.col_ctas);
    const int64_t k0 = (int64_t)cc * COLS;
    int64_t row0;
    int n;
    rows_of_block(p.offsets, p.n_experts, p.M, rb, row0, n);
    if (n == 0) return;
    Fp4Tensor t = fp4_tensor(HAS_T ? p.tensor_scale : nullptr);
    constexpr bool MOVES = NV && HAS_T && GridBits<T>::value > 0;
    __shared__ uint2 moves;
    if (MOVES && tid < 32) {
        const uint2 m = fp4_moves<T>(t.t);
        if (tid == 0) moves = m;
    }
    __syncthreads();   // and the cleared scale tiles
    if (MOVES) {
        t.moves = moves.x;
        t.ups = moves.y;
    }
    const T* x = static_cast<const T*>(p.x);

    if (LAYOUT == COL) {
        // Rows are contiguous in memory, so a warp copies 128 of them of one channel in a run; a thread then
        // takes sixteen channels of one row, lanes on neighbouring rows (no bank conflicts: the buffer's
        // row index is fastest).  The whole tile is asked for at once and quantized in pieces of 64
        // channels as they arrive (4096 x 16384 fp32 to
        // NV: 55 us; piece by piece through registers, with a buffer of one, 74; bf16 41 against 67).  Columns
        // that are not aligned to 16 bytes are copied by 4 (15322 x 2304 fp16 to MX: 28 us), 16-bit ones of
        // an odd pitch by elements (54).
        T* buf = reinterpret_cast<T*>(q_smem);                      // [COLS][ROWS]
        uint8_t* cbuf = q_smem + (size_t)COLS * ROWS * sizeof(T);   // [ROWS][COLS / 2 + 16]
        constexpr int CP = COLS / 2 + 16;
        constexpr int PER = 16 / (int)sizeof(T);                    // elements of 16 bytes
        const int kmax = (int)((p.K - k0) < COLS ? (p.K - k0) : COLS);
        const bool wide = reinterpret_cast<uintptr_t>(x + row0) % 16 == 0 &&
                          (p.sk * (int64_t)sizeof(T)) % 16 == 0;
        const bool words = sizeof(T) == 4 || (reinterpret_cast<uintptr_t>(x + row0) % 4 == 0 && p.sk % 2 == 0);
#pragma unroll
        for (int c0 = 0; c0 < COLS; c0 += COL_CHUNK) {
            constexpr int N16 = ROWS / PER;
            if (wide && n == ROWS) {   // without the tests of a ragged tile: 61 us with them
#pragma unroll 8
                for (int i = tid; i < COL_CHUNK * N16; i += THREADS) {
                    const int c = c0 + i / N16, m = (i % N16) * PER;
                    if (c < kmax) cp_async_16(buf + c * ROWS + m, x + row0 + m + (k0 + c) * p.sk);
                }
            } else if (wide) {
                for (int i = tid; i < COL_CHUNK * N16; i += THREADS) {
                    const int c = c0 + i / N16, m = (i % N16) * PER;
                    T* dst = buf + c * ROWS + m;
                    const T* src = x + row0 + m + (k0 + c) * p.sk;
                    if (c < kmax && m + PER <= n) cp_async_16(dst, src);
                    else if (c < kmax && m < n)
                        for (int e = 0; e < n - m; ++e) dst[e] = src[e];
                }
            } else if (words) {
                constexpr int PER4 = 4 / (int)sizeof(T), N4 = ROWS / PER4;
#pragma unroll 8
                for (int i = tid; i < COL_CHUNK * N4; i += THREADS) {
                    const int c = c0 + i / N4, m = (i % N4) * PER4;
                    T* dst = buf + c * ROWS + m;
                    const T* src = x + row0 + m + (k0 + c) * p.sk;
                    if (c < kmax && m + PER4 <= n) cp_async_4(dst, src);
                    else if (c < kmax && m < n) *dst = *src;
                }
            } else {
                for (int i = tid; i < COL_CHUNK * ROWS; i += THREADS) {
                    const int c = c0 + i / ROWS, m = i % ROWS;
                    if (c < kmax && m < n) buf[c * ROWS + m] = x[row0 + m + (k0 + c) * p.sk];
                }
            }
            cp_async_commit();
        }
#pragma unroll
        for (int c0 = 0; c0 < COLS; c0 += COL_CHUNK) {
            if (c0 >= kmax) break;
            const int nc = (kmax - c0) < COL_CHUNK ? (kmax - c0) : COL_CHUNK;
            if (c0 + COL_CHUNK < COLS) cp_async_wait<COLS / COL_CHUNK - 1>();
            else cp_async_wait<0>();
            __syncthreads();
            if (NV) {
                for (int i = tid; i < nc / 16 * ROWS; i += THREADS) {
                    const int g = i / ROWS, r = i % ROWS;
                    if (r < n) {
                        float v[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = Elem<T>::to_f(buf[(c0 + g * 16 + j) * ROWS + r]);
                        uint32_t c[2];
                        const Fp4Scale b = fp4_scale<T, NV, HAS_T>(absmax16(v), t);
                        fp4_codes<T, NV, HAS_T>(v, b, c);
                        put_scale<NV>(sf, r, c0 / 16 + g, b.byte);
                        store_codes(cbuf + r * CP + (c0 + g * 16) / 2, c, true);
                    }
                }
            } else {
                for (int i = tid; i < nc / 32 * ROWS; i += THREADS) {
                    const int g = i / ROWS, r = i % ROWS;
                    if (r < n) {
                        float v[2][16];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j >> 4][j & 15] = Elem<T>::to_f(buf[(c0 + g * 32 + j) * ROWS + r]);
                        const Fp4Scale b = fp4_scale<T, NV, HAS_T>(max(absmax16(v[0]), absmax16(v[1])), t);
                        put_scale<NV>(sf, r, c0 / 16 + 2 * g, b.byte);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t c[2];
                            fp4_codes<T, NV, HAS_T>(v[h], b, c);
                            store_codes(cbuf + r * CP + (c0 + g * 32 + 16 * h) / 2, c, true);
                        }
                    }
                }
            }
        }
        __syncthreads();
        // the rows' codes, eight bytes a thread
        const int pieces = kmax / 16;
        for (int i = tid; i < ROWS * LANES; i += THREADS) {
            const int r = i / LANES, c = i % LANES;
            if (r < n && c < pieces) {
                const uint2 u = *reinterpret_cast<const uint2*>(cbuf + r * CP + c * 8);
                const uint32_t w[2] = {u.x, u.y};
                store_codes(p.codes + (row0 + r) * p.ldq + k0 / 2 + c * 8, w, p.codes_vec);
            }
        }
    } else {
        const int g = tid % LANES, r0 = tid / LANES;
        const int64_t k = k0 + g * 16;
        const bool k_ok = k < p.K;
        // K is a multiple of the block: a group of sixteen is whole, and so is an MX pair
        constexpr int AHEAD = NV ? 2 : 4;   // rows whose loads are in flight, within 64 registers
        if (LAYOUT == VEC) {
#pragma unroll 1
            for (int it = 0; it < PASSES; it += AHEAD) {
                if (it * STEP >= n) break;
                Raw16<T> raw[AHEAD];
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    const int r = (it + a) * STEP + r0;
                    if (k_ok && r < n) raw[a].load(x + (row0 + r) * p.sm + k, p.x_wide);
                    else raw[a].zero();
                }
                // the blocks' scales first, side by side: each is a chain of dependent operations
                Fp4Scale b[AHEAD];
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    float v[16];
                    raw[a].values(v);
                    uint32_t amax = absmax16(v);
                    if (!NV) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    b[a] = fp4_scale<T, NV, HAS_T>(amax, t);
                }
#pragma unroll
                for (int a = 0; a < AHEAD; ++a) {
                    const int r = (it + a) * STEP + r0;
                    float v[16];
                    raw[a].values(v);
                    uint32_t c[2];
                    fp4_codes<T, NV, HAS_T>(v, b[a], c);
                    if (k_ok && r < n) {
                        put_scale<NV>(sf, r, g, b[a].byte);
                        store_codes(p.codes + (row0 + r) * p.ldq + k / 2, c, p.codes_vec);
                    }
                }
            }
        } else {
#pragma unroll 1
            for (int it = 0; it < PASSES; ++it) {
                if (it * STEP >= n) break;
                const int r = it * STEP + r0;
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    v[j] = k_ok && r < n ? Elem<T>::to_f(x[(row0 + r) * p.sm + (k + j) * p.sk]) : 0.0f;
                uint32_t amax = absmax16(v);
                if (!NV) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                const Fp4Scale b = fp4_scale<T, NV, HAS_T>(amax, t);
                uint32_t c[2];
                fp4_codes<T, NV, HAS_T>(v, b, c);
                if (k_ok && r < n) {
                    put_scale<NV>(sf, r, g, b.byte);
                    store_codes(p.codes + (row0 + r) * p.ldq + k / 2, c, p.codes_vec);
                }
            }
        }
    }
    __syncthreads();
    // the CTA's scale tiles: one contiguous run, zero past the last row and block
    const int64_t t0 = (int64_t)cc * TILES;
    const int nt = (int)((p.k_tiles - t0) < TILES ? (p.k_tiles - t0) : TILES);
    uint4* dst = reinterpret_cast<uint4*>(p.scales + (rb * p.k_tiles + t0) * kFp4TileBytes);
    for (int i = tid; i < nt * kFp4TileBytes / 16; i += THREADS)
        dst[i] = reinterpret_cast<const uint4*>(sf)[i];
}

struct Fp4DequantParams {
    const uint8_t* codes;
    int64_t ldq;
    const uint8_t* scales;
    int64_t M, K;
    const float* tensor_scale;
    const int32_t* offsets;
    int n_experts;
    int64_t k_tiles;
    int col_ctas;
    bool codes_vec, out_vec;   // 4-byte code loads, eight outputs in one store
    void* out;
    int64_t ldo;
};

template <typename T, bool NV>
__global__ void __launch_bounds__(fp4q::THREADS)
    fp4_dequant_kernel(Fp4DequantParams p) {
    using namespace fp4q;
    constexpr int TILES = COLS / 4 / fp4_block(NV);
    __shared__ __align__(16) uint8_t sf[TILES * kFp4TileBytes];
    const int tid = threadIdx.x;
    const int64_t rb = blockIdx.x / p.col_ctas;
    const int cc = (int)(blockIdx.x % p.col_ctas);
    int64_t row0;
    int n;
    rows_of_block(p.offsets, p.n_experts, p.M, rb, row0, n);
    if (n == 0) return;
    const int64_t t0 = (int64_t)cc * TILES;
    const int nt = (int)((p.k_tiles - t0) < TILES ? (p.k_tiles - t0) : TILES);
    const uint4* src = reinterpret_cast<const uint4*>(p.scales + (rb * p.k_tiles + t0) * kFp4TileBytes);
    for (int i = tid; i < nt * kFp4TileBytes / 16; i += THREADS)
        reinterpret_cast<uint4*>(sf)[i] = __ldg(src + i);
    __syncthreads();
    const float t = p.tensor_scale ? __ldg(p.tensor_scale) : 1.0f;
    // eight channels a thread: a warp's stores are whole rows of the tile, 16 or 32 bytes a lane
    constexpr int LANES8 = COLS / 8, STEP8 = THREADS / LANES8, PASSES8 = ROWS / STEP8;
    const int g = tid % LANES8, r0 = tid / LANES8;
    const int64_t k = (int64_t)cc * COLS + g * 8;
    if (k >= p.K) return;
    const int c = g / (fp4_block(NV) / 8);
    T* out = static_cast<T*>(p.out);
    uint32_t word[PASSES8];   // every row's codes in flight at once
#pragma unroll
    for (int it = 0; it < PASSES8; ++it) {
        const int r = it * STEP8 + r0;
        const uint8_t* src4 = p.codes + (row0 + r) * p.ldq + k / 2;
        word[it] = 0u;
        if (r < n && p.codes_vec) {
            word[it] = __ldg(reinterpret_cast<const uint32_t*>(src4));
        } else if (r < n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) word[it] |= (uint32_t)__ldg(src4 + i) << (8 * i);
        }
    }
#pragma unroll
    for (int it = 0; it < PASSES8; ++it) {
        const int r = it * STEP8 + r0;
        if (r >= n) break;
        const uint32_t byte = sf[(c >> 2) * kFp4TileBytes + fp4_tile_byte(r, c & 3)];
        const float s = NV ? e4m3_value(byte) : e8m0_value(byte);
        T* dst = out + (row0 + r) * p.ldo + k;
        float v[8];
        fp4_unpack8(word[it], v);
        __align__(32) T o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)   // code * scale is exact: at most six significant bits
            o[i] = Elem<T>::from_f(__fmul_rn(__fmul_rn(v[i], s), t));
        if (p.out_vec) {
            const uint32_t* u = reinterpret_cast<const uint32_t*>(o);
            if (sizeof(T) == 4)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]),
                             "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4 % (2 * sizeof(T))]),
                             "r"(u[5 % (2 * sizeof(T))]), "r"(u[6 % (2 * sizeof(T))]),
                             "r"(u[7 % (2 * sizeof(T))])
                             : "memory");
            else
                *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = o[i];
        }
    }
}

static int64_t row_blocks(int64_t M, const int32_t* offsets, int n_experts) {
    return offsets ? M / kFp4TileRows + n_experts : (M + kFp4TileRows - 1) / kFp4TileRows;
}

// Launched so that the launch's own status is returned, not what an earlier call left as the last error.
template <typename P>
static ck_status launch(void (*kern)(P), const P& p, int64_t grid, int smem, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(fp4q::THREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? CK_OK : cuda_error();
}

template <typename T, bool NV, bool HAS_T>
static ck_status quant_launch(const Fp4QuantParams& p, int64_t grid, cudaStream_t stream) {
    using namespace fp4q;
    const int64_t eb = sizeof(T);
    if (p.sk == 1 && aligned(p.x, 16) && p.sm * eb % 16 == 0)
        return launch(fp4_quant_kernel<T, NV, HAS_T, VEC>, p, grid, 0, stream);
    if (p.sm == 1 && p.M >= 32) {
        // the channel runs of at least 32 rows are worth the transposing buffer
        constexpr int smem = COLS * ROWS * (int)sizeof(T) + ROWS * (COLS / 2 + 16);
        auto kern = fp4_quant_kernel<T, NV, HAS_T, COL>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return cuda_error();
        return launch(kern, p, grid, smem, stream);
    }
    return launch(fp4_quant_kernel<T, NV, HAS_T, ANY>, p, grid, 0, stream);
}

template <typename T>
static ck_status quant_typed(const Fp4QuantParams& p, bool nv, int64_t grid, cudaStream_t stream) {
    if (!nv) return quant_launch<T, false, false>(p, grid, stream);
    if (p.tensor_scale) return quant_launch<T, true, true>(p, grid, stream);
    return quant_launch<T, true, false>(p, grid, stream);
}

ck_status launch_quant_fp4(const void* x, ck_dtype dt, int64_t M, int64_t K, int64_t sm, int64_t sk,
                           bool nv, const float* tensor_scale, const int32_t* offsets, int n_experts,
                           uint8_t* codes, int64_t ldq, uint8_t* scales, cudaStream_t stream) {
    Fp4QuantParams p;
    p.x = x;
    p.M = M;
    p.K = K;
    p.sm = sm;
    p.sk = sk;
    p.tensor_scale = tensor_scale;
    p.offsets = offsets;
    p.n_experts = n_experts;
    p.k_tiles = fp4_k_tiles(K, nv);
    p.codes = codes;
    p.ldq = ldq;
    p.codes_vec = aligned(codes, 8) && ldq % 8 == 0;
    p.x_wide = dt == CK_F32 && aligned(x, 32) && sm % 8 == 0;
    p.scales = scales;
    const int64_t cols = (K + fp4q::COLS - 1) / fp4q::COLS;
    const int64_t grid = cols * row_blocks(M, offsets, n_experts);
    if (grid >= (1LL << 31)) return CK_ERR_UNSUPPORTED;
    p.col_ctas = (int)cols;
    switch (dt) {
        case CK_F32: return quant_typed<float>(p, nv, grid, stream);
        case CK_F16: return quant_typed<__half>(p, nv, grid, stream);
        case CK_BF16: return quant_typed<__nv_bfloat16>(p, nv, grid, stream);
        default: return CK_ERR_INVALID_ARG;
    }
}

template <typename T>
static ck_status dequant_typed(const Fp4DequantParams& p, bool nv, int64_t grid, cudaStream_t stream) {
    return nv ? launch(fp4_dequant_kernel<T, true>, p, grid, 0, stream)
              : launch(fp4_dequant_kernel<T, false>, p, grid, 0, stream);
}

ck_status launch_dequant_fp4(const uint8_t* codes, int64_t ldq, const uint8_t* scales, int64_t M,
                             int64_t K, bool nv, const float* tensor_scale, const int32_t* offsets,
                             int n_experts, void* out, ck_dtype out_dt, int64_t ldo,
                             cudaStream_t stream) {
    const int64_t eb = out_dt == CK_F32 ? 4 : 2;
    Fp4DequantParams p;
    p.codes = codes;
    p.ldq = ldq;
    p.scales = scales;
    p.M = M;
    p.K = K;
    p.tensor_scale = tensor_scale;
    p.offsets = offsets;
    p.n_experts = n_experts;
    p.k_tiles = fp4_k_tiles(K, nv);
    p.codes_vec = aligned(codes, 4) && ldq % 4 == 0;
    p.out_vec = aligned(out, 8 * eb) && ldo % 8 == 0;
    p.out = out;
    p.ldo = ldo;
    const int64_t cols = (K + fp4q::COLS - 1) / fp4q::COLS;
    const int64_t grid = cols * row_blocks(M, offsets, n_experts);
    if (grid >= (1LL << 31)) return CK_ERR_UNSUPPORTED;
    p.col_ctas = (int)cols;
    switch (out_dt) {
        case CK_F32: return dequant_typed<float>(p, nv, grid, stream);
        case CK_F16: return dequant_typed<__half>(p, nv, grid, stream);
        case CK_BF16: return dequant_typed<__nv_bfloat16>(p, nv, grid, stream);
        default: return CK_ERR_INVALID_ARG;
    }
}

}  // namespace ck

// ck_fp4.cuh -- microscaled 4-bit floating point: the formats, the layout of the block scales,
// and the quantizer of one block, shared by the fp4 kernels.
//
// Elements are E2M1 (sign, two exponent bits, one mantissa bit): 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// their negatives, two to a byte with the even k in the low nibble.  Blocks along K share a scale:
//   CK_MXFP4  32 elements, E8M0 scale 2^(byte - 127), 255 = NaN (OCP Microscaling Formats v1.0)
//   CK_NVFP4  16 elements, E4M3 scale under a per-tensor fp32 scale
// The scales of 128 rows x 4 blocks form a 512-byte tile, the order in which tcgen05.cp puts them
// into tensor memory: row r, block c at byte (r % 32) * 16 + (r / 32) * 4 + c.
#pragma once

#include <stdint.h>

#include "ck_device.cuh"

namespace ck {

constexpr int kFp4TileRows = 128;
constexpr int kFp4TileBytes = 512;

__host__ __device__ constexpr int fp4_block(bool nv) { return nv ? 16 : 32; }

// 512-byte scale tiles along K.
__host__ __device__ inline int64_t fp4_k_tiles(int64_t K, bool nv) {
    const int64_t per = 4 * fp4_block(nv);
    return (K + per - 1) / per;
}

// Byte of (row r of a 128-row block, block c of a 4-block tile) within its tile.
__host__ __device__ constexpr int fp4_tile_byte(int r, int c) {
    return (r % 32) * 16 + (r / 32) * 4 + c;
}

// The rows of expert e, [lo, hi): the caller's offsets clamped to [0, M], empty where they
// decrease, so that no index derived from them leaves the tensors.
struct RowRange {
    int64_t lo, hi;
};
__device__ __forceinline__ RowRange expert_rows(const int32_t* offsets, int e, int64_t M) {
    int64_t lo = __ldg(offsets + e), hi = __ldg(offsets + e + 1);
    lo = lo < 0 ? 0 : (lo > M ? M : lo);
    hi = hi < lo ? lo : (hi > M ? M : hi);
    return {lo, hi};
}
// The 128-row scale block at which expert e's rows start.  ceil((hi - lo) / 128) is at most
// hi / 128 - lo / 128 + 1, so the blocks of different experts never overlap, and all of them lie
// below M / 128 + n_experts, without a running sum over the experts.
__host__ __device__ inline int64_t expert_scale_block(int64_t lo, int e) {
    return lo / kFp4TileRows + e;
}

// Eight values -> eight E2M1 codes, the first in the lowest nibble: round half to even,
// saturating at +-6.
__device__ __forceinline__ uint32_t fp4_pack8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight E2M1 codes -> eight values.
__device__ __forceinline__ void fp4_unpack8(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// Byte -> E4M3 value (sign bit clear; 0x7F is NaN), and a non-negative value -> E4M3 byte (round
// half to even, saturating at 448).
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h;
    const uint16_t b = (uint16_t)byte;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
    return __low2float(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t e4m3_byte(float v) {
    uint16_t b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.0f), "f"(v));
    return (uint32_t)b & 0xFFu;
}

// 2^(byte - 127) for byte 0..254 (byte 0 is the subnormal 2^-127), NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    if (byte == 255u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// fl(a / b) for b > 0, a >= 0, rounded to odd: the quotient cut to 24 bits with the last bit set
// where anything was cut.  Rounded once more to fewer than 23 bits it gives what the exact
// quotient would.  q is the correctly rounded quotient; e = a - q b is exact unless it underflows,
// which the callers exclude.
__device__ __forceinline__ float odd_from_rn(float q, float a, float b) {
    const float e = __fmaf_rn(-q, b, a);
    uint32_t u = __float_as_uint(q);
    u -= e < 0.0f ? 1u : 0u;
    u |= e != 0.0f ? 1u : 0u;
    return __uint_as_float(u);
}

// The E4M3 byte of amax / c (c = fl(6 t)), rounded from the exact quotient.
__device__ __forceinline__ uint32_t nv_scale_byte(float amax, float c) {
    if (c < 0x1p-60f) {   // far from the subnormal range; an overflow of amax saturates as it should
        amax = __fmul_rn(amax, 0x1p64f);
        c = __fmul_rn(c, 0x1p64f);
    }
    // below 2^-60 / 2^40 the quotient rounds to zero whatever the remainder's last bits say
    float q = __fdiv_rn(amax, c);
    if (q < 1024.0f && amax > 0x1p-100f) q = odd_from_rn(q, amax, c);
    return e4m3_byte(q);
}

// Code of one value by comparing it with the borders times d, exactly (3-bit border times 24-bit
// d in fp64): the path of blocks whose scale is too small or large for the fp32 quotient.
static __device__ __noinline__ uint32_t fp4_code_exact(float x, float d) {
    const double a = fabs((double)x), s = (double)d;
    uint32_t n = 0;
    n += a > 0.25 * s;
    n += a >= 0.75 * s;
    n += a > 1.25 * s;
    n += a >= 1.75 * s;
    n += a > 2.5 * s;
    n += a >= 3.5 * s;
    n += a > 5.0 * s;
    return n | (__float_as_uint(x) >> 28 & 8u);
}

// What the quantizer of a tensor keeps across its blocks.
struct Fp4Tensor {
    float t;      // the tensor scale (NV)
    float c;      // fl(6 t)
    bool t_ok;    // a positive finite number; otherwise every scale is NaN
};
__device__ __forceinline__ Fp4Tensor fp4_tensor(const float* tensor_scale) {
    Fp4Tensor p;
    p.t = tensor_scale ? __ldg(tensor_scale) : 1.0f;
    p.c = __fmul_rn(6.0f, p.t);
    p.t_ok = p.t > 0.0f && p.t <= 3.40282347e38f;
    return p;
}

// Sixteen values of one block (a whole NV block, half an MX block) with the block's absmax given
// as the bits of an fp32 number (above infinity's for a NaN) -> sixteen codes and the block's
// scale byte.  HAS_T: a tensor scale other than one may be given.
//
// MX: byte = max(exponent field - 2, 0); x 2^-(byte - 127) is exact, so the conversion's rounding
//     is the only one.
// NV: s = e4m3(amax / c), d = fl(s t), code = e2m1(x / d).  The quotient is the correctly rounded
//     one (reciprocal, one residual, one correction: see RowDivisor).  Where d = s has four bits,
//     a quotient that is not on a border between two codes is at least 2^-24 of it away, so its
//     rounding to 24 bits never moves it onto one; d = fl(s t) has 24 bits, and there the quotient
//     is rounded to odd.
template <bool NV, bool HAS_T>
__device__ __forceinline__ uint32_t fp4_quant16(const float (&x)[16], uint32_t amax_bits,
                                                const Fp4Tensor& p, uint32_t (&codes)[2]) {
    codes[0] = codes[1] = 0u;
    if (!NV) {
        if (amax_bits >= 0x7F800000u) return 0xFFu;
        const int byte = max((int)(amax_bits >> 23) - 2, 0);
        // 2^(127 - byte): exponent field 254 - byte, in 2..254
        const float r = __uint_as_float((uint32_t)(254 - byte) << 23);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(x[8 * h + i], r);
            codes[h] = fp4_pack8(v);
        }
        return (uint32_t)byte;
    }
    if (amax_bits >= 0x7F800000u || (HAS_T && !p.t_ok)) return 0x7Fu;
    const float amax = __uint_as_float(amax_bits);
    const uint32_t byte = nv_scale_byte(amax, p.c);
    const float s = e4m3_value(byte);
    const float d = HAS_T ? __fmul_rn(s, p.t) : s;
    if (d == 0.0f) return byte;
    if (d >= 0x1p-60f && d <= 0x1p60f && amax <= 16.0f * d) {
        const float r = __frcp_rn(d);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = fabsf(x[8 * h + i]);
                const float q0 = __fmul_rn(a, r);
                const float e = __fmaf_rn(-q0, d, a);
                float q = __fmaf_rn(e, r, q0);
                if (HAS_T) q = odd_from_rn(q, a, d);
                v[i] = copysignf(q, x[8 * h + i]);
            }
            codes[h] = fp4_pack8(v);
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            float v = x[0];   // x[i] without a local-memory array
#pragma unroll
            for (int j = 1; j < 16; ++j) v = i == j ? x[j] : v;
            const uint32_t n = fp4_code_exact(v, d) << (4 * (i & 7));
            if (i < 8) codes[0] |= n;
            else codes[1] |= n;
        }
    }
    return byte;
}

// Bits of the largest |x| of sixteen, as an fp32 number's; NaN gives bits above infinity's.
__device__ __forceinline__ uint32_t absmax16(const float (&x)[16]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
}

}  // namespace ck

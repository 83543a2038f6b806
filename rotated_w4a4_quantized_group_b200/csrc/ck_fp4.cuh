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

// Counts of tiles added up, at most the largest int.  Offsets that do not decrease give fewer (the host
// sees to that); others may give half of the experts all the rows, and a sum that wrapped would lead
// out of the tensors.  Still associative: every partial sum is the true one or the largest int.
__host__ __device__ inline int tiles_add(int a, int b) {
    const uint32_t s = (uint32_t)a + (uint32_t)b;
    return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int)s;
}
// Of `tiles`, those that unit u of `units` takes: u, u + units, ...
__host__ __device__ inline uint32_t tiles_of_unit(int tiles, int u, int units) {
    return tiles > u ? ((uint32_t)(tiles - u) + (uint32_t)units - 1u) / (uint32_t)units : 0u;
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

// 1 / d within one step, for d and 1 / d far from the subnormal range.
__device__ __forceinline__ float reciprocal(float d) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
    return __fmaf_rn(__fmaf_rn(-d, r, 1.0f), r, r);
}

// Code of one value by comparing it with the borders times d, exactly (3-bit border times 24-bit
// d in fp64): the path of blocks whose scale is too small or large for the fp32 quotient.
__device__ __forceinline__ uint32_t fp4_code_exact(float x, float d) {
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

// The significant bits of a type's values below which an fp32 mantissa is zero.
template <typename T> struct GridBits { static constexpr int value = 0; };          // fp32: none
template <> struct GridBits<__nv_bfloat16> { static constexpr int value = 16; };
template <> struct GridBits<__half> { static constexpr int value = 13; };

// What the quantizer of a tensor keeps across its blocks.
struct Fp4Tensor {
    float t;      // the tensor scale (NV)
    float c;      // fl(6 t), brought between 2^-83 and 2^64 by a power of two
    float rc;     // 1 / c
    float up;     // that power
    bool t_ok;    // a positive finite number; otherwise every scale is NaN
    bool t_mid;   // far enough from the ends for every s t and its reciprocal to be normal
    // bits 4 i to 4 i + 3, signed: how many steps the reciprocal of blocks whose scale has mantissa
    // 1 + i / 8 is moved; -8 where some borders want -8 and others 8
    uint32_t moves;
    uint32_t ups;   // bit 4 i + j: that scale's borders of mantissa 1 + j / 4 want the larger one
};

// x * r, r within a step of 1 / d, d = fl(s t), rounds to the code of x / d for every x of a 16-bit
// type but those on which a border (0.25 to 5; four mantissas) times d all but falls: with t an
// absmax / 2688, the usual calibration, every third block has such a border, and with a t of few bits
// x may be on it.  They want r a little larger (x above its border, or to be rounded up from it) or a
// little smaller, which depends on the mantissas of s, border and t alone, so a warp finds it once for
// all 8 x 4 pairs; where a scale's borders disagree, its blocks are rounded both ways and each code
// takes its border's.  In steps of a mantissa: r, the
// product and the border are off by less than 3 together, so seven or eight decide every such x, and no value
// further than 24 from its border is moved over it; the next value of the type is at least 2^12
// steps away.  Every lane of the warp calls it; gives Fp4Tensor::moves and ups.
template <typename T>
__device__ __forceinline__ uint2 fp4_moves(float t) {
    constexpr int GRID = GridBits<T>::value;
    constexpr int mask = (1 << GRID) - 1;
    const int lane = threadIdx.x & 31;
    const float tm = __uint_as_float((__float_as_uint(t) & 0x007FFFFFu) | 0x3F800000u);
    const float d = __fmul_rn(1.0f + 0.125f * (lane >> 2), tm), m = 1.0f + 0.25f * (lane & 3);
    const int b = __float_as_int(__fmul_rn(d, m));
    const int g = (b + (mask + 1) / 2) & ~mask;              // the type's value nearest to d m
    const float e = __fmaf_rn(-m, d, __int_as_float(g));     // its side, exactly
    const bool near = abs(g - b) <= 24;
    // on the border: the even code, which is the lower one at mantissas 1 and 5/4, the upper at 3/2 and 7/4
    const bool above = e > 0.0f || (e == 0.0f && (lane & 2));
    const uint32_t up = __ballot_sync(0xffffffffu, near && above);
    const uint32_t down = __ballot_sync(0xffffffffu, near && !above);
    const int sh = lane & 28;
    const bool u = (up >> sh & 15u) != 0u, w = (down >> sh & 15u) != 0u;
    const int move = u && w ? -8 : u ? 7 : w ? -7 : 0;
    return make_uint2(__reduce_or_sync(0xffffffffu, ((uint32_t)move & 15u) << sh), up);
}

// The tensor's constants but for `moves` and `ups`, which 16-bit values with a tensor scale need too.
__device__ __forceinline__ Fp4Tensor fp4_tensor(const float* tensor_scale) {
    Fp4Tensor p;
    p.t = tensor_scale ? __ldg(tensor_scale) : 1.0f;
    p.t_ok = p.t > 0.0f && p.t <= 3.40282347e38f;
    p.t_mid = p.t >= 0x1p-50f && p.t <= 0x1p50f;
    p.c = __fmul_rn(6.0f, p.t);
    p.up = p.c < 0x1p-60f ? 0x1p64f : p.c > 0x1p60f ? 0x1p-64f : 1.0f;
    p.c = __fmul_rn(p.c, p.up);
    if (p.c > 3.40282347e38f) {   // fl(6 t) overflowed: every quotient is zero
        p.up = 0.0f;
        p.c = 1.0f;
    }
    p.rc = reciprocal(p.c);
    p.moves = p.ups = 0u;
    return p;
}

// The E4M3 byte of amax / fl(6 t), rounded from the exact quotient: the quotient rounded by its
// residual, then to odd where it has so few bits that it may lie on a border.  Where amax was scaled
// down into the subnormal range, or is there, the quotient is below 2^-11 and rounds to zero whatever
// its last bits say; where it overflows (to a NaN, here), it saturates.
__device__ __forceinline__ uint32_t nv_scale_byte(float amax, const Fp4Tensor& p) {
    const float a = __fmul_rn(amax, p.up);
    const float q0 = __fmul_rn(a, p.rc);
    float q = fminf(__fmaf_rn(__fmaf_rn(-q0, p.c, a), p.rc, q0), 1024.0f);
    if ((__float_as_uint(q) & 0x7FFFFu) == 0u) q = odd_from_rn(q, a, p.c);
    return e4m3_byte(q);
}

// One block's scale: its byte, the factor or divisor of its elements, and how they are divided.
struct Fp4Scale {
    uint32_t byte;
    float d, r;      // NV: x / d, r its reciprocal; MX: x * r
    // 0: x * r; 1: the rounded quotient, or, for 16-bit values under a tensor scale, r and r + 16 steps
    // by border; 2: by comparison; 3: every code is zero
    int mode;
    uint32_t ups;    // mode 1 of the second kind: bit j: borders of mantissa 1 + j / 4 take the larger
};

// The scale of a block of type T's values, from its absmax as the bits of an fp32 number (above
// infinity's for a NaN).  HAS_T: a tensor scale other than one may be given.
//
// MX: byte = max(exponent field - 2, 0); x 2^-(byte - 127) is exact, so the conversion's rounding
//     is the only one.
// NV: s = e4m3(amax / c), d = fl(s t), code = e2m1(x / d).  With d = s, of four bits, the quotient is
//     rounded correctly (reciprocal, one residual, one correction: see RowDivisor): off a border it
//     is at least 2^-24 of it away, so its rounding never moves it onto one.  d = fl(s t) has 24
//     bits.  There 16-bit values take x * (1 / d), moved where a border falls on or next to one of them
//     (see fp4_moves); fp32 values the rounded quotient, and, in a block where one lies on a multiple of
//     1/4, as every border does, the quotient rounded to odd.
template <typename T, bool NV, bool HAS_T>
__device__ __forceinline__ Fp4Scale fp4_scale(uint32_t amax_bits, const Fp4Tensor& p) {
    constexpr int GRID = GridBits<T>::value;
    Fp4Scale b;
    b.ups = 0u;
    if (!NV) {
        b.byte = (uint32_t)max((int)(amax_bits >> 23) - 2, 0);
        b.r = __uint_as_float((254u - b.byte) << 23);   // 2^(127 - byte): exponent field 2 to 254
        b.d = 0.0f;
        b.mode = 0;
        if (amax_bits >= 0x7F800000u) {
            b.byte = 0xFFu;
            b.mode = 3;
        }
        return b;
    }
    const float amax = __uint_as_float(amax_bits);
    b.byte = nv_scale_byte(amax, p);
    const float s = e4m3_value(b.byte);
    b.d = HAS_T ? __fmul_rn(s, p.t) : s;
    b.r = reciprocal(b.d);
    b.mode = 1;
    if (HAS_T && GRID > 0) {
        const uint32_t i4 = __float_as_uint(s) >> 18 & 28u;
        const int move = (int)(p.moves << (i4 ^ 28u)) >> 28;
        b.r = __int_as_float(__float_as_int(b.r) + move);
        b.mode = move == -8 ? 1 : 0;
        b.ups = p.ups >> i4;
    }
    // the rounded quotient of a block that its scale saturates might overflow
    if (b.byte >= 0x7Eu && amax > 16.0f * b.d) b.mode = 2;
    if (HAS_T && !p.t_mid) b.mode = 2;
    if (b.d == 0.0f) b.mode = 3;
    if (amax_bits >= 0x7F800000u || (HAS_T && !p.t_ok)) {
        b.byte = 0x7Fu;
        b.mode = 3;
    }
    return b;
}

__device__ __forceinline__ float absmin3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// Sixteen values of a block -> sixteen codes.
template <typename T, bool NV, bool HAS_T>
__device__ __forceinline__ void fp4_codes(const float (&x)[16], const Fp4Scale& b, uint32_t (&codes)[2]) {
    constexpr bool MUL = !NV || (HAS_T && GridBits<T>::value > 0);   // mode 0 is the usual one
    if (MUL) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 q = f2_unpack(mul2s_rn(f2_pack(x[8 * h + i], x[8 * h + i + 1]), b.r));
                v[i] = q.x;
                v[i + 1] = q.y;
            }
            codes[h] = fp4_pack8(v);
        }
        if (b.mode == 0) return;
    }
    if (b.mode == 3) {
        codes[0] = codes[1] = 0u;
        return;
    }
    if (!NV) return;
    if (MUL && b.mode == 1) {
        // The codes are those of the smaller reciprocal; the larger one's differ where a value is next to
        // a border, the one above code n: mantissa 1 at n = 0, 3/2 at 1, 5/4 at 2, 4, 6 and 7/4 at 3, 5.
        constexpr uint32_t ONES = 0x11111111u;
        const float r = __int_as_float(__float_as_int(b.r) + 16);
        const uint32_t u0 = 0u - (b.ups & 1u), u1 = 0u - (b.ups >> 1 & 1u), u2 = 0u - (b.ups >> 2 & 1u),
                       u3 = 0u - (b.ups >> 3 & 1u);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 q = f2_unpack(mul2s_rn(f2_pack(x[8 * h + i], x[8 * h + i + 1]), r));
                v[i] = q.x;
                v[i + 1] = q.y;
            }
            const uint32_t lo = codes[h], hi = fp4_pack8(v), high = lo >> 1 | lo >> 2;   // bit 0: n > 1
            const uint32_t even = (u1 & high) | (u0 & ~high), odd = (u3 & high) | (u2 & ~high);
            const uint32_t take = (((odd & lo) | (even & ~lo)) & ONES) * 15u;
            codes[h] = (hi & take) | (lo & ~take);
        }
        return;
    }
    if (b.mode == 1) {
        const unsigned long long r2 = f2_pack(b.r, b.r), nd2 = f2_pack(-b.d, -b.d);
        // A quotient on a border may have been rounded there.  All borders are multiples of 1/4:
        // adding and taking away 1.5 * 2^21 rounds to those, and what changes nothing is one: a border, but
        // also zero and the codes' own values, whose blocks take the slow way for nothing (4096 x 16384 fp32
        // under a tensor scale: 49 us without, 66 with one value in a hundred zero).
        const unsigned long long big = f2_pack(0x1.8p21f, 0x1.8p21f);
        float least = 1.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const unsigned long long a = f2_pack(x[8 * h + i], x[8 * h + i + 1]);
                const unsigned long long q0 = mul2s_rn(a, b.r);
                const unsigned long long q2 = fma2_rn(fma2_rn(q0, nd2, a), r2, q0);
                const float2 q = f2_unpack(q2);
                v[i] = q.x;
                v[i + 1] = q.y;
                if (HAS_T) {
                    const float2 off = f2_unpack(sub2_rn(q2, sub2_rn(add2_rn(q2, big), big)));
                    least = absmin3(least, off.x, off.y);
                }
            }
            codes[h] = fp4_pack8(v);
        }
        const bool risky = least == 0.0f;
        if (!HAS_T || !risky) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = fabsf(x[8 * h + i]), q0 = __fmul_rn(a, b.r);
                const float q = __fmaf_rn(__fmaf_rn(-q0, b.d, a), b.r, q0);
                v[i] = copysignf(odd_from_rn(q, a, b.d), x[8 * h + i]);
            }
            codes[h] = fp4_pack8(v);
        }
        return;
    }
    codes[0] = codes[1] = 0u;
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
        float v = x[0];   // x[i] without a local-memory array
#pragma unroll
        for (int j = 1; j < 16; ++j) v = i == j ? x[j] : v;
        const uint32_t n = fp4_code_exact(v, b.d) << (4 * (i & 7));
        if (i < 8) codes[0] |= n;
        else codes[1] |= n;
    }
}

// max(|a|, |b|, |c|), NaN where one is NaN.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
    return r;
}

// Bits of the largest |x| of sixteen, as an fp32 number's; NaN gives bits above infinity's.
__device__ __forceinline__ uint32_t absmax16(const float (&x)[16]) {
    float m = absmax3(x[0], x[1], x[2]);
#pragma unroll
    for (int i = 3; i < 15; i += 2) m = absmax3(m, x[i], x[i + 1]);
    return __float_as_uint(absmax3(m, x[15], 0.0f));
}

}  // namespace ck

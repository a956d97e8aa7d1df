// The rows of a KV cache held in 4 or 8 bits.
//
// A row (one token, one KV head, one plane) is the codes of head_dim values, then a scale byte for each
// group of 16 dims. The scale's byte u is the fp16 number with the bits u << 7: five bits of exponent
// and three of mantissa, no sign, from 2^-17 on; 255 (a NaN) marks a group that held an infinity or a NaN.
// FMT 0, 4 bits: a code is a sign bit and e2m1's magnitude 0, .5, 1, 1.5, 2, 3, 4, 6; the even dim in the low
// half of a byte. FMT 1, 8 bits: an integer of [-127, 127].
//
// A value is code * scale. Its significand has at most 2 + 4 (e2m1) or 7 + 4 (int8) bits and its scale
// is bounded so that it stays below 65504: every value is an fp16 number, exactly, and a single fp16
// multiplication makes it. An integer is chosen for the 8 bits because e4m3's smallest numbers times the
// smallest scales are no fp16 numbers.
//
// The e2m1 scale is amax / 6 rounded to nearest: from scales of 2^-14 on (amax 6 * 2^-14) the largest value is clipped by 6 % at most,
// less than half of the step (a third) that it sits in, and the other values gain. Below, scales are multiples of 2^-17, and the clip is up to
// 6 * 2^-18 (a third of amax 9 * 2^-17); a group up to 6 * 2^-18 is zeros. int8's is rounded up: its steps at amax are 16 times finer
// than such a clip.
//
// A border between codes is a multiple of the scale with at most 7 (e2m1) or 12 (int8) bits, so it is an fp32 number, and the
// correctly rounded quotient of a value and its scale lies on the same side of it: the bytes follow from the inputs exactly,
// for every dtype.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace sra {
namespace kvq {

constexpr int kGroup = 16;  // dims that share a scale

__host__ __device__ constexpr int code_bytes(int fmt, int head_dim) { return fmt == KV_E2M1 ? head_dim / 2 : head_dim; }
__host__ __device__ constexpr int row_bytes(int fmt, int head_dim) { return code_bytes(fmt, head_dim) + head_dim / kGroup; }

constexpr uint32_t kScaleNaN = 255;

__device__ __forceinline__ float scale_value(uint32_t code) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(code << 7)));
}

// The scale byte of a group whose largest magnitude is amax (finite). The first guess comes from a product
// that is 2^-23 off, the scales lie 2^-4 apart, so it is the floor of the quotient or, next to a scale, its
// neighbour; comparisons with exact multiples of scales decide.
template <int FMT>
__device__ __forceinline__ uint32_t scale_code(float amax) {
    if constexpr (FMT == KV_E2M1) {
        constexpr uint32_t kMax = 226;  // 10240: 6 * 10240 is below 65504, 6 * 11264 is not
        const float t = fminf(amax * (1.0f / 6.0f), 10240.0f);
        uint32_t c = __half_as_ushort(__float2half_rz(t)) >> 7;
        const float mid6 = 3.0f * (scale_value(c) + scale_value(c + 1));
        if (amax > mid6 || (amax == mid6 && (c & 1u))) ++c;
        return c < kMax ? c : kMax;
    } else {
        constexpr uint32_t kMax = 192;  // 512: 127 * 512 is below 65504, 127 * 576 is not
        const float t = fminf(amax * (1.0f / 127.0f), 512.0f);
        uint32_t c = __half_as_ushort(__float2half_rz(t)) >> 7;
        if (127.0f * scale_value(c) < amax) ++c;
        if (127.0f * scale_value(c) < amax) ++c;
        return c < kMax ? c : kMax;
    }
}

// x / s, correctly rounded, with inv the correctly rounded 1 / s: the remainder of x * inv is exact, and adding it once gives the quotient
// (Markstein's theorem; s is at least 2^-17, and what underflows is far below the first border).
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}

// N values of one group as codes in 32-bit words (8 or 4 codes each); `code` is the group's scale byte. A group
// whose scale is 0 or NaN has codes of 0. The quotient decides as x itself would: where x is a border times the scale it is the border, and
// an x one place further is off by more than 2^-24 of it, half a place of a border or more, so its quotient lies beyond.
template <int FMT, int N>
__device__ __forceinline__ void encode(const float (&x)[N], uint32_t code, uint32_t* w) {
    const float s = scale_value(code), inv = 1.0f / s;
    const bool live = code != 0 && code != kScaleNaN;
    if constexpr (FMT == KV_E2M1) {
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
            float q[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) q[k] = copysignf(quotient(x[8 * j + k], s, inv), x[8 * j + k]);  // (-0 has lost its sign)
            uint32_t v;  // to nearest, ties to the even code, saturating
            asm("{.reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3; "
                "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d};}"
                : "=r"(v)
                : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
            w[j] = live ? v : 0u;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
            uint32_t n[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float q = fminf(fmaxf(quotient(x[4 * j + k], s, inv), -127.0f), 127.0f);
                n[k] = __float_as_uint(q + 12582912.0f);  // 1.5 * 2^23: rounds to an integer, ties to even, in the low bits
            }
            const uint32_t v = __byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410);
            w[j] = live ? v : 0u;
        }
    }
}

// Byte `i` of a word of e2m1 codes as two fp16 numbers (the low half of the byte in the low half of the result).
template <int I>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w) {
    uint32_t r;
    if constexpr (I == 0)
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(r) : "r"(w));
    else if constexpr (I == 1)
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(r) : "r"(w));
    else if constexpr (I == 2)
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(r) : "r"(w));
    else
        asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two bytes of integers (bytes LO and HI of w, sign bits already flipped: w ^ 0x80808080) as fp16 numbers: 0x64 above
// a byte is 1024 + byte, exactly.
template <int LO, int HI>
__device__ __forceinline__ uint32_t int8_pair(uint32_t flipped) {
    return sub2(__byte_perm(flipped, 0x64646464u, LO | 4 << 4 | HI << 8 | 4 << 12), 0x64806480u);  // - 1152
}
// A scale byte as fp16 in both halves.
__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) { return byte * 0x00800080u; }

// Eight codes (1 or 2 words) times their scale as four pairs of fp16 numbers, in the order of the dims.
template <int FMT>
__device__ __forceinline__ void decode8(const uint32_t* w, uint32_t scale2, uint32_t (&out)[4]) {
    if constexpr (FMT == KV_E2M1) {
        out[0] = mul2(e2m1_pair<0>(w[0]), scale2);
        out[1] = mul2(e2m1_pair<1>(w[0]), scale2);
        out[2] = mul2(e2m1_pair<2>(w[0]), scale2);
        out[3] = mul2(e2m1_pair<3>(w[0]), scale2);
    } else {
        const uint32_t a = w[0] ^ 0x80808080u, b = w[1] ^ 0x80808080u;
        out[0] = mul2(int8_pair<0, 1>(a), scale2);
        out[1] = mul2(int8_pair<2, 3>(a), scale2);
        out[2] = mul2(int8_pair<0, 1>(b), scale2);
        out[3] = mul2(int8_pair<2, 3>(b), scale2);
    }
}

}  // namespace kvq
}  // namespace sra

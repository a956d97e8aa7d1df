// Decode attention over a KV cache held in 4 or 8 bits (format: kv_format.cuh).
//
//   o = sum_t softmax_t(scale * q . K_t) V_t over a request's tokens, K_t and V_t the values that the cache holds.
//
// A CTA takes a (request, kv head) pair, or a part of it, 32 tokens (a tile) a warp at a time. A head's rows of a page lie in a row,
// so a tile is one to four bulk copies for K and as many for V into the warp's own ring in shared memory, where it alone reads
// them: warps wait for nobody. (The same rings filled by the lanes, 16 bytes a cp.async: batch 64 x 16384 72.0 -> 75.7 us, in 8 bits
// 101 -> 118. A ring that warps of their own fill for twelve that compute: 94; these could not keep up.)
//
// Codes become fp16 in registers, in the layout of the matrix instruction's operand: a value times its scale is an fp16
// number exactly, so this is one conversion (or byte permutation) and one multiplication for two values, and nothing is
// rounded. The products have the tokens (S^T = K Q^T) or the dims (O^T = V^T P^T) as their 16 rows and the up to eight
// query heads as their eight columns. V's operand holds two tokens' values of a dim side by side: for e2m1 the
// nibbles of two tokens are merged first (four bitwise operations for 16 values) and one conversion then makes the pair.
// Which dims and tokens a lane takes is free, as long as both sides of a product agree: a lane's K is one scale group of
// 16 dims in a row, its V a run of head_dim / 8 dims of four tokens in a row.
//
// q is fp16, or bf16 / fp32 times a power of two that takes its row's largest element to [2^14, 2^15) (elements below 2^-39
// of it are lost); fp32 goes in as two fp16 numbers, which hold 23 of its 24 bits (2^-23 of an element off at most: what is left
// of it behind the first is up to 2^12 units of its last place, the second holds even ones from 2^11 on). Probabilities are fp16
// at 2^14 times their size relative to the running maximum (normal numbers down to 2^-28 of the largest), rounded once, 2^-11 of
// each; two fp16 numbers for fp32. Sums, maxima and outputs are fp32; for fp32 each tile's products are added to them by ordinary
// additions, because the matrix instruction's own accumulation truncates.
//
// Without a workspace the splits of a pair are the CTAs of a cluster, which merge through distributed shared memory; with one the
// batch may be a stream of tiles cut into equal parts (stream_kernel), whose records a second kernel merges.
//
// What bounds it: the issue of instructions, a little before HBM. A tile of head_dim 128 in 4 bits is some 600 instructions a warp: 128
// conversions and 128 multiplications (two cycles each, on different pipes), 32 products, each of which holds the scheduler's dispatch
// for some six cycles (measured: a product with four conversions and four multiplications takes 14 cycles, not nine), the softmax, the
// copies. A scheduler takes 0.48 us for a tile with four warps (0.64 with two; registers and rings leave room for four), where HBM's
// copy rate would give it one in 0.41: long streams run at 5.9 TB/s. A call's start, its changes of pair and the merge come to some 20 us:
// batch 256 x 16384 of 2 heads (from 4000 tokens on, 755 MB) 157 us, 112 at the copy rate. 8 bits have half the instructions for a
// byte: 16 x 32768 of 8 heads 188 us, 169 at the copy rate. Other forms: 32 x 32768 of one head of 256 74 us (45) in 4 bits, 110 (84) in 8,
// where an SM has one CTA; 24 x 8192 of 4 heads of 128, fp32, 45 (17) and 52 (32); 64 x 8192 of 4 heads of 64 52 (22) and 62 (42).
// Measured and left: the next tile's scores beside a tile's values (64 x 16384 72 -> 75 us), a third CTA an SM in 80 registers (81), tiles of 64
// tokens (73.5), a running maximum that follows only a score of twice its weight (157.7 -> 157.3).
#pragma once

#include <cooperative_groups.h>

#include "kv_format.cuh"
#include "tma.cuh"

namespace cg = cooperative_groups;

namespace sra {
namespace qattn {

constexpr int kTile = 32;       // tokens of a warp's tile
constexpr int kHalves = 2;      // of 16 tokens
constexpr float kUnder = 14;    // the probabilities' base lies 2^14 under the maximum

// F32: fp32 queries (in two parts, and probabilities in two); otherwise bf16 or fp16 (QuantAttnArgs::bf16).
template <bool F32, int FMT, int HD, int BS>
struct Shape {
    static constexpr int R = kvq::row_bytes(FMT, HD), CODES = kvq::code_bytes(FMT, HD);
    static constexpr int KS = HD / 16;  // steps of 16 dims
    static constexpr int QP = F32 ? 2 : 1, PP = F32 ? 2 : 1;
    // q's fragments in shared memory, one copy for the CTA: where the registers do not hold them
    static constexpr bool Q_SHARED = F32 || HD == 256;
    static constexpr int Q_BYTES = Q_SHARED ? QP * KS * 32 * 8 : 0;
    static constexpr int PAGES = kTile / BS;        // of a tile
    static constexpr int STAGE = 2 * kTile * R;     // bytes of a stage: K rows, V rows
    static constexpr int WARPS = quant_attn_warps(FMT, HD);
    static constexpr int CTAS = quant_attn_ctas(FMT, HD);  // per SM
    static constexpr int FIT = (233472 / CTAS - 1024 - 512 - Q_BYTES) / (WARPS * STAGE);
    static constexpr int STAGES = FIT > 4 ? 4 : FIT;
    static_assert(STAGES >= 2, "a tile under way beside the one at work");
    // shared memory: rings, q's fragments and their factors, the stages' barriers and masks
    static constexpr int ring = WARPS * STAGES * STAGE;
    static constexpr int q_at = ring;
    static constexpr int factor_at = q_at + Q_BYTES;
    static constexpr int bar_at = factor_at + 8 * 4;
    static constexpr int mask_at = bar_at + WARPS * STAGES * 8;
    static constexpr int total = (mask_at + WARPS * STAGES * 4 + 15) / 16 * 16;
    // the merge, over the drained rings: the warps' partial outputs and statistics, then the CTA's result
    static constexpr int HS = HD + 4;  // floats between heads
    static constexpr int part_ml = WARPS * 8 * HS * 4;
    static constexpr int res_ml = part_ml + WARPS * 16 * 4;
    static constexpr int res_o = res_ml + 16 * 4;
    static_assert(res_o + 8 * HD * 4 <= ring, "the merge fits over the rings");
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v) {
    __half2 h;
    memcpy(&h, &v, 4);
    return __half22float2(h);
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {  // an 8 x 8 matrix of 16-bit values, a row's pairs over four lanes
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// N words from shared memory at a multiple of ALIGN bytes.
template <int N, int ALIGN>
__device__ __forceinline__ void words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (ALIGN % 8 == 0 && N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * i);
            w[i] = v.x, w[i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
    }
}
// Byte i (a constant once unrolled) of e2m1 codes, or bytes 2 (i & 1) and 2 (i & 1) + 1 of flipped integers, as two fp16 numbers.
__device__ __forceinline__ uint32_t e2m1_byte(uint32_t w, int i) {
    return i == 0 ? kvq::e2m1_pair<0>(w) : i == 1 ? kvq::e2m1_pair<1>(w) : i == 2 ? kvq::e2m1_pair<2>(w) : kvq::e2m1_pair<3>(w);
}
__device__ __forceinline__ uint32_t int8_half(uint32_t w, int i) { return i == 0 ? kvq::int8_pair<0, 1>(w) : kvq::int8_pair<2, 3>(w); }

__device__ __forceinline__ float from_16(uint32_t bits, bool bf16) {
    return bf16 ? __uint_as_float(bits << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
// Element i of an output row.
template <bool F32>
__device__ __forceinline__ void put(void* out, int64_t i, float v, bool bf16) {
    if constexpr (F32) static_cast<float*>(out)[i] = v;
    else static_cast<unsigned short*>(out)[i] = bf16 ? Elem<__nv_bfloat16>::to_bits16(v) : Elem<__half>::to_bits16(v);
}

// Q as B fragments: step e = 4 j + i holds dims 64 j + 16 ft + 4 i + {0, 1} (b0) and {2, 3} (b1) of head fg.
template <typename S, bool F32, int HD>
struct Query {
    static constexpr int KS = S::KS, QP = S::QP;
    uint32_t reg[S::Q_SHARED ? 1 : KS][2];
    const uint2* shared;
    float factor[2];  // of the scores of heads 2 ft and 2 ft + 1: the softmax scale's size in base 2 and q's power of two

    // Every warp loads it into its registers or, where it is kept in shared memory, warp 0 into that, and the CTA's warps meet.
    // row: the pair's first element in q.
    __device__ __forceinline__ void load(const QuantAttnArgs& a, int64_t row, unsigned char* smem, int warp, int lane) {
        const int fg = lane >> 2, ft = lane & 3;
        uint2* keep = reinterpret_cast<uint2*>(smem + S::q_at) + lane;
        float* factors = reinterpret_cast<float*>(smem + S::factor_at);
        shared = keep;
        if (!S::Q_SHARED || warp == 0) {
            float x[HD / 4];
#pragma unroll
            for (int j = 0; j < HD / 64; ++j) {
                const int64_t at = row + static_cast<int64_t>(fg) * HD + 64 * j + 16 * ft;
                if (fg >= a.group) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[16 * j + k] = 0.0f;
                } else if constexpr (F32) {
                    const float* p = static_cast<const float*>(a.q) + at;
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        if (a.wide_q) {
                            const float4 v = *reinterpret_cast<const float4*>(p + k);
                            x[16 * j + k] = v.x, x[16 * j + k + 1] = v.y, x[16 * j + k + 2] = v.z, x[16 * j + k + 3] = v.w;
                        } else {
#pragma unroll
                            for (int c = 0; c < 4; ++c) x[16 * j + k + c] = p[k + c];
                        }
                    }
                } else {
                    const unsigned short* p = static_cast<const unsigned short*>(a.q) + at;
#pragma unroll
                    for (int k = 0; k < 16; k += 8) {
                        if (a.wide_q) {
                            const uint4 v = *reinterpret_cast<const uint4*>(p + k);
#pragma unroll
                            for (int c = 0; c < 8; ++c) x[16 * j + k + c] = from_16((word(v, c / 2) >> (16 * (c & 1))) & 0xffffu, a.bf16);
                        } else {
#pragma unroll
                            for (int c = 0; c < 8; ++c) x[16 * j + k + c] = from_16(p[k + c], a.bf16);
                        }
                    }
                }
            }
            if (a.scale_log2 < 0.0f) {  // the sign goes to q: the scores' factor is not negative
#pragma unroll
                for (int k = 0; k < HD / 4; ++k) x[k] = -x[k];
            }
            float back = 1.0f;
            if (F32 || a.bf16) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < HD / 4; ++k) {
                    const float v = fabsf(x[k]);
                    top = v < INFINITY ? fmaxf(top, v) : top;
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;  // -127: 0 or subnormal
                const int up = top == 0.0f ? 0 : min(14 - e, 126);
                const float to = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                back = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
                for (int k = 0; k < HD / 4; ++k) x[k] *= to;
            }
#pragma unroll
            for (int part = 0; part < QP; ++part)
#pragma unroll
                for (int e = 0; e < KS; ++e) {
                    float* y = x + 4 * e;
                    const uint32_t b0 = pack_h2(y[0], y[1]), b1 = pack_h2(y[2], y[3]);
                    if constexpr (S::Q_SHARED) keep[(part * KS + e) * 32] = make_uint2(b0, b1);
                    else reg[e][0] = b0, reg[e][1] = b1;
                    if constexpr (QP > 1) {  // what is left (nothing of infinities and NaN)
                        const float2 f0 = unpack_h2(b0), f1 = unpack_h2(b1);
                        const float f[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
                        for (int k = 0; k < 4; ++k) y[k] = fabsf(f[k]) < INFINITY ? y[k] - f[k] : 0.0f;
                    }
                }
            const float f = back * fabsf(a.scale_log2);
            if constexpr (S::Q_SHARED) {
                if (ft == 0) factors[fg] = f;
            } else {
                factor[0] = __shfl_sync(0xffffffffu, f, 8 * ft);
                factor[1] = __shfl_sync(0xffffffffu, f, 8 * ft + 4);
            }
        }
        if constexpr (S::Q_SHARED) {
            __syncthreads();
            factor[0] = factors[2 * ft], factor[1] = factors[2 * ft + 1];
        }
    }
    __device__ __forceinline__ uint2 get(int part, int e) const {
        if constexpr (S::Q_SHARED) return shared[(part * KS + e) * 32];
        else return make_uint2(reg[e][0], reg[e][1]);
    }
};

// S^T of a tile: lane (fg, ft) gets the scores of tokens 16 u + 4 (fg / 2) + fg % 2 (k < 2) and those two further (k >= 2) for heads
// 2 ft + k % 2 in s[u][k].
template <typename S, bool F32, int FMT, int HD>
__device__ __forceinline__ void scores(const uint8_t* kt, const Query<S, F32, HD>& q, float (&s)[kHalves][4], int lane) {
    constexpr int WORDS = FMT == KV_E2M1 ? 2 : 4;  // words of a group of 16 codes
    const int fg = lane >> 2, ft = lane & 3;
    const uint8_t* r0 = kt + (4 * (fg >> 1) + (fg & 1)) * S::R;
    // fp32: the products with the lower part of q; otherwise those of every other step, so that four chains of products
    // are under way instead of two
    float fine[kHalves][4];
#pragma unroll
    for (int u = 0; u < kHalves; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[u][k] = fine[u][k] = 0.0f;
#pragma unroll
    for (int j = 0; j < HD / 64; ++j) {
        uint32_t w[kHalves][2][WORDS], sc[kHalves][2];
#pragma unroll
        for (int u = 0; u < kHalves; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* r = r0 + (16 * u + 2 * h) * S::R;
                words<WORDS, S::R>(r + (ft + 4 * j) * WORDS * 4, w[u][h]);
                sc[u][h] = kvq::scale_pair(r[S::CODES + ft + 4 * j]);
                if constexpr (FMT == KV_INT8) {
#pragma unroll
                    for (int i = 0; i < WORDS; ++i) w[u][h][i] ^= 0x80808080u;
                }
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 b = q.get(0, 4 * j + i);
#pragma unroll
            for (int u = 0; u < kHalves; ++u) {
                uint32_t a[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        a[h + 2 * c] = kvq::mul2(FMT == KV_E2M1 ? e2m1_byte(w[u][h][i >> 1], (2 * i + c) & 3)
                                                                : int8_half(w[u][h][i], c),
                                                 sc[u][h]);
                if constexpr (F32) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma(part, a, b.x, b.y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[u][k] += part[k];
                    const uint2 b1 = q.get(1, 4 * j + i);
                    mma(fine[u], a, b1.x, b1.y);
                } else {
                    mma(i & 1 ? fine[u] : s[u], a, b.x, b.y);
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kHalves; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[u][k] += fine[u][k];
}

// The running softmax over those scores (valid: a bit per token): maxima m of the lane's two heads, this lane's tokens' part l of
// their sums, corr = 2^(old m - new m); the probabilities, relative to 2^(m - kUnder), as l, as B fragments of the next
// product.
template <int PP>
__device__ __forceinline__ void softmax(float (&p)[kHalves][4], uint32_t valid, bool whole, const float (&factor)[2], float (&m)[2], float (&l)[2],
                                        float (&corr)[2], uint32_t (&pb)[PP][kHalves][2], int lane) {
    const unsigned FULL = 0xffffffffu;
    const int fg = lane >> 2;
#pragma unroll
    for (int u = 0; u < kHalves; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) p[u][k] *= factor[k & 1];
    if (!whole) {
#pragma unroll
        for (int u = 0; u < kHalves; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!((valid >> (16 * u + 4 * (fg >> 1) + (fg & 1) + (k & 2))) & 1u)) p[u][k] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(p[0][h], p[0][h + 2]);
#pragma unroll
        for (int u = 1; u < kHalves; ++u) mx[h] = fmaxf(mx[h], fmaxf(p[u][h], p[u][h + 2]));
    }
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        const float a = __shfl_xor_sync(FULL, mx[0], x), b = __shfl_xor_sync(FULL, mx[1], x);
        mx[0] = fmaxf(mx[0], a), mx[1] = fmaxf(mx[1], b);
    }
    float base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float now = fmaxf(m[h], mx[h]);
        // (no score above -inf yet: those weigh nothing. Rounded up: of a maximum past 2^25, whose neighbours lie 4 and more apart, the base
        // must not lie further below than 2^14, where fp16 ends)
        base[h] = now == -INFINITY ? 0.0f : __fsub_ru(now, kUnder);
        corr[h] = now == -INFINITY ? 1.0f : ex2(m[h] - now);
        m[h] = now;
    }
#pragma unroll
    for (int u = 0; u < kHalves; ++u) {
#pragma unroll
        for (int k = 0; k < 4; ++k) p[u][k] = ex2(p[u][k] - base[k & 1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t hi = pack_h2(p[u][2 * c], p[u][2 * c + 1]);
            pb[0][u][c] = transpose8(hi);
            if constexpr (PP > 1) {
                const float2 f = unpack_h2(hi);
                pb[1][u][c] = transpose8(pack_h2(p[u][2 * c] - f.x, p[u][2 * c + 1] - f.y));
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float sum = p[0][h] + p[0][h + 2];
#pragma unroll
        for (int u = 1; u < kHalves; ++u) sum += p[u][h] + p[u][h + 2];
        l[h] = fmaf(l[h], corr[h], sum);
    }
}

// O^T = O^T corr + V^T P^T: o[d] holds dim fg * HD / 8 + 2 d (k < 2) and the next one (k >= 2) of heads 2 ft + k % 2. Tokens that
// do not count get a scale of 0.
template <typename S, bool F32, int FMT, int HD>
__device__ __forceinline__ void values(const uint8_t* vt, const uint32_t (&pb)[S::PP][kHalves][2], const float (&corr)[2],
                                       uint32_t valid, bool whole, float (&o)[HD / 16][4], int lane) {
    constexpr int RUN = HD / 8;                         // dims of a lane
    constexpr int PER = FMT == KV_E2M1 ? 8 : 4;         // codes in a word
    constexpr int WORDS = RUN / PER;
    constexpr int GROUPS = RUN > kvq::kGroup ? RUN / kvq::kGroup : 1;
    const int fg = lane >> 2, ft = lane & 3;
    if (__any_sync(0xffffffffu, corr[0] != 1.0f || corr[1] != 1.0f)) {
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) o[d][0] *= corr[0], o[d][1] *= corr[1], o[d][2] *= corr[0], o[d][3] *= corr[1];
    }
#pragma unroll
    for (int u = 0; u < kHalves; ++u) {
        const uint8_t* r0 = vt + (16 * u + 4 * ft) * S::R;
        uint32_t w[4][WORDS], sc[2][GROUPS];
#pragma unroll
        for (int i = 0; i < 4; ++i) words<WORDS, S::R>(r0 + i * S::R + fg * WORDS * 4, w[i]);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int at = S::CODES + fg * RUN / kvq::kGroup + g;
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = r0[i * S::R + at];
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((valid >> (16 * u + 4 * ft + i)) & 1u)) b[i] = 0;
            }
            sc[0][g] = b[0] * 0x80u + b[1] * 0x800000u;
            sc[1][g] = b[2] * 0x80u + b[3] * 0x800000u;
        }
#pragma unroll
        for (int c = 0; c < WORDS; ++c) {
            const uint32_t* s2[2] = {&sc[0][c * PER / kvq::kGroup], &sc[1][c * PER / kvq::kGroup]};
            // pair[e][k]: tokens 2 e and 2 e + 1, the codes of dims k of this word (a byte, or a half, a pair)
            uint32_t even[2], odd[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t x = w[2 * e][c], y = w[2 * e + 1][c];
                if constexpr (FMT == KV_E2M1) {
                    even[e] = (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u);
                    odd[e] = ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u);
                } else {
                    even[e] = __byte_perm(x, y, 0x6240) ^ 0x80808080u;  // x0 y0 x2 y2
                    odd[e] = __byte_perm(x, y, 0x7351) ^ 0x80808080u;   // x1 y1 x3 y3
                }
            }
#pragma unroll
            for (int k = 0; k < PER / 2; ++k) {
                uint32_t a[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a[2 * e] = kvq::mul2(FMT == KV_E2M1 ? e2m1_byte(even[e], k) : int8_half(even[e], k), *s2[e]);
                    a[2 * e + 1] = kvq::mul2(FMT == KV_E2M1 ? e2m1_byte(odd[e], k) : int8_half(odd[e], k), *s2[e]);
                }
                const int d = c * (PER / 2) + k;
                if constexpr (F32) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma(part, a, pb[S::PP - 1][u][0], pb[S::PP - 1][u][1]);
                    mma(part, a, pb[0][u][0], pb[0][u][1]);
#pragma unroll
                    for (int n = 0; n < 4; ++n) o[d][n] += part[n];
                } else {
                    mma(o[d], a, pb[0][u][0], pb[0][u][1]);
                }
            }
        }
    }
}

// The warps' maxima, sums (of all their lanes) and outputs of one pair, merged over the drained rings: the CTA's maxima and sums (res_ml) and
// unnormalised output (res_o) in shared memory.
template <typename S, int HD>
__device__ __forceinline__ void merge_warps(unsigned char* smem, const float (&o)[HD / 16][4], const float (&m)[2], const float (&l)[2],
                                            int G, int warp, int lane) {
    constexpr int W = S::WARPS;
    const int fg = lane >> 2, ft = lane & 3;
    float* po = reinterpret_cast<float*>(smem) + warp * 8 * S::HS;
    float* ml = reinterpret_cast<float*>(smem + S::part_ml);
    if (fg == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) ml[warp * 16 + 2 * ft + h] = m[h], ml[warp * 16 + 8 + 2 * ft + h] = l[h];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float* row = po + (2 * ft + h) * S::HS + fg * (HD / 8);
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) *reinterpret_cast<float2*>(row + 2 * d) = make_float2(o[d][h], o[d][2 + h]);
    }
    __syncthreads();
    float* res = reinterpret_cast<float*>(smem + S::res_ml);
    float* ro = reinterpret_cast<float*>(smem + S::res_o);
    const float* all = reinterpret_cast<const float*>(smem);
    for (int i = threadIdx.x; i < G * HD; i += W * 32) {
        const int g = i / HD, d = i - g * HD;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, ml[w * 16 + g]);
        float sum = 0.0f, acc = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float lw = ml[w * 16 + 8 + g];
            // (a part without scores above -inf has a sum of 0, or NaN)
            const float f = ml[w * 16 + g] == -INFINITY ? 1.0f : ex2(ml[w * 16 + g] - top);
            sum = fmaf(f, lw, sum);
            acc = fmaf(f, all[w * 8 * S::HS + g * S::HS + d], acc);
        }
        ro[i] = acc;
        if (d == 0) res[g] = top, res[8 + g] = sum;
    }
}

// A bulk copy of a page's rows (16-byte aligned on both sides, a multiple of 16 bytes) that completes on `bar`.
__device__ __forceinline__ void copy_rows(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
template <typename S>
__device__ __forceinline__ void init_barriers(unsigned char* smem) {  // each warp its own
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < S::STAGES) {
        mbar_init(reinterpret_cast<uint64_t*>(smem + S::bar_at) + warp * S::STAGES + lane, 1);
        mbar_init_fence();
    }
    __syncwarp();
}

constexpr uint32_t kGaveUp = 1u << 31;  // a wait of this warp ran out: it asks for no more tiles

// The tiles first + warp, first + warp + stride, ... below `end` of a pair whose request has `len` tokens. Leaves the CTA's
// maxima and sums (res_ml) and unnormalised output (res_o) in shared memory; the CTA's warps meet before they are read.
template <typename S, bool F32, int FMT, int HD, int BS>
__device__ __forceinline__ void segment(const QuantAttnArgs& a, unsigned char* smem, int64_t b, int kvh, int len, int first, int stride,
                                        int end, uint32_t* turn) {
    constexpr int ST = S::STAGES, PAGES = S::PAGES;
    constexpr uint32_t PAGE_BYTES = BS * S::R;
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.group;
    unsigned char* ring = smem + warp * ST * S::STAGE;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + S::bar_at) + warp * ST;
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + S::mask_at) + warp * ST;
    const int64_t page_step = static_cast<int64_t>(a.n_kv) * PAGE_BYTES;
    const uint8_t* cache = static_cast<const uint8_t*>(a.cache) + static_cast<int64_t>(kvh) * PAGE_BYTES;
    const int32_t* table = a.table + b * a.max_blocks;

    // Lane k < PAGES has the entry of page k of a tile, asked for a tile ahead of the copies. (The entries of the first tiles are asked
    // for together with the request's length: whether they are in use shows when the copies are made.)
    auto entry = [&](int t) -> int32_t {
        const int64_t j = static_cast<int64_t>(t) * PAGES + lane;
        return lane < PAGES && j < a.max_blocks ? __ldcg(table + j) : -1;
    };
    auto issue = [&](int t, int32_t page, int stage) {
        const int left = len - t * kTile;  // tokens from here on
        const bool used = lane * BS < left && lane < PAGES;
        const bool ok = used && static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_blocks);
        const unsigned good = __ballot_sync(FULL, ok);
        uint32_t valid = FULL;
        if (good != FULL >> (32 - PAGES) || left < kTile) {  // the last tile of a request, or bad entries
            valid = 0;
#pragma unroll
            for (int k = 0; k < PAGES; ++k)
                if ((good >> k) & 1u) valid |= (FULL >> (32 - BS)) << (k * BS & 31);
            if (left < kTile) valid &= (1u << left) - 1u;
            if (used && !ok && kvh == 0 && a.err) atomicAdd(a.err, 1);
        }
        if (lane == 0) {
            mask[stage] = valid;
            mbar_arrive_expect_tx(bar + stage, 2 * PAGE_BYTES * __popc(good));
        }
        __syncwarp();
        if (ok) {
            const uint32_t dst = smem_u32(ring + stage * S::STAGE) + lane * PAGE_BYTES;
            const uint8_t* src = cache + page * page_step;
            copy_rows(dst, src, PAGE_BYTES, bar + stage);
            copy_rows(dst + kTile * S::R, src + a.plane_bytes, PAGE_BYTES, bar + stage);
        }
    };

    const int t0 = first + warp;
    int32_t page[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) page[s] = entry(t0 + s * stride);
    int32_t next = entry(t0 + ST * stride);
    uint32_t phase = *turn;  // parity of the stages' next phases, a bit each, and kGaveUp
    if (phase & kGaveUp) end = t0;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
        if (t0 + s * stride < end) issue(t0 + s * stride, page[s], s);
    }
    Query<S, F32, HD> q;  // comes in while the first tiles do
    q.load(a, b * a.qs + static_cast<int64_t>(kvh) * G * HD, smem, warp, lane);
    float o[HD / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.0f;
    int stage = 0;
    for (int t = t0; t < end; t += stride) {
        if (!__all_sync(FULL, mbar_wait(bar + stage, (phase >> stage) & 1u))) {  // counted; the results are void
            for (int s = 1; s < ST; ++s) {  // the other stages' copies are out as well: none may land in another CTA's memory
                const int other = (stage + s) % ST;
                if (t + s * stride < end) mbar_wait(bar + other, (phase >> other) & 1u);
            }
            phase |= kGaveUp;
            break;
        }
        phase ^= 1u << stage;
        const uint32_t valid = mask[stage];
        const bool whole = valid == FULL;
        const uint8_t* kt = ring + stage * S::STAGE;
        float s[kHalves][4], corr[2];
        uint32_t pb[S::PP][kHalves][2];
        scores<S, F32, FMT, HD>(kt, q, s, lane);
        softmax<S::PP>(s, valid, whole, q.factor, m, l, corr, pb, lane);
        values<S, F32, FMT, HD>(kt + kTile * S::R, pb, corr, valid, whole, o, lane);
        // this lane's reads of the stage come before the copies that fill it again, whichever lane issues them (without a branch for a
        // request's last tiles, which need none: 256 x 16384 155.0 us against 159.4)
        fence_proxy_async();
        __syncwarp();  // every lane is done with the stage
        const int32_t now = next;
        next = entry(t + (ST + 1) * stride);
        if (t + ST * stride < end) issue(t + ST * stride, now, stage);
        stage = stage + 1 == ST ? 0 : stage + 1;
    }
    *turn = phase;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        l[0] += __shfl_xor_sync(FULL, l[0], x);
        l[1] += __shfl_xor_sync(FULL, l[1], x);
    }
    __syncthreads();  // all rings are drained
    merge_warps<S, HD>(smem, o, m, l, G, warp, lane);
}

__device__ __forceinline__ int tokens_of(const QuantAttnArgs& a, int64_t b) {
    const int64_t n = __ldcg(a.seq_lens + b), cap = a.max_blocks * a.block_size;
    return static_cast<int>(n < 0 ? 0 : (n > cap ? cap : n));
}

template <bool F32, int FMT, int HD, int BS>
__global__ void __launch_bounds__(Shape<F32, FMT, HD, BS>::WARPS * 32, Shape<F32, FMT, HD, BS>::CTAS) cluster_kernel(QuantAttnArgs a) {
    using S = Shape<F32, FMT, HD, BS>;
    extern __shared__ __align__(128) unsigned char smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int splits = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t pair = blockIdx.x / splits, b = pair / a.n_kv;
    const int kvh = static_cast<int>(pair - b * a.n_kv), G = a.group;
    init_barriers<S>(smem);
    pdl_enter();
    const int len = tokens_of(a, b);
    uint32_t turn = 0;
    if (kvh == 0 && rank == 0 && threadIdx.x == 0 && a.err && a.seq_lens[b] != len) atomicAdd(a.err, 1);
    segment<S, F32, FMT, HD, BS>(a, smem, b, kvh, len, rank * S::WARPS, splits * S::WARPS, (len + kTile - 1) / kTile, &turn);
    const int64_t out = b * a.os + static_cast<int64_t>(kvh) * G * HD;
    const float* res = reinterpret_cast<const float*>(smem + S::res_ml);
    if (splits == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < G * HD; i += S::WARPS * 32) {
            const float l = res[8 + i / HD];
            put<F32>(a.out, out + i, l != 0.0f ? res[16 + i] / l : 0.0f, a.bf16);
        }
        return;
    }
    cluster.sync();
    const int slice = (G * HD + splits - 1) / splits, i0 = rank * slice, i1 = min(i0 + slice, G * HD);
    for (int i = i0 + threadIdx.x; i < i1; i += S::WARPS * 32) {
        const int g = i / HD;
        float top = -INFINITY, sum = 0.0f, acc = 0.0f;
        for (int r = 0; r < splits; ++r) top = fmaxf(top, cluster.map_shared_rank(res, r)[g]);
        for (int r = 0; r < splits; ++r) {
            const float* o = cluster.map_shared_rank(res, r);
            const float f = o[g] == -INFINITY ? 1.0f : ex2(o[g] - top);
            sum = fmaf(f, o[8 + g], sum);
            acc = fmaf(f, o[16 + i], acc);
        }
        put<F32>(a.out, out + i, sum != 0.0f ? acc / sum : 0.0f, a.bf16);
    }
    cluster.sync();  // nobody reads this CTA's part any more
}

// The whole batch as one stream of tiles (requests, their kv heads, their tiles), cut into equal parts for as many CTAs as
// the GPU holds. Before its tiles a pair has kStreamPair places of none, for what a CTA loses with it. A CTA writes the outputs of the
// pairs that it holds whole, and leaves a record [8 max][8 sum][8 x HD] of the one that began before its part (slot 0) and of the
// one that goes on behind it (slot 1). Every CTA sums the requests' places to find its part; CTA 0 leaves the sums for the
// merge.
template <bool F32, int FMT, int HD, int BS>
__global__ void __launch_bounds__(Shape<F32, FMT, HD, BS>::WARPS * 32, Shape<F32, FMT, HD, BS>::CTAS) stream_kernel(QuantAttnArgs a) {
    using S = Shape<F32, FMT, HD, BS>;
    constexpr int NT = S::WARPS * 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int warp_sum[S::WARPS], found[3];
    if (threadIdx.x == 0) found[0] = 0x40000000;  // (nobody: above every request)
    init_barriers<S>(smem);
    uint32_t turn = 0;
    pdl_enter();
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = static_cast<int>(a.B), G = a.group;
    auto length = [&](int b) -> int {
        return b < B ? tokens_of(a, b) : 0;
    };
    // a pair's room in the stream: its tiles, and kStreamPair for what it costs beside them
    auto tiles_of = [](int len) { return len > 0 ? (len + kTile - 1) / kTile + kStreamPair : 0; };
    // thread t sums requests [t * each, (t + 1) * each); the first one's length is kept
    const int each = (B + NT - 1) / NT, mine0 = threadIdx.x * each;
    const int len0 = length(mine0);
    auto own = [&](int k) { return k == 0 ? len0 : length(mine0 + k); };
    int mine = 0;
    for (int k = 0; k < each; ++k) mine += tiles_of(own(k));
    int inc = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int t = __shfl_up_sync(FULL, inc, x);
        if (lane >= x) inc += t;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < S::WARPS; ++w) {
        before += w < warp ? warp_sum[w] : 0;
        total += warp_sum[w];
    }
    const int at0 = before + inc - mine;  // tiles before this thread's requests
    // (tiles of all kv heads are counted in 64 bits)
    const int64_t all = static_cast<int64_t>(total) * a.n_kv;
    const int64_t part = stream_part(all, gridDim.x, S::WARPS);
    if (blockIdx.x == 0) {
        int at = at0;
        for (int k = 0; k < each; ++k) {
            if (mine0 + k < B) {
                a.ws_at[mine0 + k] = at;
                if (a.err && __ldcg(a.seq_lens + mine0 + k) != own(k)) atomicAdd(a.err, 1);
            }
            at += tiles_of(own(k));
        }
        if (threadIdx.x == 0) a.ws_at[B] = total;
    }
    int64_t g0 = blockIdx.x * part;
    const int64_t g1 = g0 + part < all ? g0 + part : all;
    if (g0 >= g1) return;
    // the request that tile g0 belongs to
    {
        int at = at0;
        for (int k = 0; k < each; ++k) {
            const int len = own(k), n = tiles_of(len);
            const int64_t lo = static_cast<int64_t>(at) * a.n_kv, hi = static_cast<int64_t>(at + n) * a.n_kv;
            if (lo <= g0 && g0 < hi) found[0] = mine0 + k, found[1] = at, found[2] = len;
            at += n;
        }
    }
    __syncthreads();
    int b = found[0];
    int64_t begin = static_cast<int64_t>(found[1]) * a.n_kv;  // the request's first tile in the stream
    const int b0 = b, first_len = found[2];
    int window = b, lens = length(b + lane);  // lane k: request window + k (asked for now; the first one's length is known)
    while (g0 < g1 && b < B) {
        if (b - window >= 32) window = b, lens = length(b + lane);
        const int len = b == b0 ? first_len : __shfl_sync(FULL, lens, b - window), n = tiles_of(len);
        if (g0 >= begin + static_cast<int64_t>(n) * a.n_kv) {
            begin += static_cast<int64_t>(n) * a.n_kv;
            ++b;
            continue;
        }
        const int kvh = static_cast<int>((g0 - begin) / n);
        const int t0 = static_cast<int>(g0 - begin - static_cast<int64_t>(kvh) * n);
        const int t1 = g1 - g0 < n - t0 ? t0 + static_cast<int>(g1 - g0) : n;
        g0 += t1 - t0;
        if (t1 <= kStreamPair) continue;  // (the pair's first tile is another CTA's)
        const int first = t0 > kStreamPair ? t0 - kStreamPair : 0, end = t1 - kStreamPair;
        segment<S, F32, FMT, HD, BS>(a, smem, b, kvh, len, first, S::WARPS, end, &turn);
        __syncthreads();
        const float* res = reinterpret_cast<const float*>(smem + S::res_ml);
        if (first == 0 && t1 == n) {
            const int64_t out = b * a.os + static_cast<int64_t>(kvh) * G * HD;
            for (int i = threadIdx.x; i < G * HD; i += NT) {
                const float l = res[8 + i / HD];
                put<F32>(a.out, out + i, l != 0.0f ? res[16 + i] / l : 0.0f, a.bf16);
            }
        } else {
            float* rec = a.ws_rec + (static_cast<int64_t>(blockIdx.x) * 2 + (first == 0 ? 1 : 0)) * (16 + 8 * HD);
            for (int i = threadIdx.x; i < 16 + G * HD; i += NT) rec[i] = res[i];
        }
        fence_proxy_async();  // the merge's accesses come before the copies that fill the rings again
        __syncthreads();
    }
}

// out of a pair whose tiles several parts share, and zeros for a request without tokens. A CTA takes 256 / LANES columns; LANES
// threads share a column's records. The sums meet in a fixed order.
template <bool F32, int HD, int LANES>
__global__ void __launch_bounds__(256) merge_kernel(QuantAttnArgs a, int ctas, int warps) {
    constexpr int COLS = 256 / LANES;
    __shared__ float s_acc[LANES][COLS], s_sum[LANES][COLS], s_top[LANES][COLS];
    pdl_enter();
    const int chunks = (a.group * HD + COLS - 1) / COLS;
    const int64_t pair = blockIdx.x / chunks, b = pair / a.n_kv;
    const int kvh = static_cast<int>(pair - b * a.n_kv);
    const int col = threadIdx.x % COLS, p = threadIdx.x / COLS;
    const int i = static_cast<int>(blockIdx.x - pair * chunks) * COLS + col, g = i / HD;
    const bool there = i < a.group * HD;
    const int at = __ldcg(a.ws_at + b), n = __ldcg(a.ws_at + b + 1) - at;
    const int64_t part = stream_part(static_cast<int64_t>(__ldcg(a.ws_at + a.B)) * a.n_kv, ctas, warps);
    const int64_t out = b * a.os + static_cast<int64_t>(kvh) * a.group * HD;
    if (n == 0) {
        if (p == 0 && there) put<F32>(a.out, out + i, 0.0f, a.bf16);
        return;
    }
    const int64_t first = static_cast<int64_t>(at) * a.n_kv + static_cast<int64_t>(kvh) * n;
    const int64_t c0 = (first + kStreamPair) / part, c1 = (first + n - 1) / part;
    if (c0 == c1) return;  // written by that part
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    if (there) {
        constexpr int MANY = 4;
        for (int64_t c = c0 + p; c <= c1; c += LANES * MANY) {
            float m[MANY], l[MANY], o[MANY];
#pragma unroll
            for (int k = 0; k < MANY; ++k) {
                const int64_t ck = c + k * LANES;
                const bool ok = ck <= c1;
                const float* rec = a.ws_rec + (ck * 2 + (ck == c0 ? 1 : 0)) * (16 + 8 * HD);
                m[k] = ok ? __ldcg(rec + g) : -INFINITY;
                l[k] = ok ? __ldcg(rec + 8 + g) : 0.0f;
                o[k] = ok ? __ldcg(rec + 16 + i) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < MANY; ++k) {
                const float now = fmaxf(top, m[k]);
                // (a record without scores above -inf has a sum of 0, or NaN)
                const float f0 = top == -INFINITY ? 1.0f : ex2(top - now), f1 = m[k] == -INFINITY ? 1.0f : ex2(m[k] - now);
                sum = sum * f0 + l[k] * f1;
                acc = acc * f0 + o[k] * f1;
                top = now;
            }
        }
    }
    if constexpr (LANES > 1) {
        s_top[p][col] = top, s_sum[p][col] = sum, s_acc[p][col] = acc;
        __syncthreads();
        if (p != 0) return;
#pragma unroll
        for (int k = 0; k < LANES; ++k) top = fmaxf(top, s_top[k][col]);
        sum = acc = 0.0f;
#pragma unroll
        for (int k = 0; k < LANES; ++k) {
            const float f = s_top[k][col] == -INFINITY ? 1.0f : ex2(s_top[k][col] - top);
            sum = fmaf(f, s_sum[k][col], sum);
            acc = fmaf(f, s_acc[k][col], acc);
        }
    }
    if (there) put<F32>(a.out, out + i, sum != 0.0f ? acc / sum : 0.0f, a.bf16);
}

// Bounded waits of this translation unit that ran out, on the current device.
static unsigned int unit_wait_timeouts() {
    unsigned int n = 0;
    if (cudaMemcpyFromSymbol(&n, g_wait_timeouts, sizeof(n)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

template <bool F32, int FMT, int HD, int BS>
cudaError_t launch_stream(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    using S = Shape<F32, FMT, HD, BS>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_smem_once(stream_kernel<F32, FMT, HD, BS>, S::total, true, &done);
    if (e != cudaSuccess) return e;
    e = launch_kernel(stream_kernel<F32, FMT, HD, BS>, dim3(static_cast<unsigned>(p.stream_ctas)), dim3(S::WARPS * 32), S::total, s, p.pdl,
                      1, a);
    if (e != cudaSuccess) return e;
    // pairs that many parts share: eight threads to a column
    const bool many = a.B * a.n_kv * 4 < p.stream_ctas;
    const int cols = many ? 32 : 256;
    const int64_t grid = a.B * a.n_kv * ((a.group * HD + cols - 1) / cols);
    return launch_kernel(many ? merge_kernel<F32, HD, 8> : merge_kernel<F32, HD, 1>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s,
                         true, 1, a, p.stream_ctas, S::WARPS);
}

template <bool F32, int FMT, int HD, int BS>
cudaError_t launch_cluster(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    using S = Shape<F32, FMT, HD, BS>;
    auto kernel = cluster_kernel<F32, FMT, HD, BS>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_smem_once(kernel, S::total, true, &done);
    if (e != cudaSuccess) return e;
    if (p.splits > 8) {
        static std::atomic<uint64_t> wide{0};
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
        if (!(wide.load(std::memory_order_acquire) & bit)) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_release);
        }
    }
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.B * a.n_kv * p.splits)), dim3(S::WARPS * 32), S::total, s, p.pdl, p.splits, a);
}

template <bool F32, int FMT, int HD>
cudaError_t launch_sized(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    switch (a.block_size) {
        case 8: return p.stream_ctas ? launch_stream<F32, FMT, HD, 8>(a, p, s) : launch_cluster<F32, FMT, HD, 8>(a, p, s);
        case 16: return p.stream_ctas ? launch_stream<F32, FMT, HD, 16>(a, p, s) : launch_cluster<F32, FMT, HD, 16>(a, p, s);
        default: return p.stream_ctas ? launch_stream<F32, FMT, HD, 32>(a, p, s) : launch_cluster<F32, FMT, HD, 32>(a, p, s);
    }
}
template <bool F32, int FMT>
cudaError_t launch_format(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    switch (p.head_dim) {
        case 64: return launch_sized<F32, FMT, 64>(a, p, s);
        case 128: return launch_sized<F32, FMT, 128>(a, p, s);
        default: return launch_sized<F32, FMT, 256>(a, p, s);
    }
}

}  // namespace qattn
}  // namespace sra

// Decode attention over a KV cache held in 4 or 8 bits (format: kv_format.cuh).
//
//   o = sum_t softmax_t(scale * q . K_t) V_t over a request's tokens, K_t and V_t the values that the cache holds.
//
// A CTA takes a (request, kv head) pair, or a split of it, 32 tokens (a tile) a warp at a time. A head's rows of a page
// lie in a row, so a tile is one to four bulk copies for K and as many for V into the warp's own ring in shared
// memory; the warp that reads a stage asks for its next tile, and waits for nobody else.
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
// of it are lost); fp32 goes in as three fp16 numbers. Probabilities are fp16 at 2^14 times their size relative to the running
// maximum (normal numbers down to 2^-28 of the largest), rounded once, 2^-11 of each; two fp16 numbers for fp32. Sums, maxima
// and outputs are fp32; for fp32 each tile's products are added to them by ordinary additions, because the matrix
// instruction's own accumulation truncates.
//
// Without a workspace the splits of a pair are the CTAs of a cluster, which merge through distributed shared memory; with one the
// batch is a stream of tiles cut into equal parts (stream_kernel), whose records a second kernel merges.
#include <cooperative_groups.h>

#include "kv_format.cuh"
#include "tma.cuh"

namespace cg = cooperative_groups;

namespace sra {
namespace qattn {

constexpr int kTile = 32;     // tokens of a warp's tile
constexpr float kUnder = 14;  // the probabilities' base lies 2^14 under the maximum

template <typename T, int FMT, int HD>
struct Shape {
    static constexpr int R = kvq::row_bytes(FMT, HD), CODES = kvq::code_bytes(FMT, HD);
    static constexpr int STAGE = 2 * kTile * R;  // bytes of a stage: K rows, V rows
    // (fp32 queries' fragments take a stage's room)
    static constexpr int STAGES = FMT == KV_E2M1 && HD == 64 ? 4 : FMT == KV_E2M1 && sizeof(T) == 4 ? 2 : 3;
    // warps per CTA and CTAs per SM: what the rings leave of an SM's shared memory
    static constexpr int WARPS = STAGE <= 4608 ? 8 : 4;
    static constexpr int CTAS = FMT == KV_INT8 && HD == 256 ? 1 : 2;
    static constexpr int KS = HD / 16;  // steps of 16 dims
};
__host__ __device__ constexpr int up16(int n) { return (n + 15) / 16 * 16; }
template <typename T> constexpr int kQParts = sizeof(T) == 4 ? 3 : 1;
template <typename T> constexpr int kPParts = sizeof(T) == 4 ? 2 : 1;
template <typename T, int HD> constexpr bool kQShared = sizeof(T) == 4 || HD == 256;  // q's fragments in shared memory

// Shared memory: rings, then q's fragments, barriers and masks. The merge runs over the drained rings: the warps'
// partial outputs [WARPS][8][HD + 4] and statistics, then the CTA's result.
template <typename T, int FMT, int HD>
struct Mem {
    using S = Shape<T, FMT, HD>;
    static constexpr int ring = S::WARPS * S::STAGES * S::STAGE;
    static constexpr int q_at = ring;
    static constexpr int factor_at = q_at + (kQShared<T, HD> ? kQParts<T> * S::KS * 32 * 8 : 0);
    static constexpr int bar_at = factor_at + 8 * 4;
    static constexpr int mask_at = bar_at + S::WARPS * S::STAGES * 8;
    static constexpr int total = up16(mask_at + S::WARPS * S::STAGES * 4);
    static constexpr int HS = HD + 4;  // floats between heads
    static constexpr int part_ml = S::WARPS * 8 * HS * 4;
    static constexpr int res_ml = part_ml + S::WARPS * 16 * 4;
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
// A bulk copy of a page's rows (16-byte aligned on both sides, a multiple of 16 bytes) that completes on `bar`.
__device__ __forceinline__ void copy_rows(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
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

// Q as B fragments: step e = 4 j + i holds dims 64 j + 16 ft + 4 i + {0, 1} (b0) and {2, 3} (b1) of head fg.
template <typename T, int HD>
struct Query {
    static constexpr int KS = HD / 16, QP = kQParts<T>;
    uint32_t reg[kQShared<T, HD> ? 1 : KS][2];
    const uint2* shared;
    float factor[2];  // of the scores of heads 2 ft and 2 ft + 1: the softmax scale in base 2 and q's power of two

    // Every warp loads it into its registers or, where it is kept in shared memory, warp 0 into that (the CTA's barrier and
    // shared_factors() follow).
    __device__ __forceinline__ void load(const T* row, bool there, bool wide, float scale_log2, uint2* keep, float* factors,
                                         int warp, int lane) {
        const int fg = lane >> 2, ft = lane & 3;
        shared = keep + lane;
        if (kQShared<T, HD> && warp != 0) return;
        float x[HD / 4];
#pragma unroll
        for (int j = 0; j < HD / 64; ++j) {
            const T* p = row + static_cast<int64_t>(fg) * HD + 64 * j + 16 * ft;
            if (!there) {
#pragma unroll
                for (int k = 0; k < 16; ++k) x[16 * j + k] = 0.0f;
            } else if (wide) {
                constexpr int V = vec16<T>();
#pragma unroll
                for (int k = 0; k < 16; k += V) {
                    float f[V];
                    Vec<T, V>::unpack(Vec<T, V>::load(p + k), f);
#pragma unroll
                    for (int c = 0; c < V; ++c) x[16 * j + k + c] = f[c];
                }
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) x[16 * j + k] = to_f32(p[k]);
            }
        }
        float back = 1.0f;
        if constexpr (!std::is_same_v<T, __half>) {
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < HD / 4; ++k) {
                const float a = fabsf(x[k]);
                top = a < INFINITY ? fmaxf(top, a) : top;
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
                if constexpr (kQShared<T, HD>) keep[(part * KS + e) * 32 + lane] = make_uint2(b0, b1);
                else reg[e][0] = b0, reg[e][1] = b1;
                if constexpr (QP > 1) {  // what is left (nothing of infinities and NaN)
                    const float2 f0 = unpack_h2(b0), f1 = unpack_h2(b1);
                    const float f[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k] = fabsf(f[k]) < INFINITY ? y[k] - f[k] : 0.0f;
                }
            }
        const float f = back * scale_log2;
        if constexpr (kQShared<T, HD>) {
            if (ft == 0) factors[fg] = f;
        } else {
            factor[0] = __shfl_sync(0xffffffffu, f, 8 * ft);
            factor[1] = __shfl_sync(0xffffffffu, f, 8 * ft + 4);
        }
    }
    __device__ __forceinline__ void shared_factors(const float* factors, int lane) {
        factor[0] = factors[2 * (lane & 3)], factor[1] = factors[2 * (lane & 3) + 1];
    }
    __device__ __forceinline__ uint2 get(int part, int e) const {
        if constexpr (kQShared<T, HD>) return shared[(part * KS + e) * 32];
        else return make_uint2(reg[e][0], reg[e][1]);
    }
};

// S^T of a tile: lane (fg, ft) gets the scores of tokens 16 u + 4 (fg / 2) + fg % 2 (k < 2) and those two further (k >= 2) for heads
// 2 ft + k % 2 in s[u][k].
template <typename T, int FMT, int HD>
__device__ __forceinline__ void scores(const uint8_t* kt, const Query<T, HD>& q, float (&s)[2][4], int lane) {
    using S = Shape<T, FMT, HD>;
    constexpr int WORDS = FMT == KV_E2M1 ? 2 : 4;  // words of a group of 16 codes
    const int fg = lane >> 2, ft = lane & 3;
    const uint8_t* r0 = kt + (4 * (fg >> 1) + (fg & 1)) * S::R;
    float fine[2][4];  // fp32: the products with the lower parts of q
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[u][k] = fine[u][k] = 0.0f;
#pragma unroll
    for (int j = 0; j < HD / 64; ++j) {
        uint32_t w[2][2][WORDS], sc[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
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
            for (int u = 0; u < 2; ++u) {
                uint32_t a[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        a[h + 2 * c] = kvq::mul2(FMT == KV_E2M1 ? e2m1_byte(w[u][h][i >> 1], (2 * i + c) & 3)
                                                                : int8_half(w[u][h][i], c),
                                                 sc[u][h]);
                if constexpr (sizeof(T) == 4) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma(part, a, b.x, b.y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[u][k] += part[k];
                    const uint2 b1 = q.get(1, 4 * j + i), b2 = q.get(2, 4 * j + i);
                    mma(fine[u], a, b1.x, b1.y);
                    mma(fine[u], a, b2.x, b2.y);
                } else {
                    mma(s[u], a, b.x, b.y);
                }
            }
        }
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[u][k] += fine[u][k];
    }
}

// The running softmax over those scores (valid: a bit per token): maxima m of the lane's two heads, this lane's tokens' part l of
// their sums, corr = 2^(old m - new m); the probabilities, relative to 2^(m - kUnder), as l, as B fragments of the next
// product.
template <int PP>
__device__ __forceinline__ void softmax(float (&p)[2][4], unsigned valid, const float (&factor)[2], float (&m)[2], float (&l)[2],
                                        float (&corr)[2], uint32_t (&pb)[PP][2][2], int lane) {
    const unsigned FULL = 0xffffffffu;
    const int fg = lane >> 2;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) p[u][k] *= factor[k & 1];
    if (valid != FULL) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (!((valid >> (16 * u + 4 * (fg >> 1) + (fg & 1) + (k & 2))) & 1u)) p[u][k] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) mx[h] = fmaxf(fmaxf(p[0][h], p[0][h + 2]), fmaxf(p[1][h], p[1][h + 2]));
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        const float a = __shfl_xor_sync(FULL, mx[0], x), b = __shfl_xor_sync(FULL, mx[1], x);
        mx[0] = fmaxf(mx[0], a), mx[1] = fmaxf(mx[1], b);
    }
    float base[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float now = fmaxf(m[h], mx[h]);
        base[h] = now == -INFINITY ? 0.0f : now - kUnder;  // (no score above -inf yet: those weigh nothing)
        corr[h] = now == -INFINITY ? 1.0f : ex2(m[h] - now);
        m[h] = now;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
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
    for (int h = 0; h < 2; ++h) l[h] = fmaf(l[h], corr[h], (p[0][h] + p[0][h + 2]) + (p[1][h] + p[1][h + 2]));
}

// O^T = O^T corr + V^T P^T: o[d] holds dim fg * HD / 8 + 2 d (k < 2) and the next one (k >= 2) of heads 2 ft + k % 2. Tokens that
// do not count get a scale of 0.
template <typename T, int FMT, int HD>
__device__ __forceinline__ void values(const uint8_t* vt, const uint32_t (&pb)[kPParts<T>][2][2], const float (&corr)[2],
                                       unsigned valid, float (&o)[HD / 16][4], int lane) {
    using S = Shape<T, FMT, HD>;
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
    for (int u = 0; u < 2; ++u) {
        const uint8_t* r0 = vt + (16 * u + 4 * ft) * S::R;
        uint32_t w[4][WORDS], sc[2][GROUPS];
#pragma unroll
        for (int i = 0; i < 4; ++i) words<WORDS, S::R>(r0 + i * S::R + fg * WORDS * 4, w[i]);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int at = S::CODES + fg * RUN / kvq::kGroup + g;
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b[i] = r0[i * S::R + at];
                if (valid != 0xffffffffu && !((valid >> (16 * u + 4 * ft + i)) & 1u)) b[i] = 0;
            }
            sc[0][g] = (b[0] | b[1] << 16) << 7;
            sc[1][g] = (b[2] | b[3] << 16) << 7;
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
                if constexpr (sizeof(T) == 4) {
                    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma(part, a, pb[kPParts<T> - 1][u][0], pb[kPParts<T> - 1][u][1]);
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

// Tiles [t0, t1) of a pair. Leaves the CTA's maxima and sums (res_ml) and unnormalised output (res_o) in shared memory.
template <typename T, int FMT, int HD>
__device__ __forceinline__ void segment(const QuantAttnArgs& a, unsigned char* smem, int64_t b, int kvh, int len, int t0, int t1,
                                        uint32_t* turn) {
    using S = Shape<T, FMT, HD>;
    using M = Mem<T, FMT, HD>;
    constexpr int W = S::WARPS, ST = S::STAGES;
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, fg = lane >> 2, ft = lane & 3;
    const int G = a.group, bs_log2 = __ffs(a.block_size) - 1, per_tile = kTile >> bs_log2;
    const uint32_t page_bytes = static_cast<uint32_t>(S::R) << bs_log2;
    unsigned char* ring = smem + warp * ST * S::STAGE;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + M::bar_at) + warp * ST;
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + M::mask_at) + warp * ST;
    const uint8_t* cache = static_cast<const uint8_t*>(a.cache) + static_cast<int64_t>(kvh) * page_bytes;
    const int64_t page_step = static_cast<int64_t>(a.n_kv) * page_bytes;
    const int32_t* table = a.table + b * a.max_blocks;
    const int pages = (len + a.block_size - 1) >> bs_log2;

    // Lane k < per_tile has the entry of page k of a tile; asked for a tile ahead of the copies.
    auto entry = [&](int t) -> int32_t {
        const int j = t * per_tile + lane;
        return t < t1 && lane < per_tile && j < pages ? __ldcg(table + j) : -1;
    };
    const unsigned all_pages = FULL >> (32 - per_tile);
    auto issue = [&](int t, int32_t page, int stage) {
        const bool ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_blocks);  // (-1 where unused)
        const unsigned good = __ballot_sync(FULL, ok);
        uint32_t count = FULL;
        if (good != all_pages || len - t * kTile < kTile) {
            count = 0;
            for (int k = 0; k < per_tile; ++k)
                if ((good >> k) & 1u) count |= (FULL >> (32 - a.block_size)) << (k << bs_log2);
            const int left = len - t * kTile;
            if (left < kTile) count &= (1u << left) - 1u;
            if (!ok && lane < per_tile && t * per_tile + lane < pages && kvh == 0 && a.err) atomicAdd(a.err, 1);
        }
        if (lane == 0) {
            mask[stage] = count;
            mbar_arrive_expect_tx(bar + stage, 2 * page_bytes * __popc(good));
        }
        __syncwarp();
        if (ok) {
            const uint32_t dst = smem_u32(ring + stage * S::STAGE) + lane * page_bytes;
            const uint8_t* src = cache + page * page_step;
            copy_rows(dst, src, page_bytes, bar + stage);
            copy_rows(dst + kTile * S::R, src + a.plane_bytes, page_bytes, bar + stage);
        }
    };

    int32_t page[ST];
#pragma unroll
    for (int s = 0; s < ST; ++s) page[s] = entry(t0 + warp + s * W);
    int32_t next = entry(t0 + warp + ST * W);
    // q's fragments come in while the first tiles do
    Query<T, HD> q;
#pragma unroll
    for (int s = 0; s < ST; ++s)
        if (t0 + warp + s * W < t1) issue(t0 + warp + s * W, page[s], s);
    {
        const T* row = static_cast<const T*>(a.q) + b * a.qs + static_cast<int64_t>(kvh) * G * HD;
        float* factors = reinterpret_cast<float*>(smem + M::factor_at);
        q.load(row, fg < G, a.wide_q, a.scale_log2, reinterpret_cast<uint2*>(smem + M::q_at), factors, warp, lane);
        if constexpr (kQShared<T, HD>) {
            __syncthreads();
            q.shared_factors(factors, lane);
        }
    }
    float o[HD / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < HD / 16; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.0f;
    int stage = 0;
    uint32_t phase = *turn;  // parity of the stages' next phases, a bit each
    for (int t = t0 + warp; t < t1; t += W) {
        mbar_wait(bar + stage, (phase >> stage) & 1u);
        phase ^= 1u << stage;
        const unsigned valid = mask[stage];
        const uint8_t* kt = ring + stage * S::STAGE;
        float s[2][4], corr[2];
        uint32_t pb[kPParts<T>][2][2];
        scores<T, FMT, HD>(kt, q, s, lane);
        softmax<kPParts<T>>(s, valid, q.factor, m, l, corr, pb, lane);
        values<T, FMT, HD>(kt + kTile * S::R, pb, corr, valid, o, lane);
        __syncwarp();  // every lane is done with the stage
        const int32_t p = next;
        next = entry(t + (ST + 1) * W);
        if (t + ST * W < t1) issue(t + ST * W, p, stage);
        stage = stage + 1 == ST ? 0 : stage + 1;
    }
    *turn = phase;
    // the warps' parts
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        l[0] += __shfl_xor_sync(FULL, l[0], x);
        l[1] += __shfl_xor_sync(FULL, l[1], x);
    }
    __syncthreads();  // all rings are drained
    float* po = reinterpret_cast<float*>(smem) + warp * 8 * M::HS;
    float* ml = reinterpret_cast<float*>(smem + M::part_ml);
    if (fg == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) ml[warp * 16 + 2 * ft + h] = m[h], ml[warp * 16 + 8 + 2 * ft + h] = l[h];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float* row = po + (2 * ft + h) * M::HS + fg * (HD / 8);
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) *reinterpret_cast<float2*>(row + 2 * d) = make_float2(o[d][h], o[d][2 + h]);
    }
    __syncthreads();
    float* res = reinterpret_cast<float*>(smem + M::res_ml);
    float* ro = reinterpret_cast<float*>(smem + M::res_o);
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
            acc = fmaf(f, all[w * 8 * M::HS + g * M::HS + d], acc);
        }
        ro[i] = acc;
        if (d == 0) res[g] = top, res[8 + g] = sum;
    }
}

template <typename T, int FMT, int HD>
__global__ void __launch_bounds__(Shape<T, FMT, HD>::WARPS * 32, Shape<T, FMT, HD>::CTAS) cluster_kernel(QuantAttnArgs a) {
    using S = Shape<T, FMT, HD>;
    using M = Mem<T, FMT, HD>;
    extern __shared__ __align__(128) unsigned char smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int splits = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t pair = blockIdx.x / splits, b = pair / a.n_kv;
    const int kvh = static_cast<int>(pair - b * a.n_kv), G = a.group;
    if (threadIdx.x < S::WARPS * S::STAGES) {
        mbar_init(reinterpret_cast<uint64_t*>(smem + M::bar_at) + threadIdx.x, 1);
        mbar_init_fence();
    }
    __syncthreads();
    pdl_enter();
    int64_t n = __ldcg(a.seq_lens + b);
    const int64_t cap = a.max_blocks * a.block_size;
    if ((n < 0 || n > cap) && kvh == 0 && rank == 0 && threadIdx.x == 0 && a.err) atomicAdd(a.err, 1);
    const int len = static_cast<int>(n < 0 ? 0 : (n > cap ? cap : n));
    const int tiles = (len + kTile - 1) / kTile, per = (tiles + splits - 1) / splits;
    const int t0 = min(rank * per, tiles), t1 = min(t0 + per, tiles);
    uint32_t turn = 0;
    segment<T, FMT, HD>(a, smem, b, kvh, len, t0, t1, &turn);
    T* out = static_cast<T*>(a.out) + b * a.os + static_cast<int64_t>(kvh) * G * HD;
    const float* res = reinterpret_cast<const float*>(smem + M::res_ml);
    const float* ro = reinterpret_cast<const float*>(smem + M::res_o);
    if (splits == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < G * HD; i += S::WARPS * 32) {
            const float l = res[8 + i / HD];
            out[i] = from_f32<T>(l != 0.0f ? ro[i] / l : 0.0f);
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
        out[i] = from_f32<T>(sum != 0.0f ? acc / sum : 0.0f);
    }
    cluster.sync();  // nobody reads this CTA's part any more
}

// The whole batch as one stream of tiles (requests, their kv heads, their tiles), cut into equal parts for as many CTAs as
// the GPU holds. A CTA writes the outputs of the pairs that it holds whole, and leaves a record [8 max][8 sum][8 x HD] of
// the one that began before its part (slot 0) and of the one that goes on behind it (slot 1). Every CTA sums the
// requests' tiles to find its part; CTA 0 leaves the sums for the merge.
template <typename T, int FMT, int HD>
__global__ void __launch_bounds__(Shape<T, FMT, HD>::WARPS * 32, Shape<T, FMT, HD>::CTAS) stream_kernel(QuantAttnArgs a) {
    using S = Shape<T, FMT, HD>;
    using M = Mem<T, FMT, HD>;
    constexpr int NT = S::WARPS * 32;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int warp_sum[S::WARPS], found[2];
    if (threadIdx.x == 0) found[0] = 0x7fffffff;
    if (threadIdx.x < S::WARPS * S::STAGES) {
        mbar_init(reinterpret_cast<uint64_t*>(smem + M::bar_at) + threadIdx.x, 1);
        mbar_init_fence();
    }
    pdl_enter();
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = static_cast<int>(a.B), G = a.group;
    const int64_t cap = a.max_blocks * a.block_size;
    auto length = [&](int b) -> int {
        if (b >= B) return 0;
        const int64_t n = __ldcg(a.seq_lens + b);
        return static_cast<int>(n < 0 ? 0 : (n > cap ? cap : n));
    };
    auto tiles_of = [](int len) { return (len + kTile - 1) / kTile; };
    // thread t sums requests [t * each, (t + 1) * each)
    const int each = (B + NT - 1) / NT, mine0 = threadIdx.x * each;
    int mine = 0;
    for (int k = 0; k < each; ++k) {
        const int b = mine0 + k;
        if (blockIdx.x == 0 && a.err && b < B) {
            const int32_t n = __ldcg(a.seq_lens + b);
            if (n < 0 || n > cap) atomicAdd(a.err, 1);
        }
        mine += tiles_of(length(b));
    }
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
            if (mine0 + k < B) a.ws_at[mine0 + k] = at;
            at += tiles_of(length(mine0 + k));
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
            const int n = tiles_of(length(mine0 + k));
            const int64_t lo = static_cast<int64_t>(at) * a.n_kv, hi = static_cast<int64_t>(at + n) * a.n_kv;
            if (lo <= g0 && g0 < hi) found[0] = mine0 + k, found[1] = at;
            at += n;
        }
    }
    __syncthreads();
    int b = found[0];
    int64_t begin = static_cast<int64_t>(found[1]) * a.n_kv;  // the request's first tile in the stream
    uint32_t turn = 0;
    int window = b, lens = length(b + lane);  // lane k: request window + k
    while (g0 < g1 && b < B) {
        if (b - window >= 32) window = b, lens = length(b + lane);
        const int len = __shfl_sync(FULL, lens, b - window), n = tiles_of(len);
        if (g0 >= begin + static_cast<int64_t>(n) * a.n_kv) {
            begin += static_cast<int64_t>(n) * a.n_kv;
            ++b;
            continue;
        }
        const int kvh = static_cast<int>((g0 - begin) / n);
        const int t0 = static_cast<int>(g0 - begin - static_cast<int64_t>(kvh) * n);
        const int t1 = g1 - g0 < n - t0 ? t0 + static_cast<int>(g1 - g0) : n;
        segment<T, FMT, HD>(a, smem, b, kvh, len, t0, t1, &turn);
        __syncthreads();
        const float* res = reinterpret_cast<const float*>(smem + M::res_ml);
        const float* ro = reinterpret_cast<const float*>(smem + M::res_o);
        if (t0 == 0 && t1 == n) {
            T* out = static_cast<T*>(a.out) + b * a.os + static_cast<int64_t>(kvh) * G * HD;
            for (int i = threadIdx.x; i < G * HD; i += NT) {
                const float l = res[8 + i / HD];
                out[i] = from_f32<T>(l != 0.0f ? ro[i] / l : 0.0f);
            }
        } else {
            float* rec = a.ws_rec + (static_cast<int64_t>(blockIdx.x) * 2 + (t0 == 0 ? 1 : 0)) * (16 + 8 * HD);
            for (int i = threadIdx.x; i < 16 + G * HD; i += NT) rec[i] = res[i];
        }
        g0 += t1 - t0;
        fence_proxy_async();  // the merge's accesses come before the copies that fill the rings again
        __syncthreads();
    }
}

// out of a pair whose tiles several parts share, and zeros for a request without tokens. A CTA takes 256 / LANES columns; LANES
// threads share a column's records. The sums meet in a fixed order.
template <typename T, int HD, int LANES>
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
    const int at = a.ws_at[b], n = a.ws_at[b + 1] - at;
    const int64_t part = stream_part(static_cast<int64_t>(a.ws_at[a.B]) * a.n_kv, ctas, warps);
    T* out = static_cast<T*>(a.out) + b * a.os + static_cast<int64_t>(kvh) * a.group * HD;
    if (n == 0) {
        if (p == 0 && there) out[i] = from_f32<T>(0.0f);
        return;
    }
    const int64_t first = static_cast<int64_t>(at) * a.n_kv + static_cast<int64_t>(kvh) * n;
    const int64_t c0 = first / part, c1 = (first + n - 1) / part;
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
    if (there) out[i] = from_f32<T>(sum != 0.0f ? acc / sum : 0.0f);
}

template <typename T, int FMT, int HD>
cudaError_t launch_stream(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    using M = Mem<T, FMT, HD>;
    using S = Shape<T, FMT, HD>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_smem_once(stream_kernel<T, FMT, HD>, M::total, true, &done);
    if (e != cudaSuccess) return e;
    e = launch_kernel(stream_kernel<T, FMT, HD>, dim3(static_cast<unsigned>(p.stream_ctas)), dim3(S::WARPS * 32), M::total, s, p.pdl, 1, a);
    if (e != cudaSuccess) return e;
    // pairs that many parts share: eight threads to a column
    const bool many = a.B * a.n_kv * 8 < p.stream_ctas;
    const int cols = many ? 32 : 256;
    const int64_t grid = a.B * a.n_kv * ((a.group * HD + cols - 1) / cols);
    return launch_kernel(many ? merge_kernel<T, HD, 8> : merge_kernel<T, HD, 1>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, true,
                         1, a, p.stream_ctas, S::WARPS);
}

template <typename T, int FMT, int HD>
cudaError_t launch_cluster(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    using M = Mem<T, FMT, HD>;
    auto kernel = cluster_kernel<T, FMT, HD>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_smem_once(kernel, M::total, true, &done);
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
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.B * a.n_kv * p.splits)), dim3(Shape<T, FMT, HD>::WARPS * 32), M::total, s,
                         p.pdl, p.splits, a);
}

template <typename T, int FMT>
cudaError_t launch(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    switch (p.head_dim) {
        case 64: return p.stream_ctas ? launch_stream<T, FMT, 64>(a, p, s) : launch_cluster<T, FMT, 64>(a, p, s);
        case 128: return p.stream_ctas ? launch_stream<T, FMT, 128>(a, p, s) : launch_cluster<T, FMT, 128>(a, p, s);
        default: return p.stream_ctas ? launch_stream<T, FMT, 256>(a, p, s) : launch_cluster<T, FMT, 256>(a, p, s);
    }
}

}  // namespace qattn

int quant_attn_warps(int format, int head_dim) {
    return 2 * qattn::kTile * kv_row_bytes(format, head_dim) <= 4608 ? 8 : 4;  // Shape::WARPS
}
int quant_attn_ctas_per_sm(int format, int head_dim) { return format == KV_INT8 && head_dim == 256 ? 1 : 2; }  // Shape::CTAS

unsigned int quant_attn_wait_timeouts() {
    unsigned int n = 0;
    if (cudaMemcpyFromSymbol(&n, g_wait_timeouts, sizeof(n)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

cudaError_t launch_attention_quant(const QuantAttnArgs& a, const QuantAttnPlan& p, int dtype, cudaStream_t s) {
    using namespace qattn;
    const bool e = p.format == KV_E2M1;
    switch (dtype) {
        case DT_F32: return e ? launch<float, KV_E2M1>(a, p, s) : launch<float, KV_INT8>(a, p, s);
        case DT_F16: return e ? launch<__half, KV_E2M1>(a, p, s) : launch<__half, KV_INT8>(a, p, s);
        case DT_BF16: return e ? launch<__nv_bfloat16, KV_E2M1>(a, p, s) : launch<__nv_bfloat16, KV_INT8>(a, p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace sra

// RoPE with a store that quantises, and the read back: the write side of the KV cache held in 4 or 8 bits
// (format: kv_format.cuh). Cache layout [2, num_blocks, n_kv_head, block_size, row_bytes]: a head's rows of a
// page lie in a row, so the attention copies them as one piece.
//
// Store. A thread takes a task of 16 values of one head: of Q and K eight rotation pairs, of V 16 dims in a row. In the
// neox pairing a K task holds half of two groups, whose other halves the neighbouring thread has (one shuffle
// each); otherwise a task is a group.
//
// K's rotation is the correctly rounded fp32 number, rounded once more to the dtype: an interval that holds the difference of
// products settles nearly all, the others are evaluated exactly (16384 tokens as below 28.4 us with neither, 28.7; in fp32, whose interval takes
// more work, 4096 tokens of 8 / 8 heads 16.8 and 18.2). A code can hang on the last place of its value, and with this the cache's bytes
// follow from the definition, whoever evaluates it. (Q is rotated exactly as sra_rope_kv_store does it.)
//
// It is bound by a launch and a round trip to memory (2.3 us for 64 tokens), then by what a CTA does in turn, loads, tables, stores, which five
// CTAs an SM cover in part (4: 8.8 us, 6: 8.4 and spills): 4096 tokens of 12 / 2 heads of 128 (bf16, 33 MB in 4 bits) 8.5 us, 4.8 at the copy
// rate, 16384 28.6 and 18.7; in 8 bits 9.0 and 28.9; behind the Q/K norm, whose parameters every task reads, 12.8 and 43.6. At 16384 tokens
// 0.61 of the issue slots are taken and L1 stands at 70 % of its peak; of 13.4 warps a scheduler 4.5 wait for loads, 2.5 for their turn, 1.2 for
// the load and store unit. (All three tensors' tasks in the same CTAs: 4 us more; two heads of Q a thread 11.7, K's and V's CTAs among
// Q's 10.9 for 4096 tokens.)
//
// Read. A CTA takes a tile of output tokens, finds each one's place in the cache once, and its threads turn groups of 16
// codes into one 32-byte store each (two in fp32), four groups at a time: 16 requests of up to 8192 tokens of 8 heads of 128 (4 bits to
// bf16, 285 MB written) 68 us, 54 at the copy rate. 16 x 4096 of 8 heads of 128: 4 bits to bf16 63 us (51 at the copy rate), 8 bits 71 (61), to
// fp32 109 (90) and 123 (100), 5.5 to 5.8 TB/s. Neither HBM nor the issue of instructions is full (in 8 bits to bf16 0.60 of the slots, 30 warps an
// SM by their registers): of 12.4 warps a scheduler 4.5 wait for codes and places, 1.7 at the barrier while places are found. One group at a time
// and 16-byte stores 107; two groups at a time 72; the next tile's places found while a tile is read 70.
#include "kv_format.cuh"
#include "rope_math.cuh"

namespace sra {
namespace kvq {

constexpr int kThreads = 256;

// The bits of the largest magnitude (those of infinities and NaN are above all others).
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    return m;
}
// K's rotation: a * c - b * s rounded once to fp32, then to T. Each operation below is rounded by itself, whatever the compiler may
// contract elsewhere: the error-free sums rest on it.

// By 64-bit arithmetic: the products are exact there, and a difference rounded to odd (53 bits) gives the same fp32 number as the
// exact one (Boldo and Melquiond).
__device__ __forceinline__ float rotate_wide(float a, float c, float b, float s) {
    const double p = __dmul_rn(a, c), q = __dmul_rn(b, s);
    double d = __dsub_rn(p, q);
    const double bb = __dsub_rn(d, p), e = __dsub_rn(__dsub_rn(p, __dsub_rn(d, bb)), __dadd_rn(q, bb));  // p - q = d + e
    const long long bits = __double_as_longlong(d);
    if ((e > 0.0 || e < 0.0) && !(bits & 1)) d = __longlong_as_double((e > 0.0) == (d > 0.0) ? bits + 1 : bits - 1);  // (then d is not 0)
    return __double2float_rn(d);
}
// x + y = the result + *err, exactly (Knuth's two-sum).
__device__ __forceinline__ float two_sum(float x, float y, float* err) {
    const float z = __fadd_rn(x, y), yy = __fsub_rn(z, x);
    *err = __fadd_rn(__fsub_rn(x, __fsub_rn(z, yy)), __fsub_rn(y, yy));
    return z;
}
// Whether x y is 0 or so large that its rounding error is an fp32 number.
__device__ __forceinline__ bool splits(float xy, float x, float y) { return fabsf(xy) >= 0x1p-100f || x == 0.0f || y == 0.0f; }
// Exactly, in fp32 where two of its numbers hold the difference (the ties and zeros of 16-bit inputs).
__device__ __forceinline__ float rotate_exact(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
    const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(b, s, -q);
    float e, el, tl;
    const float d = two_sum(p, -q, &e), g = two_sum(ep, -eq, &el), t = two_sum(e, g, &tl);
    // (without a t the sign of a zero is d's, IEEE's)
    if (el == 0.0f && tl == 0.0f && splits(p, a, c) && splits(q, b, s)) return t == 0.0f ? d : __fadd_rn(d, t);
    return rotate_wide(a, c, b, s);
}
// Nearly always: an interval that holds the difference. Where both ends of it are the same as T, so is the exact result; where not, and for
// a difference of 0, an infinity or a NaN, `doubt` becomes other than 0 or the result is not finite.
template <typename T>
__device__ __forceinline__ float rotate_near(float a, float c, float b, float s, uint32_t& doubt) {
    float ends[2];
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        // diff_of_products is off by 2^-23 of the difference at most (Jeannerod, Louvet and Muller), two places of fp32: a warp's 512
        // values need the exact form once in 32 times (in fp16, whose numbers lie closer, it would be once in four)
        const uint32_t bits = __float_as_uint(rope::diff_of_products(a, c, b, s));
        ends[0] = __uint_as_float(bits - 2), ends[1] = __uint_as_float(bits + 2);
    } else {
        // d + t, t off by less than 2^-44 (|p| + |q|): its three roundings come to 2.5 * 2^-47, and what a product loses below 2^-149
        // is far less than 2^-144
        const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
        const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(b, s, -q);
        float e;
        const float d = two_sum(p, -q, &e), t = __fadd_rn(e, __fsub_rn(ep, eq));
        const float size = fmaxf(__fadd_rn(fabsf(p), fabsf(q)), 0x1p-100f);
        ends[0] = __fadd_rn(d, __fmaf_rn(size, -0x1p-44f, t)), ends[1] = __fadd_rn(d, __fmaf_rn(size, 0x1p-44f, t));
    }
    if constexpr (sizeof(T) == 4) {
        doubt |= __float_as_uint(ends[0]) ^ __float_as_uint(ends[1]);
        return ends[0];
    } else {
        const uint32_t v = Elem<T>::pack_word(ends);
        doubt |= v ^ __byte_perm(v, v, 0x1032);
        float f[2];
        Elem<T>::unpack_word(v, f);
        return f[0];
    }
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool wide, float (&f)[8]) {
    if (wide) {
        constexpr int V = vec16<T>();
#pragma unroll
        for (int j = 0; j < 8; j += V) {
            float g[V];
            Vec<T, V>::unpack(Vec<T, V>::load(p + j), g);
#pragma unroll
            for (int k = 0; k < V; ++k) f[j + k] = g[k];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = to_f32(p[j]);
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool wide, const float (&f)[8]) {
    if (wide) {
        constexpr int V = vec16<T>();
#pragma unroll
        for (int j = 0; j < 8; j += V) {
            float g[V];
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] = f[j + k];
            Vec<T, V>::store(p + j, Vec<T, V>::pack(g));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = from_f32<T>(f[j]);
    }
}

template <int FMT>
__device__ __forceinline__ uint32_t scale_of(uint32_t bits) {
    return bits >= 0x7f800000u ? kScaleNaN : scale_code<FMT>(__uint_as_float(bits));
}
template <int W>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[W]) {
#pragma unroll
    for (int j = 0; j < W; ++j) reinterpret_cast<uint32_t*>(p)[j] = w[j];  // rows are multiples of 4 bytes
}

// n / d for n < 2^31 as a product and a shift: m = ceil(2^(31 + l) / d) with 2^l >= d, and n m / 2^(31 + l) exceeds n / d by less than
// n / 2^(31 + l) < 1 / d (Granlund and Montgomery).
struct Divisor {
    uint32_t d, mul, shift;
    explicit Divisor(uint32_t by) : d(by) {
        uint32_t l = 0;
        while ((uint64_t(1) << l) < by) ++l;
        mul = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + by - 1) / by);
        shift = 31 + l;
    }
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return static_cast<uint32_t>(static_cast<uint64_t>(n) * mul >> shift); }
};

// Which tensor a CTA's tasks come from; each has CTAs of its own (K's first: they have the most to do), so that no warp
// walks through two kinds' code. Tasks are numbered over tokens, heads, groups; they, and a slot's page, are found by
// multiplications (by divisions 4096 tokens of 12 / 2 heads took 0.5 us more).
struct StoreGrid {
    int64_t k_ctas, v_ctas;
    bool wide;
    bool narrow;  // every tensor's tasks are fewer than 2^31
    Divisor q_tasks, kv_tasks, page;
};

// Whether all sixteen are zeros (of either sign).
__device__ __forceinline__ bool zeros(const float (&x)[8], const float (&y)[8]) {
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) any |= __float_as_uint(x[j]) | __float_as_uint(y[j]);
    return any << 1 == 0;
}

template <typename T, int FMT, bool IL, bool NORM, int KIND>  // KIND: 0 Q, 1 K, 2 V
__device__ __forceinline__ void store_task(const RopeArgs& a, const StoreGrid& grid, int64_t cta) {
    const bool wide = grid.wide;
    constexpr int CB = FMT == KV_E2M1 ? 4 : 8;  // bits per code
    constexpr bool ROW = IL || KIND == 2;       // 16 dims in a row
    const int D = a.head_dim, h = D >> 1, lg = __ffs(D) - 5;  // 2^lg tasks a head
    const Divisor& per_token = KIND == 0 ? grid.q_tasks : grid.kv_tasks;
    int64_t t;
    int u;
    if (grid.narrow) {
        const uint32_t i = static_cast<uint32_t>(cta) * kThreads + threadIdx.x, lt = per_token.of(i);
        t = lt, u = static_cast<int>(i - lt * per_token.d);
    } else {
        const int64_t i = cta * kThreads + threadIdx.x;
        t = i / per_token.d, u = static_cast<int>(i - t * per_token.d);
    }
    const int head = u >> lg, g = u & ((1 << lg) - 1);
    bool live = t < a.T;
    int64_t p = 0, slot = -1;
    float x0[8], x1[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x0[j] = x1[j] = 0.0f;
    // offsets of the task's two runs of eight values
    const int o0 = ROW ? 16 * g : 8 * g, o1 = ROW ? 16 * g + 8 : h + 8 * g;
    T* q = nullptr;
    const T* src = nullptr;
    if (live) {
        const int64_t capacity = a.num_blocks * static_cast<int64_t>(a.block_size), ho = static_cast<int64_t>(head) * D;
        p = a.pos[t];
        if (KIND != 0) slot = a.slot[t];
        if (KIND == 0) src = q = static_cast<T*>(a.q) + t * a.qs + ho;
        else src = KIND == 1 ? static_cast<const T*>(a.k) + t * a.ks + ho : static_cast<const T*>(a.v) + t * a.vs + ho;
        load8(src + o0, wide, x0);
        load8(src + o1, wide, x1);
        const bool pos_ok = p >= 0 && p < a.max_pos, past = slot >= capacity;
        if (KIND == 1 && u == 0 && a.err != nullptr) {
            const int bad = (pos_ok ? 0 : 1) + (past ? 1 : 0);
            if (bad) atomicAdd(a.err, bad);
        }
        live = pos_ok && (KIND == 0 || (slot >= 0 && !past));
    }
    if (KIND != 2 && live) {
        const float* pa = KIND == 0 ? a.qa : a.ka;
        const float* pg = KIND == 0 ? a.qg : a.kg;
        float c[8], s[8];
        load8(a.cos + p * h + 8 * g, wide, c);
        load8(a.sin + p * h + 8 * g, wide, s);
        if constexpr (NORM) {
            float al[8], ga[8];
            load8(pa + o0, wide, al);
            load8(pg + o0, wide, ga);
#pragma unroll
            for (int j = 0; j < 8; ++j) x0[j] = round_trip<T>(rope::uclip1(x0[j], al[j], ga[j], a.clip_lo, a.clip_hi));
            load8(pa + o1, wide, al);
            load8(pg + o1, wide, ga);
#pragma unroll
            for (int j = 0; j < 8; ++j) x1[j] = round_trip<T>(rope::uclip1(x1[j], al[j], ga[j], a.clip_lo, a.clip_hi));
        }
        // pair j: neox (x0[j], x1[j]); interleaved elements 2j and 2j + 1 of the two runs
        auto first = [&](int j) -> float& { return IL ? (j < 4 ? x0[2 * j & 7] : x1[2 * j & 7]) : x0[j]; };
        auto second = [&](int j) -> float& { return IL ? (j < 4 ? x0[(2 * j + 1) & 7] : x1[(2 * j + 1) & 7]) : x1[j]; };
        if constexpr (KIND == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float lo = first(j), hi = second(j);
                first(j) = rope::diff_of_products(lo, c[j], hi, s[j]);
                second(j) = rope::diff_of_products(hi, c[j], -lo, s[j]);
            }
        } else if (zeros(x0, x1)) {  // (rotate_near settles none; padded dims, tokens without keys)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float lo = first(j), hi = second(j);
                first(j) = __fsub_rn(__fmul_rn(lo, c[j]), __fmul_rn(hi, s[j]));
                second(j) = __fsub_rn(__fmul_rn(hi, c[j]), __fmul_rn(-lo, s[j]));
            }
        } else {
            uint32_t again = 0;  // pairs that rotate_near does not settle
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float lo = first(j), hi = second(j);
                uint32_t doubt = 0;
                first(j) = rotate_near<T>(lo, c[j], hi, s[j], doubt);
                second(j) = rotate_near<T>(hi, c[j], -lo, s[j], doubt);
                if (doubt != 0) again |= 1u << j;
            }
            if (max(amax_bits(x0), amax_bits(x1)) >= 0x7f800000u) again = 0xff;
            while (again != 0) {  // (their inputs are read once more; a rolled loop, because unrolled its code comes in from far)
                const int j = __ffs(again) - 1;
                again &= again - 1;
                const int i0 = IL ? o0 + 2 * j : o0 + j, i1 = IL ? i0 + 1 : o1 + j;
                float lo = to_f32(src[i0]), hi = to_f32(src[i1]);
                if constexpr (NORM) {
                    lo = round_trip<T>(rope::uclip1(lo, pa[i0], pg[i0], a.clip_lo, a.clip_hi));
                    hi = round_trip<T>(rope::uclip1(hi, pa[i1], pg[i1], a.clip_lo, a.clip_hi));
                }
                const float cj = a.cos[p * h + 8 * g + j], sj = a.sin[p * h + 8 * g + j];
                const float y0 = round_trip<T>(rotate_exact(lo, cj, hi, sj)), y1 = round_trip<T>(rotate_exact(hi, cj, -lo, sj));
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k == j) first(k) = y0, second(k) = y1;
            }
        }
    }
    if constexpr (KIND == 0) {
        if (live) {
            store8(q + o0, wide, x0);
            store8(q + o1, wide, x1);
        }
    } else {
        uint32_t m0 = amax_bits(x0), m1 = amax_bits(x1);
        if constexpr (ROW) {
            m0 = m1 = max(m0, m1);
        } else {  // a warp's lanes meet here: the neighbour holds the groups' other halves
            m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
            m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
        }
        if (!live) return;
        const int R = row_bytes(FMT, D), codes = code_bytes(FMT, D);
        const int64_t blk = slot < 0x80000000 ? grid.page.of(static_cast<uint32_t>(slot)) : slot / a.block_size,
                      off = slot - blk * a.block_size;
        uint8_t* row = static_cast<uint8_t*>(a.cache) +
                       ((((KIND == 2 ? a.num_blocks : 0) + blk) * a.n_kv + head) * a.block_size + off) * R;
        const uint32_t c0 = scale_of<FMT>(m0), c1 = ROW ? c0 : scale_of<FMT>(m1);
        uint32_t w0[CB / 4], w1[CB / 4];
        encode<FMT>(x0, c0, w0);
        encode<FMT>(x1, c1, w1);
        store_words(row + o0 * CB / 8, w0);
        store_words(row + o1 * CB / 8, w1);
        if constexpr (ROW) {
            row[codes + g] = static_cast<uint8_t>(c0);
        } else if (!(g & 1)) {
            row[codes + (g >> 1)] = static_cast<uint8_t>(c0);
            row[codes + h / kGroup + (g >> 1)] = static_cast<uint8_t>(c1);
        }
    }
}

template <typename T, int FMT, bool IL, bool NORM>
__global__ void __launch_bounds__(kThreads, 5) store_kernel(RopeArgs a, StoreGrid grid) {
    pdl_enter();
    const int64_t cta = blockIdx.x;
    if (cta < grid.k_ctas) store_task<T, FMT, IL, NORM, 1>(a, grid, cta);
    else if (cta < grid.k_ctas + grid.v_ctas) store_task<T, FMT, IL, NORM, 2>(a, grid, cta - grid.k_ctas);
    else store_task<T, FMT, IL, NORM, 0>(a, grid, cta - grid.k_ctas - grid.v_ctas);
}

template <typename T, int FMT>
cudaError_t launch_store(const RopeArgs& a, const KvQuantPlan& p, cudaStream_t s) {
    void (*kernel)(RopeArgs, StoreGrid) =
        p.style == 0 ? (p.qk_norm ? store_kernel<T, FMT, false, true> : store_kernel<T, FMT, false, false>)
                     : (p.qk_norm ? store_kernel<T, FMT, true, true> : store_kernel<T, FMT, true, false>);
    const int64_t per_head = a.T * (a.head_dim / kGroup);
    const int64_t kv_ctas = (per_head * a.n_kv + kThreads - 1) / kThreads, q_ctas = (per_head * a.n_head + kThreads - 1) / kThreads;
    const int groups = a.head_dim / kGroup;
    const int64_t all = 2 * kv_ctas + q_ctas;
    const StoreGrid g{kv_ctas,
                      kv_ctas,
                      p.wide,
                      q_ctas * kThreads <= 0x7fffffff,
                      Divisor(static_cast<uint32_t>(a.n_head * groups)),
                      Divisor(static_cast<uint32_t>(a.n_kv * groups)),
                      Divisor(static_cast<uint32_t>(a.block_size))};
    return launch_kernel(kernel, dim3(static_cast<unsigned>(all)), dim3(kThreads), 0, s, p.pdl, 1, a, g);
}

// ------------------------------------------------------------------- read back
constexpr int kReadTokens = 32;  // of a CTA's tile, at most
constexpr int kReadRows = 1024;  // cu_lens entries kept in shared memory

// 16 values (pairs of fp16 numbers) as T, in stores of 32 bytes where `wide` is 2, of 16 where it is 1.
template <typename T>
__device__ __forceinline__ void store16(T* p, int wide, const uint32_t (&h)[8]) {
    constexpr int W = static_cast<int>(sizeof(T)) * 4;  // words
    uint32_t w[W];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (std::is_same_v<T, __half>) {
            w[j] = h[j];
        } else {
            __half2 v;
            memcpy(&v, &h[j], 4);
            const float2 x = __half22float2(v);
            if constexpr (sizeof(T) == 4) {
                w[2 * j] = __float_as_uint(x.x), w[2 * j + 1] = __float_as_uint(x.y);
            } else {
                const float f[2] = {x.x, x.y};
                w[j] = Elem<T>::pack_word(f);
            }
        }
    }
    if (wide == 2) {
#pragma unroll
        for (int j = 0; j < W; j += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint32_t*>(p) + j),
                         "r"(w[j]), "r"(w[j + 1]), "r"(w[j + 2]), "r"(w[j + 3]), "r"(w[j + 4]), "r"(w[j + 5]), "r"(w[j + 6]),
                         "r"(w[j + 7])
                         : "memory");
    } else if (wide == 1) {
#pragma unroll
        for (int j = 0; j < W; j += 4) reinterpret_cast<uint4*>(p)[j / 4] = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = __uint_as_float(w[j]);
    } else {
        unsigned short* q = reinterpret_cast<unsigned short*>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[2 * j] = static_cast<unsigned short>(w[j]), q[2 * j + 1] = static_cast<unsigned short>(w[j] >> 16);
    }
}

// A thread's items are groups of 16 values: four at a time, whose bytes are all asked for before the first is used.
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) read_kernel(KvReadArgs a, int tile, int wide) {
    constexpr int WORDS = FMT == KV_E2M1 ? 2 : 4;  // of sixteen codes
    constexpr int MANY = 4;
    __shared__ int32_t s_cu[kReadRows + 1];
    __shared__ int64_t s_at[kReadTokens];  // page * n_kv * block_size + offset of each token; -1: zeros, -2: not written
    pdl_enter();
    const int D = a.head_dim, lg = __ffs(D) - 5, R = row_bytes(FMT, D), codes = code_bytes(FMT, D);
    const bool cached = a.rows <= kReadRows;
    if (cached) {
        for (int64_t i = threadIdx.x; i <= a.rows; i += kThreads) s_cu[i] = a.cu[i];
        __syncthreads();
    }
    auto cu = [&](int64_t r) { return cached ? s_cu[r] : a.cu[r]; };
    const int per_token = 2 * a.n_kv << lg;  // items: planes, heads, groups
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile; t0 < a.total; t0 += static_cast<int64_t>(gridDim.x) * tile) {
        if (threadIdx.x < tile) {
            const int64_t i = t0 + threadIdx.x;
            int64_t at = -2;
            if (i < a.total && i >= cu(0) && i < cu(a.rows)) {
                int64_t lo = 0, hi = a.rows;  // the last row that starts at or before i
                while (hi - lo > 1) {
                    const int64_t mid = (lo + hi) >> 1;
                    if (cu(mid) <= i) lo = mid;
                    else hi = mid;
                }
                const int64_t first = cu(lo);
                const int64_t from = a.starts ? a.starts[lo] : 0;
                const int64_t tok = from + (i - first);
                const bool in_row = tok >= 0 && tok < a.max_blocks * a.block_size;
                const int64_t j = in_row ? tok / a.block_size : 0, off = tok - j * a.block_size;
                const int32_t page = in_row ? a.table[lo * a.max_blocks + j] : -1;
                const bool ok = page >= 0 && page < a.num_blocks;
                // one count for a bad entry (at the first of its tokens in the results), one for each row that leaves its table (likewise)
                const int64_t seen = first < 0 ? 0 : first;
                if (!ok && a.err && (i == seen || (in_row ? off == 0 : from + (seen - first) >= 0 && tok == a.max_blocks * a.block_size)))
                    atomicAdd(a.err, 1);
                at = ok ? static_cast<int64_t>(page) * a.n_kv * a.block_size + off : -1;
            }
            s_at[threadIdx.x] = at;
        }
        __syncthreads();
        const int n = static_cast<int>(a.total - t0 < tile ? a.total - t0 : tile) * per_token;
        for (int base = threadIdx.x; base < n; base += MANY * kThreads) {
            uint32_t w[MANY][WORDS];
            uint32_t scale[MANY];
            T* out[MANY];
#pragma unroll
            for (int k = 0; k < MANY; ++k) {
                const unsigned it = base + k * kThreads;
                out[k] = nullptr;
                scale[k] = 0;
#pragma unroll
                for (int j = 0; j < WORDS; ++j) w[k][j] = 0;
                if (it < static_cast<unsigned>(n)) {
                    const unsigned lt = it / static_cast<unsigned>(per_token), rest = it - lt * per_token;
                    const int g = rest & ((1 << lg) - 1);
                    int head = rest >> lg;
                    const bool plane = head >= a.n_kv;
                    if (plane) head -= a.n_kv;
                    const int64_t at = s_at[lt];
                    if (at != -2)
                        out[k] = static_cast<T*>(plane ? a.v : a.k) + (t0 + lt) * (plane ? a.vs : a.ks) + head * D + g * kGroup;
                    if (at >= 0) {
                        const uint8_t* row = static_cast<const uint8_t*>(a.cache) + (plane ? a.plane_bytes : 0) +
                                             (at + static_cast<int64_t>(head) * a.block_size) * R;
                        scale[k] = row[codes + g];
                        if (R % 8 == 0) {  // rows of head_dim 64 are multiples of 4 bytes only
#pragma unroll
                            for (int j = 0; j < WORDS; j += 2) {
                                const uint2 v = *reinterpret_cast<const uint2*>(row + (g * WORDS + j) * 4);
                                w[k][j] = v.x, w[k][j + 1] = v.y;
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < WORDS; ++j) w[k][j] = reinterpret_cast<const uint32_t*>(row)[g * WORDS + j];
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < MANY; ++k) {
                if (!out[k]) continue;
                uint32_t lo[4], hi[4];
                decode8<FMT>(w[k], scale_pair(scale[k]), lo);
                decode8<FMT>(w[k] + WORDS / 2, scale_pair(scale[k]), hi);
                const uint32_t h[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                store16(out[k], wide, h);
            }
        }
        __syncthreads();
    }
}

template <typename T, int FMT>
cudaError_t launch_read(const KvReadArgs& a, const KvQuantPlan& p, cudaStream_t s) {
    auto kernel = read_kernel<T, FMT>;
    // up to 32 tokens in a tile; for few tokens as many as give every thread of a CTA an item
    const int per_token = 2 * a.n_kv * (a.head_dim / kGroup);
    int tile = kReadTokens;
    while (tile > 1 && tile / 2 * per_token >= kThreads && (a.total + tile - 1) / tile < 4 * static_cast<int64_t>(p.num_sms)) tile >>= 1;
    const dim3 grid(persistent_grid(kernel, kThreads, 0, p.num_sms, (a.total + tile - 1) / tile));
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                           static_cast<uintptr_t>((a.ks | a.vs) * static_cast<int64_t>(sizeof(T)));
    const int wide = bits % 32 == 0 ? 2 : bits % 16 == 0 ? 1 : 0;
    return launch_kernel(kernel, grid, dim3(kThreads), 0, s, p.pdl, 1, a, tile, wide);
}

}  // namespace kvq

cudaError_t launch_rope_kv_store_quant(const RopeArgs& a, const KvQuantPlan& p, int dtype, cudaStream_t s) {
    using namespace kvq;
    const bool e = p.format == KV_E2M1;
    switch (dtype) {
        case DT_F32: return e ? launch_store<float, KV_E2M1>(a, p, s) : launch_store<float, KV_INT8>(a, p, s);
        case DT_F16: return e ? launch_store<__half, KV_E2M1>(a, p, s) : launch_store<__half, KV_INT8>(a, p, s);
        case DT_BF16: return e ? launch_store<__nv_bfloat16, KV_E2M1>(a, p, s) : launch_store<__nv_bfloat16, KV_INT8>(a, p, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv_quant_read(const KvReadArgs& a, const KvQuantPlan& p, int dtype, cudaStream_t s) {
    using namespace kvq;
    const bool e = p.format == KV_E2M1;
    switch (dtype) {
        case DT_F32: return e ? launch_read<float, KV_E2M1>(a, p, s) : launch_read<float, KV_INT8>(a, p, s);
        case DT_F16: return e ? launch_read<__half, KV_E2M1>(a, p, s) : launch_read<__half, KV_INT8>(a, p, s);
        case DT_BF16: return e ? launch_read<__nv_bfloat16, KV_E2M1>(a, p, s) : launch_read<__nv_bfloat16, KV_INT8>(a, p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace sra

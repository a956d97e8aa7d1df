// RoPE with a store that quantises, and the read back: the write side of the KV cache held in 4 or 8 bits
// (format: kv_format.cuh). Cache layout [2, num_blocks, n_kv_head, block_size, row_bytes]: a head's rows of a
// page lie in a row, so the attention copies them as one piece.
//
// Store. A token's work is (n_head + 2 n_kv_head) * head_dim / 16 tasks of 16 values: Q and K as eight rotation
// pairs, V as 16 dims in a row. In the neox pairing a K task holds half of two groups, whose other halves the
// neighbouring thread has (one shuffle each); otherwise a task is a group.
//
// K's rotation is the correctly rounded fp32 number (the product difference is kept as a sum of two fp32 numbers), rounded
// once more to the dtype. A code can hang on the last place of its value, and with this the cache's bytes
// follow from the definition, whoever evaluates it. (Q is rotated exactly as sra_rope_kv_store does it.)
//
// Read. A CTA takes a tile of output tokens, finds each one's row of the cache once, and its threads turn eight codes
// into one 16-byte store (two in fp32).
#include "kv_format.cuh"
#include "rope_math.cuh"

namespace sra {
namespace kvq {

constexpr int kThreads = 256;

// The fp32 number nearest to a * c - b * s (of a sum that is known to about 2^-46 of the products).
__device__ __forceinline__ float rotate_exact(float a, float c, float b, float s) {
    const float p = a * c, q = b * s;
    const float ep = fmaf(a, c, -p), eq = fmaf(b, s, -q);
    const float d = p - q, bb = d - p;
    const float e = (p - (d - bb)) + (-q - bb);  // p - q = d + e, exactly (Knuth's two-sum)
    return d + (e + (ep - eq));
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

// The bits of the largest magnitude (those of infinities and NaN are above all others).
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float (&x)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    return m;
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

template <typename T, int FMT, bool IL, bool NORM>
__global__ void __launch_bounds__(kThreads) store_kernel(RopeArgs a, int tokens_per_cta, bool wide) {
    constexpr int CB = FMT == KV_E2M1 ? 4 : 8;  // bits per code
    pdl_enter();
    const int D = a.head_dim, h = D >> 1, per_head = D / kGroup;
    const int U = (a.n_head + 2 * a.n_kv) * per_head;
    const int R = row_bytes(FMT, D), codes = code_bytes(FMT, D);
    const int64_t capacity = a.num_blocks * static_cast<int64_t>(a.block_size);
    const int tasks = U * tokens_per_cta;  // of a CTA at a time; more than kThreads only for one token
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_cta; t0 < a.T;
         t0 += static_cast<int64_t>(gridDim.x) * tokens_per_cta) {
        for (int base = 0; base < tasks; base += kThreads) {
            const int i = base + threadIdx.x;
            const int lt = tokens_per_cta == 1 ? 0 : i / U, u = i - lt * U;
            const int64_t t = t0 + lt;
            bool live = i < tasks && t < a.T;
            const int unit = u / per_head, g = u - unit * per_head;
            const int kind = unit < a.n_head ? 0 : (unit < a.n_head + a.n_kv ? 1 : 2);  // Q, K, V head
            const int head = kind == 0 ? unit : (kind == 1 ? unit - a.n_head : unit - a.n_head - a.n_kv);
            int64_t p = 0, slot = -1;
            if (live) {
                p = a.pos[t];
                slot = a.slot[t];
                const bool pos_ok = p >= 0 && p < a.max_pos, past = slot >= capacity;
                if (u == 0 && a.err != nullptr) {
                    const int bad = (pos_ok ? 0 : 1) + (past ? 1 : 0);
                    if (bad) atomicAdd(a.err, bad);
                }
                live = pos_ok && (kind == 0 || (slot >= 0 && !past));
            }
            // offsets of the task's two runs of eight values
            const bool in_a_row = IL || kind == 2;
            const int o0 = in_a_row ? 16 * g : 8 * g, o1 = in_a_row ? 16 * g + 8 : h + 8 * g;
            float x0[8], x1[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x0[j] = x1[j] = 0.0f;
            T* q = nullptr;
            if (live) {
                const int64_t ho = static_cast<int64_t>(head) * D;
                q = static_cast<T*>(a.q) + t * a.qs + ho;
                const T* src = kind == 0 ? q : kind == 1 ? static_cast<const T*>(a.k) + t * a.ks + ho
                                                        : static_cast<const T*>(a.v) + t * a.vs + ho;
                load8(src + o0, wide, x0);
                load8(src + o1, wide, x1);
                if (kind != 2) {
                    float c[8], s[8];
                    load8(a.cos + p * h + 8 * g, wide, c);
                    load8(a.sin + p * h + 8 * g, wide, s);
                    if constexpr (NORM) {
                        const float* pa = kind == 0 ? a.qa : a.ka;
                        const float* pg = kind == 0 ? a.qg : a.kg;
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
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float& lo = IL ? (j < 4 ? x0[2 * j & 7] : x1[2 * j & 7]) : x0[j];
                        float& hi = IL ? (j < 4 ? x0[(2 * j + 1) & 7] : x1[(2 * j + 1) & 7]) : x1[j];
                        float y0, y1;
                        if (kind == 0) {
                            y0 = rope::diff_of_products(lo, c[j], hi, s[j]);
                            y1 = rope::diff_of_products(hi, c[j], -lo, s[j]);
                        } else {
                            y0 = round_trip<T>(rotate_exact(lo, c[j], hi, s[j]));
                            y1 = round_trip<T>(rotate_exact(hi, c[j], -lo, s[j]));
                        }
                        lo = y0, hi = y1;
                    }
                    if (kind == 0) {
                        store8(q + o0, wide, x0);
                        store8(q + o1, wide, x1);
                    }
                }
            }
            // a warp's lanes meet here for the groups' maxima
            uint32_t m0 = amax_bits(x0), m1 = amax_bits(x1);
            const uint32_t n0 = __shfl_xor_sync(0xffffffffu, m0, 1), n1 = __shfl_xor_sync(0xffffffffu, m1, 1);
            if (in_a_row) m0 = m1 = max(m0, m1);
            else m0 = max(m0, n0), m1 = max(m1, n1);
            if (!live || kind == 0) continue;
            const int64_t blk = slot / a.block_size, off = slot - blk * a.block_size;
            uint8_t* row = static_cast<uint8_t*>(a.cache) +
                           ((((kind == 2 ? a.num_blocks : 0) + blk) * a.n_kv + head) * a.block_size + off) * R;
            const uint32_t c0 = scale_of<FMT>(m0), c1 = in_a_row ? c0 : scale_of<FMT>(m1);
            uint32_t w0[CB / 4], w1[CB / 4];
            encode<FMT>(x0, c0, w0);
            encode<FMT>(x1, c1, w1);
            store_words(row + o0 * CB / 8, w0);
            store_words(row + o1 * CB / 8, w1);
            if (in_a_row) {
                row[codes + g] = static_cast<uint8_t>(c0);
            } else if (!(g & 1)) {
                row[codes + (g >> 1)] = static_cast<uint8_t>(c0);
                row[codes + h / kGroup + (g >> 1)] = static_cast<uint8_t>(c1);
            }
        }
    }
}

template <typename T, int FMT>
cudaError_t launch_store(const RopeArgs& a, const KvQuantPlan& p, cudaStream_t s) {
    void (*kernel)(RopeArgs, int, bool) =
        p.style == 0 ? (p.qk_norm ? store_kernel<T, FMT, false, true> : store_kernel<T, FMT, false, false>)
                     : (p.qk_norm ? store_kernel<T, FMT, true, true> : store_kernel<T, FMT, true, false>);
    const int U = (a.n_head + 2 * a.n_kv) * (a.head_dim / kGroup);
    const int tokens = U < kThreads ? kThreads / U : 1;
    const dim3 grid(persistent_grid(kernel, kThreads, 0, p.num_sms, (a.T + tokens - 1) / tokens));
    return launch_kernel(kernel, grid, dim3(kThreads), 0, s, p.pdl, 1, a, tokens, p.wide);
}

// ------------------------------------------------------------------- read back
constexpr int kReadTokens = 32;   // of a CTA's tile, at most
constexpr int kReadRows = 1024;   // cu_lens entries kept in shared memory

// The pair of fp16 numbers as T.
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, bool wide, const uint32_t (&h)[4]) {
    if constexpr (std::is_same_v<T, __half>) {
        if (wide) {
            *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
            return;
        }
    }
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __half2 v;
        memcpy(&v, &h[j], 4);
        const float2 x = __half22float2(v);
        f[2 * j] = x.x, f[2 * j + 1] = x.y;
    }
    store8(p, wide, f);
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads) read_kernel(KvReadArgs a, int tile, bool wide) {
    constexpr int WORDS = FMT == KV_E2M1 ? 1 : 2;  // of eight codes
    __shared__ int32_t s_cu[kReadRows + 1];
    __shared__ int64_t s_at[kReadTokens];  // (page * n_kv * block_size + offset) of each token; -1: zeros, -2: not written
    pdl_enter();
    const int D = a.head_dim, per_head = D / 8, R = row_bytes(FMT, D), codes = code_bytes(FMT, D);
    const bool cached = a.rows <= kReadRows;
    if (cached) {
        for (int64_t i = threadIdx.x; i <= a.rows; i += kThreads) s_cu[i] = a.cu[i];
        __syncthreads();
    }
    auto cu = [&](int64_t r) { return cached ? s_cu[r] : __ldg(a.cu + r); };
    const int per_token = 2 * a.n_kv * per_head;  // items: both planes
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
                const bool in_row = from >= 0 && tok < a.max_blocks * a.block_size;
                const int64_t j = in_row ? tok / a.block_size : 0, off = tok - j * a.block_size;
                const int32_t page = in_row ? a.table[lo * a.max_blocks + j] : -1;
                const bool ok = page >= 0 && page < a.num_blocks;
                // one count for a bad entry (at its first token), one for each row that leaves its table (likewise)
                if (!ok && a.err && (i == first || (in_row ? off == 0 : from >= 0 && tok == a.max_blocks * a.block_size)))
                    atomicAdd(a.err, 1);
                at = ok ? static_cast<int64_t>(page) * a.n_kv * a.block_size + off : -1;
            }
            s_at[threadIdx.x] = at;
        }
        __syncthreads();
        const int n = static_cast<int>(a.total - t0 < tile ? a.total - t0 : tile) * per_token;
        for (int it = threadIdx.x; it < n; it += kThreads) {
            const int lt = it / per_token;
            int rest = it - lt * per_token;
            const int plane = rest >= per_token / 2 ? 1 : 0;
            rest -= plane * (per_token / 2);
            const int head = rest / per_head, d = (rest - head * per_head) * 8;
            const int64_t at = s_at[lt];
            if (at == -2) continue;
            uint32_t v[4] = {0, 0, 0, 0};
            if (at >= 0) {
                const uint8_t* row = static_cast<const uint8_t*>(a.cache) + plane * a.plane_bytes +
                                     (at + static_cast<int64_t>(head) * a.block_size) * R;
                uint32_t w[WORDS];
#pragma unroll
                for (int j = 0; j < WORDS; ++j) w[j] = reinterpret_cast<const uint32_t*>(row + d * WORDS / 2)[j];
                decode8<FMT>(w, scale_pair(row[codes + d / kGroup]), v);
            }
            T* out = static_cast<T*>(plane ? a.v : a.k) + (t0 + lt) * (plane ? a.vs : a.ks) + head * D + d;
            store_pairs(out, wide, v);
        }
        __syncthreads();
    }
}

template <typename T, int FMT>
cudaError_t launch_read(const KvReadArgs& a, const KvQuantPlan& p, cudaStream_t s) {
    auto kernel = read_kernel<T, FMT>;
    // few tokens: a CTA for each; many: up to 32 in a tile
    int tile = kReadTokens;
    while (tile > 1 && (a.total + tile - 1) / tile < 4 * static_cast<int64_t>(p.num_sms)) tile >>= 1;
    const dim3 grid(persistent_grid(kernel, kThreads, 0, p.num_sms, (a.total + tile - 1) / tile));
    return launch_kernel(kernel, grid, dim3(kThreads), 0, s, p.pdl, 1, a, tile, p.wide);
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

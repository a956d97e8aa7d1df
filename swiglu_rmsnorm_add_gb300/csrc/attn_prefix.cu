// Attention of a decode batch over the prefix that its requests share: the prefix's K and V are read
// for all requests together.
//
// For one KV head the queries of all requests (rows = B * G, G query heads per KV head) meet the same
// K and V, so S = Q K^T and O = P V are matrix products of up to some thousand rows with the prefix's
// tokens: 4 * rows * head_dim operations per token against 4 * head_dim bytes, tensor-core work from
// about 280 rows on. prefix_tc_kernel below does them on the fifth-generation tensor cores; each
// request's own tokens go through the decode kernels of attn.cu (launch_prefix_tail), and merge_kernel
// joins the parts: with (m_i, l_i, o_i) the maximum, sum of exponentials and weighted V of part i,
// out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, M = max m_i.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace sra {
namespace prefix {

constexpr int kTok = 128;           // tokens of a K / V tile
constexpr int kRows = 128;          // query rows of a tile (the MMA's M)
constexpr int kThreads = 384;       // producer, MMA, two spare warps; two softmax warpgroups
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.0f;    // base-2 headroom of the running maximum, see softmax below

template <int HD>
struct Smem {
    static constexpr int kHalves = HD / 64;
    static constexpr int kHalfBytes = kTok * 128;              // 64 dims of a tile's 128 rows
    static constexpr int kTileBytes = kHalves * kHalfBytes;    // a K, V or Q tile
    static constexpr int kStages = HD == 128 ? 5 : 10;         // K or V tiles in flight
    static constexpr size_t kTotal = 1024 + (2 + kStages) * static_cast<size_t>(kTileBytes);
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What CTA `c` of a KV head's works on.
struct Work {
    int row0;      // first query row
    bool pair;     // two row tiles on the same K / V tiles, or one row tile on two K / V tiles at a time
    int t0, n;     // K / V tiles
    int rec;       // record of stream 0 (stream 1: the same in a pair, the next otherwise)
};
__device__ __forceinline__ Work work_of(const PrefixArgs& a, int c, int64_t tiles) {
    Work w;
    int split, splits;
    if (c < a.pair_blocks * a.pair_splits) {
        const int blk = c / a.pair_splits;
        split = c - blk * a.pair_splits, splits = a.pair_splits;
        w.pair = true;
        w.row0 = blk * 2 * kRows;
        w.rec = split;
    } else {
        split = c - a.pair_blocks * a.pair_splits, splits = a.single_splits;
        w.pair = false;
        w.row0 = a.pair_blocks * 2 * kRows;
        w.rec = 2 * split;
    }
    const int64_t b = tiles * split / splits, e = tiles * (split + 1) / splits;
    w.t0 = static_cast<int>(b);
    w.n = static_cast<int>(e - b);
    return w;
}
// Whole pages of the prefix, and its K / V tiles.
__device__ __forceinline__ int64_t whole_pages(const PrefixArgs& a) {
    const int64_t P = *a.plen, cap = a.pblocks * a.block_size;
    return (P < 0 ? 0 : (P > cap ? cap : P)) / a.block_size;
}

// The order in which K and V tiles go through the ring (both sides follow it): entry s of 2 n is V or K
// of tile t. A pair uses K0 V0 K1 V1 ...; a single block, whose streams take even and odd tiles, needs
// K0 K1 V0 K2 V1 K3 ... V(n-1).
__device__ __forceinline__ void ring_entry(bool pair, int n, int s, bool* is_v, int* t) {
    if (pair) {
        *is_v = s & 1, *t = s >> 1;
    } else if (s == 2 * n - 1) {
        *is_v = true, *t = n - 1;
    } else {
        *is_v = s != 0 && (s & 1) == 0;
        *t = s == 0 ? 0 : *is_v ? (s - 2) / 2 : (s + 1) / 2;
    }
}
__device__ __forceinline__ int ring_k(bool pair, int t) { return pair ? 2 * t : t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int ring_v(bool pair, int n, int t) {
    return pair ? 2 * t + 1 : 2 + 2 * t < 2 * n - 1 ? 2 + 2 * t : 2 * n - 1;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    float f[2] = {x, y};
    return Elem<T>::pack_word(f);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(PrefixArgs a, const __grid_constant__ CUtensorMap tmC) {
    using L = Smem<HD>;
    constexpr int ST = L::kStages;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // tensor memory: S of the two streams, then O; P (16-bit, 64 columns) over S's first columns
    constexpr uint32_t kS = 0, kO = 256;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* qs = smem;                          // two Q tiles
    unsigned char* ring = smem + 2 * L::kTileBytes;    // ST K / V tiles
    __shared__ uint64_t full[ST], empty[ST], s_full[2], p_full[2], pv_done[2];
    __shared__ uint32_t tmem_base;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int x = 0; x < 2; ++x) mbar_init(&s_full[x], 1), mbar_init(&p_full[x], 4), mbar_init(&pv_done[x], 1);
        mbar_init_fence();
    }
    if (warp == 1) {
        tc::alloc(&tmem_base, kTmemCols);
        tc::relinquish();
    }
    pdl_enter();
    const int kvh = blockIdx.x / a.ctas_per_kv;
    const int64_t pages = whole_pages(a);
    const int ppt = kTok / a.block_size;  // pages of a tile
    const Work w = work_of(a, blockIdx.x - kvh * a.ctas_per_kv, (pages + ppt - 1) / ppt);
    const int n0 = w.pair ? w.n : (w.n + 1) / 2, n1 = w.pair ? w.n : w.n / 2;  // tiles of the streams

    // the query rows, swizzled as a TMA copy would leave them; rows past the last are zero
    {
        constexpr int kChunks = HD / 8;
        const int tiles = w.pair ? 2 : 1;
        for (int i = threadIdx.x; i < tiles * kRows * kChunks && w.n > 0; i += kThreads) {
            const int r = i / kChunks, c = i - r * kChunks, row = w.row0 + r;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row < a.rows) {
                const int b = row / a.group, g = row - b * a.group;
                const T* src = static_cast<const T*>(a.q) + b * a.qs + (kvh * a.group + g) * HD + c * 8;
                if (a.q16) {
                    v = *reinterpret_cast<const uint4*>(src);
                } else {
                    const unsigned short* e = reinterpret_cast<const unsigned short*>(src);
                    v.x = e[0] | static_cast<uint32_t>(e[1]) << 16, v.y = e[2] | static_cast<uint32_t>(e[3]) << 16;
                    v.z = e[4] | static_cast<uint32_t>(e[5]) << 16, v.w = e[6] | static_cast<uint32_t>(e[7]) << 16;
                }
                if (a.negate) v.x ^= 0x80008000u, v.y ^= 0x80008000u, v.z ^= 0x80008000u, v.w ^= 0x80008000u;
            }
            const int rr = r % kRows;
            *reinterpret_cast<uint4*>(qs + (r / kRows) * L::kTileBytes + (c / 8) * L::kHalfBytes + rr * 128 +
                                      (((c & 7) ^ (rr & 7)) * 16)) = v;
        }
        fence_proxy_async();  // before the tensor core reads them
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    bool dead = false;  // a bounded wait ran out (counted): this thread waits no more
    auto wait = [&](uint64_t* bar, int phase) {
        if (!dead) dead = !mbar_wait(bar, static_cast<uint32_t>(phase & 1));
    };

    if (warp == 0) {
        // producer: a tile is a box of 64 dims x block_size tokens per page and half. A page past the
        // prefix, or an entry that is no page, is copied from past the cache's end: zeros.
        const int boxes = ppt * L::kHalves;
        for (int s = 0; s < 2 * w.n; ++s) {
            bool is_v;
            int t;
            ring_entry(w.pair, w.n, s, &is_v, &t);
            const int stage = s % ST;
            if (s >= ST) wait(&empty[stage], s / ST - 1);
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], L::kTileBytes);
            __syncwarp();
            for (int i = lane; i < boxes; i += 32) {
                const int half = i / ppt, p = i - half * ppt;
                const int64_t j = static_cast<int64_t>(w.t0 + t) * ppt + p;
                int64_t blk = j < pages ? a.ptable[j] : -1;
                if (blk < 0 || blk >= a.num_blocks) blk = a.num_blocks;
                tma_load_4d(ring + stage * L::kTileBytes + half * L::kHalfBytes + p * a.block_size * 128, &tmC,
                            half * 64, kvh, static_cast<int>(blk * a.block_size), is_v ? 1 : 0, &full[stage]);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t kIdescS = tc::idesc_f16(kBf16, kRows, kTok);
            constexpr uint32_t kIdescO = tc::idesc_f16(kBf16, kRows, HD) | tc::kTransposeB;
            auto qk = [&](int x, int t) {
                const unsigned char* k = ring + (ring_k(w.pair, t) % ST) * L::kTileBytes;
                const unsigned char* q = qs + (w.pair ? x : 0) * L::kTileBytes;
#pragma unroll
                for (int s = 0; s < HD / 16; ++s) {
                    const int off = (s / 4) * L::kHalfBytes;
                    tc::mma_f16(tmem + kS + x * kTok, tc::sdesc_sw128(q + off, (s % 4) * 32),
                                tc::sdesc_sw128(k + off, (s % 4) * 32), kIdescS, s > 0);
                }
                tc::commit(&s_full[x]);
            };
            auto pv = [&](int x, int t, bool acc) {
                const unsigned char* v = ring + (ring_v(w.pair, w.n, t) % ST) * L::kTileBytes;
#pragma unroll
                for (int s = 0; s < kTok / 16; ++s)
                    tc::mma_f16_ts(tmem + kO + x * HD, tmem + kS + x * kTok + 8 * s,
                                   tc::sdesc_sw128_mn(v, L::kHalfBytes, s), kIdescO, acc || s > 0);
                tc::commit(&pv_done[x]);
            };
            auto ready = [&](int s) {
                wait(&full[s % ST], s / ST);
                tc::fence_after();
            };
            auto release = [&](int s) { tc::commit(&empty[s % ST]); };
            const int nx[2] = {n0, n1};
            auto tile = [&](int x, int i) { return w.pair ? i : 2 * i + x; };
            auto load_k = [&](int x, int i) {  // S of stream x's tile i
                const int s = ring_k(w.pair, tile(x, i));
                if (!w.pair || x == 0) ready(s);
                qk(x, tile(x, i));
                if (!w.pair || x == 1) release(s);
            };
            for (int x = 0; x < 2; ++x)
                if (nx[x] > 0) load_k(x, 0);
            for (int i = 0; i < n0; ++i)
                for (int x = 0; x < 2; ++x) {
                    if (i >= nx[x]) continue;
                    const int s = ring_v(w.pair, w.n, tile(x, i));
                    if (!w.pair || x == 0) ready(s);
                    wait(&p_full[x], i);
                    tc::fence_after();
                    pv(x, tile(x, i), i > 0);
                    if (!w.pair || x == 1) release(s);
                    if (i + 1 < nx[x]) {
                        wait(&pv_done[x], i);  // P has been read: S may go over it
                        load_k(x, i + 1);
                    }
                }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // softmax: thread = query row of stream x. The running maximum m (base 2, scaled) is moved only
        // when a tile's maximum passes it by more than kRescale: o and l are sums of 2^(s - m) for one
        // m, so any m will do as long as nothing overflows (2^8 times a row's sum of values does not),
        // and O in tensor memory is scaled seldom.
        const int x = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lanes + kS + x * kTok, tO = tmem + lanes + kO + x * HD;
        const int n = x == 0 ? n0 : n1;
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.0f;
        // the tile's pages that count, asked for a tile ahead
        auto ask = [&](int i) -> int32_t {
            const int64_t j = static_cast<int64_t>(w.t0 + (w.pair ? i : 2 * i + x)) * ppt + lane;
            return i < n && lane < ppt && j < pages ? a.ptable[j] : -1;
        };
        int32_t entry = ask(0);
        const unsigned all_pages = static_cast<unsigned>((1ull << ppt) - 1);
        const int bs_log2 = __ffs(a.block_size) - 1;
        for (int i = 0; i < n; ++i) {
            const unsigned valid = __ballot_sync(0xffffffffu, entry >= 0 && entry < a.num_blocks);
            entry = ask(i + 1);
            wait(&s_full[x], i);
            tc::fence_after();
            uint32_t lo[2][32], hi[32];
            tc::ld32(tS, lo[0]);
            tc::ld32(tS + 32, lo[1]);
            tc::wait_ld();
            auto mask = [&](uint32_t(&v)[32], int c0) {
                if (valid == all_pages) return;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (!((valid >> ((c0 + k) >> bs_log2)) & 1u)) v[k] = __float_as_uint(-INFINITY);
            };
            float mx = -INFINITY;
            auto top = [&](const uint32_t(&v)[32]) {
#pragma unroll
                for (int k = 0; k < 32; ++k) mx = fmaxf(mx, __uint_as_float(v[k]));
            };
            mask(lo[0], 0), mask(lo[1], 32);
            top(lo[0]), top(lo[1]);
#pragma unroll
            for (int h = 2; h < 4; ++h) {
                tc::ld32(tS + 32 * h, hi);
                tc::wait_ld();
                mask(hi, 32 * h);
                top(hi);
            }
            mx *= c;
            if (i == 0) {
                m = mx;
            } else {
                const bool move = mx > m + kRescale;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? ex2(m - mx) : 1.0f;
                    if (move) l *= f, m = mx;
                    wait(&pv_done[x], i - 1);
                    tc::fence_after();
#pragma unroll 1
                    for (int d = 0; d < HD; d += 32) {
                        tc::ld32(tO + d, hi);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) hi[k] = __float_as_uint(__uint_as_float(hi[k]) * f);
                        tc::st32(tO + d, hi);
                    }
                    tc::wait_st();
                }
            }
            const float base = m == -INFINITY ? 0.0f : m;
            // p = 2^(c s - m), summed in fp32, rounded once to T: a relative error of half a step of T
            // per probability, which the product with V averages over the tokens
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            auto expo = [&](uint32_t(&v)[32], uint32_t* packed) {
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float p0 = ex2(fmaf(__uint_as_float(v[k]), c, -base));
                    const float p1 = ex2(fmaf(__uint_as_float(v[k + 1]), c, -base));
                    part[k & 2] += p0, part[(k & 2) + 1] += p1;
                    packed[k / 2] = pack2<T>(p0, p1);
                }
            };
            uint32_t pk[32];
            expo(lo[0], pk), expo(lo[1], pk + 16);
            tc::st32(tS, pk);  // over columns 0-31 of S, which this thread has read
            tc::ld32(tS + 64, lo[0]);
            tc::ld32(tS + 96, lo[1]);
            tc::wait_ld();
            mask(lo[0], 64), mask(lo[1], 96);
            expo(lo[0], pk), expo(lo[1], pk + 16);
            tc::st32(tS + 32, pk);
            l += (part[0] + part[1]) + (part[2] + part[3]);
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x]);
        }
        // this stream's record: maximum, sum, O (no tile: a maximum of -inf, and O is not read)
        const int r = w.row0 + (w.pair ? x * kRows : 0) + quarter * 32 + lane;
        const int64_t at = (static_cast<int64_t>(kvh) * a.rows + r) * a.records + w.rec + (w.pair ? 0 : x);
        if (r < a.rows) a.part_ml[at] = make_float2(m, l);
        if (n > 0) {
            wait(&pv_done[x], n - 1);
            tc::fence_after();
#pragma unroll 1
            for (int d = 0; d < HD; d += 32) {
                uint32_t v[32];
                tc::ld32(tO + d, v);
                tc::wait_ld();
                if (r < a.rows) {
                    uint4* dst = reinterpret_cast<uint4*>(a.part_o + at * HD + d);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::dealloc(tmem, kTmemCols);
    }
}

template <typename T, int HD>
cudaError_t launch_tc(const PrefixArgs& a, const void* cache, bool pdl, cudaStream_t s) {
    const int BS = a.block_size;
    const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * BS;
    const uint64_t dims[4] = {static_cast<uint64_t>(HD), static_cast<uint64_t>(a.n_kv), rows, 2};
    const uint64_t strides[3] = {static_cast<uint64_t>(HD) * 2, static_cast<uint64_t>(a.n_kv) * HD * 2,
                                 rows * a.n_kv * HD * 2};
    const uint32_t box[4] = {64, 1, static_cast<uint32_t>(BS), 1};
    CUtensorMap tm;
    if (!encode_tmap_16_nd(&tm, cache, 4, dims, strides, box, std::is_same<T, __nv_bfloat16>::value, true))
        return cudaErrorNotSupported;
    auto kernel = prefix_tc_kernel<T, HD>;
    constexpr size_t smem = Smem<HD>::kTotal;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.ctas_per_kv * a.n_kv)), dim3(kThreads), smem, s, pdl, 1,
                         a, tm);
}

// ------------------------------------------------------------------ merge
// CTA = one output row (request, query head). Its parts are the prefix's records, unless the request
// does not reach past the prefix's whole pages (then its own part holds all of its tokens), and its own
// splits' records. Warp w takes records w, w + warps, ... and the warps' sums meet in shared memory, in a
// fixed order.
constexpr int kMergeWarps = 4;
template <typename T, int HD>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(PrefixArgs a) {
    constexpr int V = HD / 32;  // outputs per lane
    __shared__ float s_m[kMergeWarps], s_l[kMergeWarps], s_o[kMergeWarps][HD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t head = blockIdx.x;
    const int64_t b = head / (a.n_kv * a.group);
    const int h = static_cast<int>(head - b * a.n_kv * a.group);
    const int kvh = h / a.group, g = h - kvh * a.group;
    pdl_enter();
    int64_t len = a.seq_lens[b];
    len = len < 0 ? 0 : (len > a.cap ? a.cap : len);
    const int64_t row = b * a.group + g;
    const int tile = static_cast<int>(row / kRows);
    int recs = tile < 2 * a.pair_blocks ? a.pair_splits : 2 * a.single_splits;
    if (len < whole_pages(a) * a.block_size) recs = 0;
    const int64_t first = (static_cast<int64_t>(kvh) * a.rows + row) * a.records;
    const float* tail = a.tail + (b * a.n_kv + kvh) * a.tail_splits * (16 + 8 * HD);
    const int all = recs + a.tail_splits;
    auto stat = [&](int i) -> float2 {
        if (i < recs) return a.part_ml[first + i];
        const float* t = tail + (i - recs) * (16 + 8 * HD);
        return make_float2(t[g], t[8 + g]);
    };
    float M = -INFINITY;
    for (int i = threadIdx.x; i < all; i += blockDim.x) M = fmaxf(M, stat(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) s_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) M = fmaxf(M, s_m[k]);
    float den = 0.0f, acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int i = warp; i < all; i += kMergeWarps) {
        const float2 ml = stat(i);
        // a part without a token that counts has no sum (NaN among its scores leaves one that is NaN)
        if (ml.x == -INFINITY && ml.y == 0.0f) continue;
        const float e = ml.x == -INFINITY ? 1.0f : ex2(ml.x - M);
        den = fmaf(e, ml.y, den);
        const float* o = i < recs ? a.part_o + (first + i) * HD : tail + (i - recs) * (16 + 8 * HD) + 16 + g * HD;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(e, o[lane + 32 * k], acc[k]);
    }
    if (lane == 0) s_l[warp] = den;
#pragma unroll
    for (int k = 0; k < V; ++k) s_o[warp][lane + 32 * k] = acc[k];
    __syncthreads();
    den = 0.0f;
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) den += s_l[k];
    T* out = static_cast<T*>(a.out) + b * a.os + static_cast<int64_t>(h) * HD;
    for (int d = threadIdx.x; d < HD; d += blockDim.x) {
        float num = 0.0f;
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) num += s_o[k][d];
        out[d] = from_f32<T>(den != 0.0f ? num / den : 0.0f);
    }
}

template <typename T>
cudaError_t merge_typed(const PrefixArgs& a, int head_dim, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.B * a.n_kv * a.group)), block(kMergeWarps * 32);
    switch (head_dim) {
        case 64: return launch_kernel(merge_kernel<T, 64>, grid, block, 0, s, true, 1, a);
        case 128: return launch_kernel(merge_kernel<T, 128>, grid, block, 0, s, true, 1, a);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace prefix

size_t prefix_tc_smem(int head_dim) { return head_dim == 64 ? prefix::Smem<64>::kTotal : prefix::Smem<128>::kTotal; }

cudaError_t launch_prefix_tc(const PrefixArgs& a, const void* cache, int head_dim, int dtype, bool pdl, cudaStream_t s) {
    if (dtype == DT_BF16)
        return head_dim == 64 ? prefix::launch_tc<__nv_bfloat16, 64>(a, cache, pdl, s)
                              : prefix::launch_tc<__nv_bfloat16, 128>(a, cache, pdl, s);
    return head_dim == 64 ? prefix::launch_tc<__half, 64>(a, cache, pdl, s)
                          : prefix::launch_tc<__half, 128>(a, cache, pdl, s);
}

cudaError_t launch_prefix_merge(const PrefixArgs& a, int head_dim, int dtype, cudaStream_t s) {
    switch (dtype) {
        case DT_F16: return prefix::merge_typed<__half>(a, head_dim, s);
        case DT_BF16: return prefix::merge_typed<__nv_bfloat16>(a, head_dim, s);
        default: return prefix::merge_typed<float>(a, head_dim, s);
    }
}

// Bounded waits of this file's kernels that ran out (the counter in tma.cuh is per translation unit).
unsigned int prefix_wait_timeouts() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return v;
}

}  // namespace sra

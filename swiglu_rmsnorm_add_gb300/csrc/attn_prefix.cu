// Attention of a decode batch over the prefix that its requests share: the prefix's K and V are read
// for all requests together.
//
// For one KV head the queries of all requests (rows = B * G, G query heads per KV head) meet the same
// K and V, so S = Q K^T and O = P V are matrix products of up to some thousand rows with the prefix's
// tokens: 4 * rows * head_dim operations per token against 4 * head_dim bytes, tensor-core work from
// about 280 rows on. prefix_tc_kernel below does them on the fifth-generation tensor cores; each
// request's own tokens go through tail_kernel of attn.cu (fp32: its decode_kernel; launch_prefix_tail), and
// merge_kernel joins the parts: with (m_i, l_i, o_i) the maximum, sum of exponentials and weighted V of part i,
// out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i, M = max m_i.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace sra {
namespace prefix {

constexpr int kTok = 64;            // tokens of a K / V tile
constexpr int kRows = 128;          // query rows of a tile (the MMA's M)
constexpr int kThreads = 384;       // producer, MMA issuer, two warps that help to set up; two softmax warpgroups
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.0f;    // powers of two that a maximum may rise before its base moves, see softmax below

template <int HD>
struct Smem {
    static constexpr int kHalves = HD / 64;
    static constexpr int kHalfBytes = kTok * 128;              // 64 dims of a K or V tile's rows
    static constexpr int kTileBytes = kHalves * kHalfBytes;    // a K or V tile
    static constexpr int kQHalf = kRows * 128, kQBytes = kHalves * kQHalf;
    // head_dim 256: one row tile, its streams take a half of V's dims each (and compute the same S and P)
    static constexpr bool kSplitV = HD > 128;
    static constexpr int kDims = kSplitV ? 128 : HD;           // of a stream's O
    static constexpr int kQTiles = kSplitV ? 1 : 2;
    // K or V tiles in flight; what is left of an SM's shared memory takes a CTA of the tail kernel (attn.cu)
    // for head_dim 64 and 128
    static constexpr int kStages = HD == 64 ? 10 : 5;
    // a single block has one Q tile, whose streams have half of the stages each
    static constexpr int kOwn = kSplitV ? 0 : (kStages + kQBytes / kTileBytes) / 2;
    static constexpr int kBars = kSplitV ? kStages : 2 * kOwn;
    static constexpr size_t kTotal =
        1024 + kQTiles * static_cast<size_t>(kQBytes) + kStages * static_cast<size_t>(kTileBytes);
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 in a 64-bit register: one instruction per pair, each half rounded as the plain operation.
__device__ __forceinline__ uint64_t f32x2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// What CTA `c` of a KV head's works on (RPB: query rows of a pair block): its rows, which follow from
// `c`, and its tiles, which follow from the prefix's length.
struct Work {
    int row0;      // first query row
    bool pair;     // two row tiles on the same K / V tiles, or one row tile on two K / V tiles at a time
    int split, splits;
    int t0 = 0, n = 0;  // K / V tiles
    __device__ __forceinline__ void cut(int64_t tiles) {
        const int64_t b = tiles * split / splits, e = tiles * (split + 1) / splits;
        t0 = static_cast<int>(b);
        n = static_cast<int>(e - b);
    }
};
template <int RPB>
__device__ __forceinline__ Work rows_of(const PrefixArgs& a, int c) {
    Work w;
    if (c < a.pair_blocks * a.pair_splits) {
        const int blk = c / a.pair_splits;
        w.split = c - blk * a.pair_splits, w.splits = a.pair_splits;
        w.pair = true;
        w.row0 = blk * RPB;
    } else {
        w.split = c - a.pair_blocks * a.pair_splits, w.splits = a.single_splits;
        w.pair = false;
        w.row0 = a.pair_blocks * RPB;
    }
    return w;
}
// Whole pages of the prefix, and its K / V tiles.
__device__ __forceinline__ int64_t whole_pages(const PrefixArgs& a) {
    const int64_t P = *a.plen, cap = a.pblocks * a.block_size;
    return (P < 0 ? 0 : (P > cap ? cap : P)) / a.block_size;
}

// A place in a ring of tiles: its stage, and the parity of the phase in which that is filled. A pair's streams
// both use every tile of one ring. A single block's streams use every other tile, each in a ring of its
// own: whoever waits for a stage's phase has waited for the phase before it, as a wait on a parity requires.
// (In one ring a stage could pass from one stream to the other, which then took a tile that was still on its
// way for the one after it.) A ring carries K of its tile 0, then K of tile i + 1 and V of tile i for i = 0, 1, ...
struct Place {
    int stage, first, end, phase = 0;
    __device__ __forceinline__ Place(int first, int stages) : stage(first), first(first), end(first + stages) {}
    __device__ __forceinline__ void next() {
        if (++stage == end) stage = first, phase ^= 1;
    }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    float f[2] = {x, y};
    return Elem<T>::pack_word(f);
}

// A CTA takes 256 query rows (two row tiles, one per softmax warpgroup: "streams") through its split's
// K / V tiles of 64 tokens, or 128 rows with the streams on alternate tiles. Per stream and tile:
// S = Q K^T (fp32, tensor memory), the softmax warpgroup reads it (a thread is a row), frees it, and
// writes P (16-bit) back to tensor memory, and O += P V takes P from there.
// Tensor memory, 512 columns: S 64 per stream, P 32 per stream and buffer (two), O head_dim per stream.
// S, P and O never share columns, so the next tile's S needs only that this one's has been read: the
// product S runs under the softmax, and the tensor cores have work of one stream while the other's
// softmax is under way. (With P over S in 128-token tiles the chain S -> softmax -> P V -> next S has no
// such overlap within a stream: measured 4700 clocks per 128 tokens of both streams, against 2070 of tensor-core
// work, in a form whose one warp also issued for both streams from a branch of one lane, at 75 clocks an instruction;
// what the tile alone costs or gives has not been measured apart from that.
// The price is that S in tiles of 64 tokens reads Q from shared memory twice as often: 48 clocks per
// K step of 16 instead of 2 x 32, shared-memory bandwidth, so a tile cannot run above 81 % of the peak.)
// With head_dim 256 O alone would fill tensor memory for two row tiles, so a CTA has one, and its streams take half
// of V's dims each with an S and P of their own, which are the same: S is computed twice (62 % of the work is needed
// work; batch 100 x 12000 with 16 / 2 heads 57 us, the needed products 10.3 at the measured peak). One O of 256
// columns beside two S and two P, 448 columns in all, would fit and need S once; it has not been built.
template <typename T, int HD>
__global__ void __maxnreg__(120) prefix_tc_kernel(PrefixArgs a, const __grid_constant__ CUtensorMap tmC) {
    using L = Smem<HD>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t kS = 0, kP = 128, kO = 256;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char* qs = smem;                              // two Q tiles (head_dim 256: one)
    __shared__ uint64_t full[L::kBars], empty[L::kBars], s_full[2], s_free[2], p_full[2][2], pv_done[2][2];
    __shared__ uint32_t tmem_base;
    __shared__ int s_ragged;
    __shared__ float2 s_ml[kRows];  // a single block's stream 1: maxima and sums
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        // a pair's streams both release a tile
        const bool pair = static_cast<int>(blockIdx.x) % a.ctas_per_kv < a.pair_blocks * a.pair_splits;
        for (int i = 0; i < L::kBars; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], pair ? 2 : 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1), mbar_init(&s_free[x], 4);
            for (int b = 0; b < 2; ++b) mbar_init(&p_full[x][b], 4), mbar_init(&pv_done[x][b], 1);
        }
        mbar_init_fence();
        s_ragged = 0;
    }
    if (warp == 0) {
        tc::alloc(&tmem_base, kTmemCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = tmem_base;
    const int kvh = blockIdx.x / a.ctas_per_kv;
    Work w = rows_of<L::kQTiles * kRows>(a, blockIdx.x - kvh * a.ctas_per_kv);
    unsigned char* ring = smem + (w.pair ? L::kQTiles : 1) * L::kQBytes;  // K / V tiles
    auto ring_of = [&](int x) { return w.pair ? Place(0, L::kStages) : Place(x * L::kOwn, L::kOwn); };
    // The threads that set up (all but the producers) ask for the query rows first, the prefix's length after. A
    // thread's 16-byte chunks share their place in the row and lie kStep rows apart: one division, then steps.
    const bool producer = warp == 0 || warp == 3;
    constexpr int kSetup = kThreads - 64, kChunks = HD / 8, kStep = kSetup / kChunks;
    constexpr int kEach = (L::kQTiles * kRows * kChunks + kSetup - 1) / kSetup;
    static_assert(kSetup % kChunks == 0, "a thread's chunks share a column");
    const int setup_tid = threadIdx.x - (warp < 3 ? 32 : 64);
    const int chunk = setup_tid % kChunks, r0 = setup_tid / kChunks, count = (w.pair ? L::kQTiles : 1) * kRows;
    uint4 qv[kEach];
    pdl_enter();
    if (!producer) {
        const int dg = kStep % a.group;
        int g = (w.row0 + r0) % a.group;
        const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>((w.row0 + r0) / a.group) * a.qs +
                       (kvh * a.group + g) * HD + chunk * 8;
        const int64_t step = static_cast<int64_t>(kStep / a.group) * a.qs + dg * HD, wrap = a.qs - a.group * HD;
        const int rows = count < a.rows - w.row0 ? count : a.rows - w.row0;
        auto advance = [&]() {
            src += step;
            if ((g += dg) >= a.group) g -= a.group, src += wrap;
        };
        if (a.q16) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {  // all loads in flight before the first store
                qv[e] = make_uint4(0u, 0u, 0u, 0u);
                if (r0 + e * kStep < rows) qv[e] = *reinterpret_cast<const uint4*>(src);
                advance();
            }
        } else {
#pragma unroll 1
            for (int e = 0; e < kEach; ++e) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (r0 + e * kStep < rows) {
                    const unsigned short* h = reinterpret_cast<const unsigned short*>(src);
                    u.x = h[0] | static_cast<uint32_t>(h[1]) << 16, u.y = h[2] | static_cast<uint32_t>(h[3]) << 16;
                    u.z = h[4] | static_cast<uint32_t>(h[5]) << 16, u.w = h[6] | static_cast<uint32_t>(h[7]) << 16;
                }
                advance();
#pragma unroll
                for (int k = 0; k < kEach; ++k)
                    if (k == e) qv[k] = u;
            }
        }
    }
    const int64_t pages = whole_pages(a);
    const int ppt = kTok >> (__ffs(a.block_size) - 1);  // pages of a tile
    w.cut((pages + ppt - 1) / ppt);
    const int tpr = w.pair ? 1 : 2;  // tiles per round
    const int n0 = w.pair ? w.n : (w.n + 1) / 2, n1 = w.pair ? w.n : w.n / 2;  // tiles of the streams
    bool dead = false;  // a bounded wait ran out (counted): this thread waits no more
    auto wait = [&](uint64_t* bar, int phase) {
        if (!dead) dead = !mbar_wait(bar, static_cast<uint32_t>(phase & 1));
        __syncwarp();  // tensor-memory accesses behind it are a whole warp's
    };

    if (producer) {
        // producers: a tile is a box of 64 dims x block_size tokens per page and half, dealt to two warps
        // (a warp issues a box in about 80 clocks). A page past the prefix, or an entry that is no page, is
        // copied from past the cache's end: zeros. The page entries are read 32 at a time (lane k: entry k
        // of the group), a group ahead of their use and apart for K and V, so no copy waits for the table.
        const int ppt_log2 = __ffs(ppt) - 1, boxes = ppt * L::kHalves;
        const int box = lane * 2 + (warp == 0 ? 0 : 1), half = box >> ppt_log2, p = box & (ppt - 1);
        unsigned char* dst = ring + half * L::kHalfBytes + p * a.block_size * 128;
        Place at0 = ring_of(0), at1 = ring_of(1);  // at1: a single block's odd tiles
        int group[2] = {-1, -1};
        int32_t cur[2] = {-1, -1}, next[2] = {-1, -1};
        auto entries = [&](int g) -> int32_t {
            const int64_t j = static_cast<int64_t>(w.t0) * ppt + static_cast<int64_t>(g) * 32 + lane;
            return j < pages ? a.ptable[j] : -1;
        };
        auto load = [&](int t, int plane, int32_t& c, int32_t& nx, int& g) {
            const int first = t << ppt_log2;
            if (first >> 5 != g) {
                c = g < 0 ? entries(0) : nx;
                ++g;
                nx = entries(g + 1);
            }
            int64_t blk = __shfl_sync(0xffffffffu, c, (first + p) & 31);
            if (blk < 0 || blk >= a.num_blocks) blk = a.num_blocks;
            const bool odd = !w.pair && (t & 1);
            const int stage = odd ? at1.stage : at0.stage;
            wait(&empty[stage], (odd ? at1.phase : at0.phase) ^ 1);  // (passes at once the first time round)
            if (warp == 0 && lane == 0) mbar_arrive_expect_tx(&full[stage], L::kTileBytes);
            if (box < boxes)
                tma_load_4d(dst + stage * L::kTileBytes, &tmC, half * 64, kvh, static_cast<int>(blk * a.block_size), plane,
                            &full[stage]);
            __syncwarp();
            if (odd)
                at1.next();
            else
                at0.next();
        };
        auto load_k = [&](int t) { load(t, 0, cur[0], next[0], group[0]); };
        auto load_v = [&](int t) { load(t, 1, cur[1], next[1], group[1]); };
        for (int t = 0; t < tpr && t < w.n; ++t) load_k(t);
        for (int r = 0; r < n0; ++r) {
            for (int t = (r + 1) * tpr; t < (r + 2) * tpr && t < w.n; ++t) load_k(t);
            for (int t = r * tpr; t < (r + 1) * tpr && t < w.n; ++t) load_v(t);
        }
    } else {
        // the query rows into shared memory, swizzled as a TMA copy would leave them (rows past the last are
        // zero), and whether every page of this CTA's tiles counts
        bool bad = false;
        for (int64_t k = setup_tid; k < static_cast<int64_t>(w.n) * ppt; k += kSetup) {
            const int64_t j = static_cast<int64_t>(w.t0) * ppt + k;
            const int32_t e = j < pages ? a.ptable[j] : -1;
            bad |= e < 0 || e >= a.num_blocks;
        }
        if (bad) s_ragged = 1;
        const uint32_t flip = a.negate ? 0x80008000u : 0u;
        auto place = [&](int r) {
            return reinterpret_cast<uint4*>(qs + (r / kRows) * L::kQBytes + (chunk / 8) * L::kQHalf + r % kRows * 128 +
                                            (((chunk & 7) ^ (r & 7)) * 16));
        };
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int r = r0 + e * kStep;
            if (r < count) *place(r) = make_uint4(qv[e].x ^ flip, qv[e].y ^ flip, qv[e].z ^ flip, qv[e].w ^ flip);
        }
        if (a.zero) {  // a query element counts as 0 times itself: 0, or NaN for infinities and NaN
            auto half = [](uint32_t h) -> uint32_t {
                constexpr uint32_t kExp = kBf16 ? 0x7f80u : 0x7c00u;
                return (h & kExp) == kExp ? 0x7fffu : 0u;
            };
            auto word = [&](uint32_t w) { return half(w & 0xffffu) | half(w >> 16) << 16; };
#pragma unroll 1
            for (int r = r0; r < count; r += kStep) {  // (its own chunks, as stored above)
                const uint4 u = *place(r);
                *place(r) = make_uint4(word(u.x), word(u.y), word(u.z), word(u.w));
            }
        }
        fence_proxy_async();  // before the tensor core reads them
        asm volatile("bar.sync 1, %0;" ::"r"(kSetup) : "memory");
    }

    if (warp == 1 || warp == 2) {
        // MMA issuers, one warp per stream: the whole warp runs the loop, one lane issues. (Issued from a branch
        // of one lane, whose descriptors the compiler must move to uniform registers one by one, an
        // instruction took 75 clocks, more than the product itself. A wait or a commit costs about
        // 120 clocks, so one warp for both streams was busy for 2300 clocks per tile of both, against
        // 1290 of tensor-core work.)
        const int x = warp - 1, n = x == 0 ? n0 : n1;
        constexpr uint32_t kIdescS = tc::idesc_f16(kBf16, kRows, kTok);
        constexpr uint32_t kIdescO = tc::idesc_f16(kBf16, kRows, L::kDims) | tc::kTransposeB;
        const uint32_t elected = tc::elect();
        const uint32_t q = tc::sdesc_lo(qs, 16) + (w.pair && !L::kSplitV ? x : 0) * (L::kQBytes / 16);
        const uint32_t k_lo = tc::sdesc_lo(ring, 16), v_lo = tc::sdesc_lo(ring + (L::kSplitV ? 2 * x * L::kHalfBytes : 0), L::kHalfBytes);
        const uint32_t tS = tmem + kS + x * kTok, tP = tmem + kP + x * 64, tO = tmem + kO + x * L::kDims;
        Place at = ring_of(x);
        auto take = [&]() -> int {
            const int stage = at.stage;
            wait(&full[stage], at.phase);
            tc::fence_after();
            at.next();
            return stage;
        };
        auto qk = [&]() {
            const int stage = take();
            const uint32_t k = k_lo + stage * (L::kTileBytes / 16);
#pragma unroll
            for (int e = 0; e < HD / 16; ++e)
                tc::mma_f16_ss(elected, tS, q + (e / 4) * (L::kQHalf / 16) + (e % 4) * 2,
                               k + (e / 4) * (L::kHalfBytes / 16) + (e % 4) * 2, kIdescS, e > 0);
            tc::commit(elected, &s_full[x]);
            tc::commit(elected, &empty[stage]);
        };
        if (n > 0) qk();
        for (int i = 0; i < n; ++i) {
            if (i + 1 < n) {
                wait(&s_free[x], i);
                qk();
            }
            wait(&p_full[x][i & 1], i >> 1);
            const int stage = take();
            const uint32_t v = v_lo + stage * (L::kTileBytes / 16), p = tP + (i & 1) * 32;
#pragma unroll
            for (int e = 0; e < kTok / 16; ++e)
                tc::mma_f16_ts(elected, tO, p + 8 * e, v + e * 128, kIdescO, i > 0 || e > 0);
            tc::commit(elected, &pv_done[x][i & 1]);
            tc::commit(elected, &empty[stage]);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // softmax: thread = query row of stream x. The base m of the exponents (base 2, scaled) is moved only
        // when a tile's maximum leaves the kRescale powers of two that the last move left room for: o and l are
        // sums of 2^(s - m) for one m, so any m will do as long as nothing overflows or is lost, and O in tensor
        // memory is scaled seldom. bf16 has fp32's exponents, for P and for V: there m is put 8 above the maximum, so
        // that no p is above 1 and O stays within the sum of |V|. fp16 has few: there m is put 7 below the maximum (p up to
        // 2^15 of V up to 2^16, far from fp32's end), so that probabilities down to 2^-21 of the largest are
        // normal numbers and those to 2^-32 are not lost.
        constexpr float kUnder = kBf16 ? -kRescale : kUnderMax<T>;
        const int x = (warp - 4) >> 2, quarter = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lanes + kS + x * kTok, tP = tmem + lanes + kP + x * 64,
                       tO = tmem + lanes + kO + x * L::kDims;
        const int n = x == 0 ? n0 : n1;
        const bool ragged = s_ragged != 0;
        const int bs_log2 = __ffs(a.block_size) - 1;
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.0f;
        for (int i = 0; i < n; ++i) {
            wait(&s_full[x], i);
            tc::fence_after();
            uint32_t v[2][32];
            tc::ld32(tS, v[0]);
            tc::ld32(tS + 32, v[1]);
            tc::wait_ld();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[x]);  // this warp has read its rows of S
            if (ragged) {
                // some page of the CTA's range does not count: its tokens' scores become -inf
                const int64_t j = static_cast<int64_t>(w.t0 + (w.pair ? i : 2 * i + x)) * ppt + lane;
                const int32_t e = lane < ppt && j < pages ? a.ptable[j] : -1;
                const unsigned valid = __ballot_sync(0xffffffffu, e >= 0 && e < a.num_blocks);
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (!((valid >> (k >> bs_log2)) & 1u)) v[k / 32][k % 32] = __float_as_uint(-INFINITY);
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 64; k += 8)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    top[u] = fmaxf(fmaxf(top[u], __uint_as_float(v[k / 32][k % 32 + u])),
                                   __uint_as_float(v[k / 32][k % 32 + 4 + u]));
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
            if (i == 0) {
                m = mx - kUnder;
            } else {
                const bool move = mx > m + (kUnder + kRescale);
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? ex2(m - (mx - kUnder)) : 1.0f;
                    if (move) l *= f, m = mx - kUnder;
                    wait(&pv_done[x][(i - 1) & 1], (i - 1) / 2);
                    tc::fence_after();
#pragma unroll 1
                    for (int d = 0; d < L::kDims; d += 16) {
                        uint32_t o[16];
                        tc::ld16(tO + d, o);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tc::st16(tO + d, o);
                    }
                    tc::wait_st();
                }
            }
            // p = 2^(c s - m), summed in fp32, rounded once to T: a relative error of up to half a step of T
            // per probability, so that O is off by about as much again as its own rounding to T costs (batch 64 and
            // 256, bf16: 2.3e-3 of the exact result's norm where that rounding alone is 1.7e-3). Pairs of fp32 go
            // through the packed multiply-add and add.
            const float base = m == -INFINITY ? 0.0f : m;
            const uint64_t c2 = f32x2(c, c), b2 = f32x2(-base, -base);
            uint64_t part[2] = {0, 0};  // (+0, +0)
            uint32_t pk[32];
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                float p0, p1;
                split2(fma2(f32x2(__uint_as_float(v[k / 32][k % 32]), __uint_as_float(v[k / 32][k % 32 + 1])), c2, b2), p0, p1);
                p0 = ex2(p0), p1 = ex2(p1);
                part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], f32x2(p0, p1));
                pk[k / 2] = pack2<T>(p0, p1);
            }
            if (i >= 2) {  // the product that read this buffer of P is done
                wait(&pv_done[x][i & 1], i / 2 - 1);
                tc::fence_after();
            }
            tc::st32(tP + (i & 1) * 32, pk);
            float s0, s1, s2, s3;
            split2(part[0], s0, s1);
            split2(part[1], s2, s3);
            l += (s0 + s1) + (s2 + s3);
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[x][i & 1]);
        }
        // The record of this CTA's rows: maximum, sum, O; no tile, or no token that counts, leaves a maximum of
        // -inf. The streams of a single block, two parts of the same rows, are merged first. O goes out through
        // shared memory, over the tiles, which are done with: blocks of 32 columns x 128 rows, their 16-byte
        // chunks XOR-swizzled by row, so that the threads of a warp, a row each, meet different banks, and so do
        // those that then write a row together. (128 KB take 4100 clocks, 32 bytes a clock, what an SM stores;
        // straight from registers, 16 bytes per row and instruction, 10900; by TMA 4500.)
        constexpr int kBlock = kRows * 128, kBlocks = L::kDims / 32;
        const int rr = quarter * 32 + lane;
        unsigned char* mine = smem + x * kBlocks * kBlock + rr * 128;
        auto at16 = [&](int c) { return (c >> 3) * kBlock + (((c & 7) ^ (rr & 7)) << 4); };  // 16-byte chunk c of the row
        if (n > 0) {
            wait(&pv_done[x][(n - 1) & 1], (n - 1) / 2);
            tc::fence_after();
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");  // both streams' products are done: the tiles may go
        if (w.pair || x == 1) {
            if (n > 0) {
#pragma unroll 1
                for (int d = 0; d < L::kDims; d += 32) {
                    uint32_t v[32];
                    tc::ld32(tO + d, v);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(mine + at16(d / 4 + k)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            }
        }
        if (!w.pair) {
            if (x == 1) s_ml[rr] = make_float2(m, l);
            asm volatile("bar.sync 2, 256;" ::: "memory");
            if (x == 0 && n > 0) {
                const unsigned char* other = mine + kBlocks * kBlock;
                const float2 o = s_ml[rr];
                const bool some = n1 > 0 && !(o.x == -INFINITY && o.y == 0.0f);
                const float M = some ? fmaxf(m, o.x) : m;
                // a part without weight is not read: it may hold anything
                const float wa = m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : ex2(m - M);
                const float wb = some ? (o.x == -INFINITY ? 1.0f : ex2(o.x - M)) : 0.0f;
                l = wa * l + (some ? wb * o.y : 0.0f);
                m = M;
#pragma unroll 1
                for (int d = 0; d < L::kDims; d += 32) {
                    uint32_t v[32];
                    tc::ld32(tO + d, v);
                    tc::wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (some) q = *reinterpret_cast<const float4*>(other + at16((d + k) / 4));
                        float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            f[u] = (wa != 0.0f ? wa * __uint_as_float(v[k + u]) : 0.0f) + (some ? wb * f[u] : 0.0f);
                        *reinterpret_cast<float4*>(mine + at16((d + k) / 4)) = make_float4(f[0], f[1], f[2], f[3]);
                    }
                }
            }
        }
        if (w.pair || x == 0) {
            const int first = w.row0 + (w.pair && !L::kSplitV ? x * kRows : 0), r = first + rr;
            const int64_t rec = static_cast<int64_t>(kvh) * a.records + w.split;
            if (r < a.rows && (!L::kSplitV || x == 0)) a.part_ml[rec * a.rows + r] = make_float2(m, l);
            if (n > 0) {
                // a warp writes its own 32 rows, a row per instruction
                __syncwarp();
                constexpr int kLanes = L::kDims / 4;  // 16-byte chunks of a row
                const int row0 = quarter * 32 + lane / kLanes, c = lane % kLanes;
                const unsigned char* from = smem + x * kBlocks * kBlock + (c >> 3) * kBlock;
                float* to = a.part_o + (rec * a.rows + first) * HD + (L::kSplitV ? x * L::kDims : 0) + c * 4;
#pragma unroll 8
                for (int k = 0; k < 32; k += 32 / kLanes) {
                    const int row = row0 + k;
                    if (first + row < a.rows)
                        *reinterpret_cast<uint4*>(to + static_cast<int64_t>(row) * HD) =
                            *reinterpret_cast<const uint4*>(from + row * 128 + (((c & 7) ^ (row & 7)) << 4));
                }
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
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
    // all of the SM's shared memory, so that a CTA of the tail kernel finds room beside this one's
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_once(kernel, smem, true, &done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.ctas_per_kv * a.n_kv)), dim3(kThreads), smem, s, pdl, 1,
                         a, tm);
}

// ------------------------------------------------------------------ fp32
// The same cut for fp32, on the CUDA cores (the tensor cores have no fp32 products. Three bf16 parts of each operand
// and the six products of them that matter would be a sixth of the bf16 rate, 317 TFLOP/s at the measured peak, more
// than the CUDA cores have: not built, and so not known is whether that holds the error. Batch 100 x 4800, 16 / 2
// heads of 128: 171 us, 23 TFLOP/s): a CTA takes 64 query rows through its split's K / V tiles of 64
// tokens. A thread holds 4 rows x 4 tokens of S and 4 rows x head_dim / 16 dims of O, so that a load of 16
// bytes from shared memory feeds 5 (S) to 6 (O) FMAs a lane; the rows of its operands are padded by 16 bytes, so
// that the lanes of a load meet different banks. K of the next tile is copied under P V, V under Q K^T.
constexpr int kF32Rows = 64, kF32Tok = 64, kF32Threads = 256;
template <int HD>
struct SmemF32 {
    static constexpr int kRow = HD + 4;        // floats of a Q, K or V row
    static constexpr int kPRow = kF32Tok + 4;  // floats of a P row
    static constexpr size_t kTotal = (static_cast<size_t>(kF32Rows + 2 * kF32Tok) * kRow + kF32Rows * kPRow) * 4;
};

template <int HD>
__global__ void __launch_bounds__(kF32Threads) prefix_f32_kernel(PrefixArgs a, const float* cache) {
    using L = SmemF32<HD>;
    constexpr int RS = L::kRow, PS = L::kPRow, J = HD / 64, CPR = HD / 4;
    extern __shared__ __align__(16) float sm[];
    float *qs = sm, *ks = qs + kF32Rows * RS, *vs = ks + kF32Tok * RS, *ps = vs + kF32Tok * RS;
    __shared__ int page[2][kF32Tok / 8];
    const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;  // rows 4 tr + i; tokens tc + 16 j, dims 4 tc + 64 j
    pdl_enter();
    const int kvh = blockIdx.x / a.ctas_per_kv;
    const int64_t pages = whole_pages(a);
    const int bs_log2 = __ffs(a.block_size) - 1, ppt = kF32Tok >> bs_log2;
    Work w = rows_of<kF32Rows>(a, blockIdx.x - kvh * a.ctas_per_kv);
    w.cut((pages + ppt - 1) / ppt);
    const int64_t tok_stride = static_cast<int64_t>(a.n_kv) * HD, v_plane = a.num_blocks * a.block_size * tok_stride;
    // the pages of tile t (-1: does not count), then its rows of a plane, zero where they do not count
    auto find = [&](int t) {
        if (tid < ppt) {
            const int64_t j = static_cast<int64_t>(w.t0 + t) * ppt + tid;
            const int32_t e = j < pages ? a.ptable[j] : -1;
            page[t & 1][tid] = e >= 0 && e < a.num_blocks ? e : -1;
        }
    };
    auto copy = [&](float* dst, int t, int64_t plane) {
        for (int i = tid; i < kF32Tok * CPR; i += kF32Threads) {
            const int r = i / CPR, c = i % CPR, e = page[t & 1][r >> bs_log2];
            const float* src = cache + plane +
                               ((static_cast<int64_t>(e) << bs_log2) + (r & (a.block_size - 1))) * tok_stride + kvh * HD + c * 4;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + r * RS + c * 4)),
                         "l"(e >= 0 ? src : cache), "r"(e >= 0 ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (w.n > 0) {
        find(0);
        for (int i = tid; i < kF32Rows * HD; i += kF32Threads) {
            const int r = i / HD, d = i % HD, row = w.row0 + r;
            float v = 0.0f;
            if (row < a.rows) {
                const int b = row / a.group, g = row - b * a.group;
                v = static_cast<const float*>(a.q)[b * a.qs + (kvh * a.group + g) * HD + d];
            }
            qs[r * RS + d] = a.zero ? 0.0f * v : a.negate ? -v : v;
        }
        __syncthreads();
        copy(ks, 0, 0);
    }
    float m[4], l[4], o[4][4 * J];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4 * J; ++j) o[i][j] = 0.0f;
    }
    for (int t = 0; t < w.n; ++t) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // K has landed; everyone is done with V and P of the tile before
        copy(vs, t, v_plane);
        if (t + 1 < w.n) find(t + 1);
        float s[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < HD; d += 4) {
            float4 qv[4], kv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(qs + (4 * tr + i) * RS + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(ks + (tc + 16 * j) * RS + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                    s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                    s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                    s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
                }
        }
        // the running softmax: a row's 64 scores lie in 16 lanes
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = page[t & 1][(tc + 16 * j) >> bs_log2] >= 0 ? s[i][j] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float now = fmaxf(m[i], mx), base = now == -INFINITY ? 0.0f : now;
            const float f = now == -INFINITY ? 1.0f : exp2f(m[i] - now);
            m[i] = now;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                ps[(4 * tr + i) * PS + tc + 16 * j] = p;
                sum += p;
            }
            l[i] = l[i] * f + sum;  // this lane's tokens' part
#pragma unroll
            for (int j = 0; j < 4 * J; ++j) o[i][j] *= f;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // V has landed, P is written, everyone is done with K
        if (t + 1 < w.n) copy(ks, t + 1, 0);
#pragma unroll 2
        for (int k = 0; k < kF32Tok; k += 4) {
            float4 pv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4*>(ps + (4 * tr + i) * PS + k);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(vs + (k + u) * RS + 4 * tc + 64 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = u == 0 ? pv[i].x : u == 1 ? pv[i].y : u == 2 ? pv[i].z : pv[i].w;
                        o[i][4 * j] = fmaf(p, v.x, o[i][4 * j]);
                        o[i][4 * j + 1] = fmaf(p, v.y, o[i][4 * j + 1]);
                        o[i][4 * j + 2] = fmaf(p, v.z, o[i][4 * j + 2]);
                        o[i][4 * j + 3] = fmaf(p, v.w, o[i][4 * j + 3]);
                    }
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = w.row0 + 4 * tr + i;
#pragma unroll
        for (int x = 1; x < 16; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        if (row >= a.rows) continue;
        const int64_t at = (static_cast<int64_t>(kvh) * a.records + w.split) * a.rows + row;
        if (tc == 0) a.part_ml[at] = make_float2(m[i], l[i]);
#pragma unroll
        for (int j = 0; j < J; ++j)
            *reinterpret_cast<float4*>(a.part_o + at * HD + 4 * tc + 64 * j) =
                make_float4(o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]);
    }
}

template <int HD>
cudaError_t launch_f32(const PrefixArgs& a, const void* cache, bool pdl, cudaStream_t s) {
    auto kernel = prefix_f32_kernel<HD>;
    constexpr size_t smem = SmemF32<HD>::kTotal;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = set_smem_once(kernel, smem, false, &done);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.ctas_per_kv * a.n_kv)), dim3(kF32Threads), smem, s, pdl, 1,
                         a, static_cast<const float*>(cache));
}

// ------------------------------------------------------------------ merge
// CTA = one output row (request, query head). Its parts are the prefix's records, unless the request
// does not reach past the prefix's whole pages (then its own part holds all of its tokens), and its own
// records. Warp w takes parts w, w + warps, ..., kBatch of them loaded at a time (statistics and values
// together, one round trip), with a running maximum of its own; the warps' sums meet in shared memory, in a
// fixed order.
constexpr int kMergeWarps = 4, kBatch = 4;
template <typename T, int HD>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_kernel(PrefixArgs a) {
    constexpr int V = HD / 32;  // outputs per lane
    __shared__ float s_m[kMergeWarps], s_l[kMergeWarps], s_o[kMergeWarps][HD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned heads = static_cast<unsigned>(a.n_kv * a.group);
    const int64_t b = blockIdx.x / heads;
    const int h = static_cast<int>(blockIdx.x % heads);
    const int kvh = h / a.group, g = h - kvh * a.group;
    pdl_enter();
    int64_t len = a.seq_lens[b];
    const bool stream = a.tail_at != nullptr;  // fp32: every split of the own tokens leaves a record
    const int part = stream ? a.tail_at[a.B] : 1, before = stream ? a.tail_at[b] : 0;
    const int64_t behind = whole_pages(a) * a.block_size;
    len = len < 0 ? 0 : (len > a.cap ? a.cap : len);
    const int64_t row = b * a.group + g;
    const int tile = static_cast<int>(row / kRows);
    int recs = tile < (HD > 128 ? 1 : 2) * a.pair_blocks ? a.pair_splits : a.single_splits;
    const int64_t lo = len >= behind ? behind : 0;
    if (len < behind) recs = 0;
    const int64_t first = static_cast<int64_t>(kvh) * a.records * a.rows + row;  // record i: i * rows further
    const float* tail = a.tail + (b * a.n_kv + kvh) * a.tail_splits * (16 + 8 * HD);
    // its own tokens' records: the parts of the tail's stream that its tiles touch
    const int tiles = static_cast<int>((len - lo + kTailTok - 1) / kTailTok);
    const int count = !stream ? a.tail_splits : tiles > 0 ? (before + tiles - 1) / max(part, 1) - before / max(part, 1) + 1 : 0;
    const int all = recs + min(max(count, 0), a.tail_splits);  // (in range whatever the lengths do meanwhile)
    float m = -INFINITY, l = 0.0f, acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    for (int i0 = warp; i0 < all; i0 += kMergeWarps * kBatch) {
        float pm[kBatch], pl[kBatch], po[kBatch][V];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kMergeWarps;
            pm[u] = -INFINITY, pl[u] = 0.0f;
            const float* o = tail;
            if (i < recs) {
                const float2 ml = a.part_ml[first + static_cast<int64_t>(i) * a.rows];
                pm[u] = ml.x, pl[u] = ml.y;
                o = a.part_o + (first + static_cast<int64_t>(i) * a.rows) * HD;
            } else if (i < all) {
                const float* t = tail + (i - recs) * (16 + 8 * HD);
                pm[u] = t[g], pl[u] = t[8 + g];
                o = t + 16 + g * HD;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) po[u][k] = i < all ? o[lane + 32 * k] : 0.0f;
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) top = fmaxf(top, pm[u]);
        const float keep = m == top ? 1.0f : ex2(m - top);  // (the first time m is -inf: 0, and l and acc are 0)
        l *= keep;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] *= keep;
        m = top;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            // a part without a token that counts has no sum, and its values are not its own (NaN among a part's
            // scores leaves a sum that is NaN)
            if (pm[u] == -INFINITY && pl[u] == 0.0f) continue;
            const float e = pm[u] == m ? 1.0f : ex2(pm[u] - m);
            l = fmaf(e, pl[u], l);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = fmaf(e, po[u][k], acc[k]);
        }
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int k = 0; k < V; ++k) s_o[warp][lane + 32 * k] = acc[k];
    __syncthreads();
    float M = -INFINITY, w[kMergeWarps], den = 0.0f;
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) M = fmaxf(M, s_m[k]);
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) {
        w[k] = s_m[k] == M ? 1.0f : ex2(s_m[k] - M);
        den = fmaf(w[k], s_l[k], den);
    }
    T* out = static_cast<T*>(a.out) + b * a.os + static_cast<int64_t>(h) * HD;
    for (int d = threadIdx.x; d < HD; d += blockDim.x) {
        float num = 0.0f;
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) num = fmaf(w[k], s_o[k][d], num);
        out[d] = from_f32<T>(den != 0.0f ? num / den : 0.0f);
    }
}

template <typename T>
cudaError_t merge_typed(const PrefixArgs& a, int head_dim, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.B * a.n_kv * a.group)), block(kMergeWarps * 32);
    switch (head_dim) {
        case 64: return launch_kernel(merge_kernel<T, 64>, grid, block, 0, s, true, 1, a);
        case 128: return launch_kernel(merge_kernel<T, 128>, grid, block, 0, s, true, 1, a);
        case 256: return launch_kernel(merge_kernel<T, 256>, grid, block, 0, s, true, 1, a);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace prefix

size_t prefix_smem(int head_dim, int dtype) {
    if (dtype == DT_F32)
        return head_dim == 64    ? prefix::SmemF32<64>::kTotal
               : head_dim == 128 ? prefix::SmemF32<128>::kTotal
                                 : prefix::SmemF32<256>::kTotal;
    return head_dim == 64 ? prefix::Smem<64>::kTotal : head_dim == 128 ? prefix::Smem<128>::kTotal : prefix::Smem<256>::kTotal;
}

template <typename T>
static cudaError_t launch_prefix_tc_typed(const PrefixArgs& a, const void* cache, int head_dim, bool pdl, cudaStream_t s) {
    switch (head_dim) {
        case 64: return prefix::launch_tc<T, 64>(a, cache, pdl, s);
        case 128: return prefix::launch_tc<T, 128>(a, cache, pdl, s);
        case 256: return prefix::launch_tc<T, 256>(a, cache, pdl, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_prefix_whole(const PrefixArgs& a, const void* cache, int head_dim, int dtype, bool pdl, cudaStream_t s) {
    if (dtype == DT_F32) {
        switch (head_dim) {
            case 64: return prefix::launch_f32<64>(a, cache, pdl, s);
            case 128: return prefix::launch_f32<128>(a, cache, pdl, s);
            case 256: return prefix::launch_f32<256>(a, cache, pdl, s);
            default: return cudaErrorInvalidValue;
        }
    }
    return dtype == DT_BF16 ? launch_prefix_tc_typed<__nv_bfloat16>(a, cache, head_dim, pdl, s)
                            : launch_prefix_tc_typed<__half>(a, cache, head_dim, pdl, s);
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

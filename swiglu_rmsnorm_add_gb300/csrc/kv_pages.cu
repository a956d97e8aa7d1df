// Pages of the paged KV cache: copying them, sharing them between rows (fork), growing,
// truncating and freeing rows (resize) and moving the live ones together (compact).
//
// The state is the caller's: block_table [R, M] and seq_lens [R] say which pages hold row r's
// tokens (the first pages(seq_lens[r]) entries, pages(L) = ceil(L / block_size)), and
// ref_counts [num_blocks] says how many rows hold a page; a page whose count is not positive
// is free. Everything a call decides follows from that state and its arguments in a fixed
// order (the lowest free page first, entries of a call in their order), so results do not
// depend on timing: counts change by integer atomics, whose order does not matter, and every
// other word has one writer.
//
// What bounds these kernels: the copies are HBM traffic (each byte read and written once; a
// page is contiguous in each plane, so threads move 16 bytes at a time, kUnroll of them in
// flight); the bookkeeping reads a few kilobytes and is bound by dependent round trips to the
// L2, so each call is one to three launches, chained by programmatic dependent launch.
#include "common.cuh"
#include "internal.h"

namespace sra {
namespace pages {

constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ void count_error(int32_t* err, int n = 1) {
    if (err && n) atomicAdd(err, n);
}
__device__ __forceinline__ int64_t pages_of(int64_t len, int bs) { return (len + bs - 1) / bs; }

// ref_counts[page] -= k, never below zero: what exceeds the count is put back and counted as
// errors (final count and errors are the same for every order of such calls).
__device__ __forceinline__ void drop_refs(int32_t* ref, int32_t page, int k, int32_t* err) {
    const int old = atomicSub(ref + page, k);
    if (old < k) {
        const int excess = k - (old > 0 ? old : 0);
        atomicAdd(ref + page, excess);
        count_error(err, excess);
    }
}

// ------------------------------------------------------------------ copying
// (Plain loads and stores: with streaming hints 1021 pages of 28 layers, 937 MB read and written, took 171 us,
// without 147 at the time.)
template <typename V>
__device__ __forceinline__ void copy_span(char* dst, const char* src, int64_t nvec, int tid, int threads) {
    constexpr int kUnroll = 4;
    V* d = reinterpret_cast<V*>(dst);
    const V* s = reinterpret_cast<const V*>(src);
    int64_t i = tid;
    for (; i + (kUnroll - 1) * threads < nvec; i += kUnroll * threads) {
        V v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = s[i + u * threads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) d[i + u * threads] = v[u];
    }
    for (; i < nvec; i += threads) d[i] = s[i];
}

struct Pair {
    int32_t src, dst;
    int64_t bytes;  // of the page's start, in each plane (0: nothing)
};

// The CTAs [0, ctas) of a launch copy: item (cache, plane, pair) per step, pairs fastest, so that a page that is
// the source of several copies is read again while the L2 has it (1021 copies, some of one source, 140 us
// with the pairs slowest, 122 so).
template <typename V, typename F>
__device__ __forceinline__ void copy_items(const CacheList& c, int64_t count, int64_t cta, int64_t ctas, F&& pair) {
    const int64_t per = 2 * static_cast<int64_t>(c.n);
    for (int64_t item = cta; item < count * per; item += ctas) {
        const int rest = static_cast<int>(item / count);
        const int64_t i = item - rest * count;
        const Pair p = pair(i, rest == 0);
        if (p.bytes <= 0) continue;
        char* base = static_cast<char*>(c.p[rest >> 1]) + (rest & 1) * c.plane_bytes;
        copy_span<V>(base + p.dst * c.page_bytes, base + p.src * c.page_bytes,
                     p.bytes / static_cast<int64_t>(sizeof(V)), threadIdx.x, blockDim.x);
    }
}

constexpr int kCopyThreads = 128;

// (All CTAs that fit: five an SM with the 92 registers that 16-byte units compile to here. A form of 72, seven an SM,
// took 137 us for 1021 pages, 937 MB, where this one takes 123.)
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CacheList c, PageCopyArgs a) {
    pdl_enter();
    copy_items<V>(c, a.n, blockIdx.x, gridDim.x, [&](int64_t i, bool first) {
        const int32_t s = a.src[i], d = a.dst[i];
        Pair p{s, d, 0};
        if (s < 0 || d < 0 || s == d) {  // padding, or nothing to move
            if (s == d && s >= a.num_blocks && first && threadIdx.x == 0 && a.count_errors) count_error(a.err);
            return p;
        }
        if (s >= a.num_blocks || d >= a.num_blocks) {
            if (first && threadIdx.x == 0 && a.count_errors) count_error(a.err);
            return p;
        }
        p.bytes = c.page_bytes;
        return p;
    });
}

// ------------------------------------------------------------------ fork
constexpr int kRows = 8;        // entries of a call that one CTA takes together
constexpr int kCols = 128;      // table columns of a CTA, one per thread

// Whether an entry of idx[0 .. i) equals idx[i]; the whole warp asks. `other` (or null): an entry whose other
// index is negative is padding and names nothing.
__device__ __forceinline__ bool named_before(const int32_t* idx, const int32_t* other, int64_t i, int lane) {
    const int32_t me = idx[i];
    bool hit = false;
    for (int64_t k = lane; k < i; k += 32) hit |= idx[k] == me;
    if (!__any_sync(FULL, hit)) return false;
    if (!other) return true;
    hit = false;
    for (int64_t k = lane; k < i; k += 32) hit |= idx[k] == me && other[k] >= 0;
    return __any_sync(FULL, hit);
}

// A group of kCols threads takes kRows entries of a call, a thread a column of the table (every
// `x_groups` x kCols columns). The table kernels run these steps either with a group to a CTA and a launch
// per step, or, for small calls, with all groups in one CTA and a barrier between the steps: a launch costs
// about 3 us, a step on 640 entries less than 2.
struct Group {
    int tid;            // thread of the group
    int64_t i0;         // first entry
    int x, x_groups;    // column slice
    int barrier;        // named barrier of the group
    __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(kCols) : "memory"); }
};
__device__ __forceinline__ Group group_of_cta() {
    return {static_cast<int>(threadIdx.x), static_cast<int64_t>(blockIdx.y) * kRows, static_cast<int>(blockIdx.x),
            static_cast<int>(gridDim.x), 1};
}
// Group threadIdx.x / kCols of a CTA that holds all of a call's (round: its groups so far).
__device__ __forceinline__ Group group_of_all(int64_t round) {
    const int g = static_cast<int>(threadIdx.x) / kCols;
    return {static_cast<int>(threadIdx.x) % kCols, (round + g) * kRows, 0, 1, 1 + g};
}
constexpr int kGroups = 8;              // groups of a CTA that holds all of a call's
constexpr int64_t kSmallCall = 16384;   // table entries of such a call

// What entry i of a fork does: the parent's and the child's length at entry, or parent_len -1
// where it does nothing. Written by the first column slice, used by both steps.
// Entries of table row `row` at column j are changed by runs: rows of a group that hold the
// same page in a column change its count once.
__device__ __forceinline__ void fork_take(const ForkArgs& a, const Group& q, int (&s_len)[kRows], int (&s_row)[kRows]) {
    const int lane = threadIdx.x & 31, warp = q.tid >> 5;
    const int64_t i0 = q.i0;
    const bool first = q.x == 0;
    for (int r = warp; r < kRows; r += kCols / 32) {
        const int64_t i = i0 + r;
        int plen = -1, clen = -1, prow = 0;
        if (i < a.n) {
            const int32_t p = a.parents[i], c = a.children[i];
            if (p >= 0 && c >= 0) {
                bool bad = p >= a.rows || c >= a.rows;
                if (!bad) {
                    plen = a.seq_lens[p];
                    clen = a.seq_lens[c];
                    prow = p;
                    bad = plen < 0 || plen > a.cap || clen < 0 || clen > a.cap;
                }
                bad = named_before(a.children, a.parents, i, lane) || bad;
                if (bad) {
                    plen = -1;
                    if (first && lane == 0) count_error(a.err);
                }
            }
            if (first && lane == 0) {
                a.ws_plen[i] = plen;
                a.ws_clen[i] = clen;
            }
        }
        if (lane == 0) s_len[r] = plen, s_row[r] = prow;
    }
    q.sync();
    for (int64_t j = static_cast<int64_t>(q.x) * kCols + q.tid; j < a.max_blocks; j += static_cast<int64_t>(q.x_groups) * kCols) {
        int32_t e[kRows];
        unsigned has = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            e[r] = 0;
            if (s_len[r] > 0 && j < pages_of(s_len[r], a.block_size)) {
                has |= 1u << r;
                e[r] = a.table[static_cast<int64_t>(s_row[r]) * a.max_blocks + j];
            }
        }
        int32_t run = -1;
        int k = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (!((has >> r) & 1u)) continue;
            a.ws_snap[(i0 + r) * a.max_blocks + j] = e[r];
            if (e[r] < 0 || e[r] >= a.num_blocks) {
                count_error(a.err);
                continue;
            }
            if (e[r] != run) {
                if (k) atomicAdd(a.ref + run, k);
                run = e[r], k = 0;
            }
            ++k;
        }
        if (k) atomicAdd(a.ref + run, k);
    }
}

__device__ __forceinline__ void fork_give(const ForkArgs& a, const Group& q, int (&s_plen)[kRows], int (&s_clen)[kRows],
                                          int (&s_row)[kRows]) {
    const int64_t i0 = q.i0;
    if (q.tid < kRows) {
        const int64_t i = i0 + q.tid;
        const int plen = i < a.n ? a.ws_plen[i] : -1;
        s_plen[q.tid] = plen;
        s_clen[q.tid] = plen >= 0 ? a.ws_clen[i] : 0;
        s_row[q.tid] = plen >= 0 ? a.children[i] : 0;
        if (plen >= 0 && q.x == 0) a.seq_lens[a.children[i]] = plen;
    }
    q.sync();
    for (int64_t j = static_cast<int64_t>(q.x) * kCols + q.tid; j < a.max_blocks; j += static_cast<int64_t>(q.x_groups) * kCols) {
        int32_t old[kRows], now[kRows];
        unsigned has = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            old[r] = 0;
            if (s_plen[r] >= 0 && j < pages_of(s_clen[r], a.block_size)) {
                has |= 1u << r;
                old[r] = a.table[static_cast<int64_t>(s_row[r]) * a.max_blocks + j];
            }
            now[r] = s_plen[r] >= 0 && j < pages_of(s_plen[r], a.block_size) ? a.ws_snap[(i0 + r) * a.max_blocks + j]
                                                                            : -1;
        }
        int32_t run = -1;
        int k = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (s_plen[r] < 0) continue;
            a.table[static_cast<int64_t>(s_row[r]) * a.max_blocks + j] = now[r];
            if (!((has >> r) & 1u)) continue;
            if (old[r] < 0 || old[r] >= a.num_blocks) {
                count_error(a.err);
                continue;
            }
            if (old[r] != run) {
                if (k) drop_refs(a.ref, run, k, a.err);
                run = old[r], k = 0;
            }
            ++k;
        }
        if (k) drop_refs(a.ref, run, k, a.err);
    }
}

__global__ void __launch_bounds__(kCols) fork_take_kernel(ForkArgs a) {
    __shared__ int len[kRows], row[kRows];
    pdl_enter();
    fork_take(a, group_of_cta(), len, row);
}
__global__ void __launch_bounds__(kCols) fork_give_kernel(ForkArgs a) {
    __shared__ int plen[kRows], clen[kRows], row[kRows];
    pdl_enter();
    fork_give(a, group_of_cta(), plen, clen, row);
}
__global__ void __launch_bounds__(kGroups * kCols) fork_small_kernel(ForkArgs a) {
    __shared__ int s[3][kGroups][kRows];
    const int g = threadIdx.x / kCols;
    pdl_enter();
    for (int64_t round = 0; round * kRows < a.n; round += kGroups) {
        fork_take(a, group_of_all(round), s[0][g], s[1][g]);
        __syncthreads();
    }
    for (int64_t round = 0; round * kRows < a.n; round += kGroups) {
        fork_give(a, group_of_all(round), s[0][g], s[1][g], s[2][g]);
        __syncthreads();
    }
}

// ------------------------------------------------------------------ resize
// Release: the pages that shrinking rows hold past their new length. Also what each entry
// will do (ws_old: the row's length at entry, or -1 where the entry does nothing).
__device__ __forceinline__ void resize_release(const ResizeArgs& a, const Group& q, int (&s_old)[kRows],
                                               int (&s_new)[kRows], int (&s_row)[kRows]) {
    const int lane = threadIdx.x & 31, warp = q.tid >> 5;
    const int64_t i0 = q.i0;
    const bool first = q.x == 0;
    for (int r = warp; r < kRows; r += kCols / 32) {
        const int64_t i = i0 + r;
        int old = -1, len = 0, row = 0;
        if (i < a.n) {
            const int32_t want = a.row_idx[i];
            if (want >= 0) {
                len = a.lens[i];
                bool bad = want >= a.rows || len < 0 || len > a.cap;
                if (!bad) {
                    row = want;
                    old = a.seq_lens[row];
                    bad = old < 0 || old > a.cap;
                }
                bad = named_before(a.row_idx, nullptr, i, lane) || bad;
                if (bad) {
                    old = -1;
                    if (first && lane == 0) count_error(a.err);
                }
            }
            if (first && lane == 0) a.ws_old[i] = old;
        }
        if (lane == 0) s_old[r] = old, s_new[r] = len, s_row[r] = row;
    }
    q.sync();
    for (int64_t j = static_cast<int64_t>(q.x) * kCols + q.tid; j < a.max_blocks; j += static_cast<int64_t>(q.x_groups) * kCols) {
        int32_t e[kRows];
        unsigned has = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            e[r] = 0;
            if (s_old[r] > s_new[r] && j >= pages_of(s_new[r], a.block_size) && j < pages_of(s_old[r], a.block_size)) {
                has |= 1u << r;
                e[r] = a.table[static_cast<int64_t>(s_row[r]) * a.max_blocks + j];
            }
        }
        int32_t run = -1;
        int k = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (!((has >> r) & 1u)) continue;
            a.table[static_cast<int64_t>(s_row[r]) * a.max_blocks + j] = -1;
            if (e[r] < 0 || e[r] >= a.num_blocks) {
                count_error(a.err);
                continue;
            }
            if (e[r] != run) {
                if (k) drop_refs(a.ref, run, k, a.err);
                run = e[r], k = 0;
            }
            ++k;
        }
        if (k) drop_refs(a.ref, run, k, a.err);
    }
}

__global__ void __launch_bounds__(kCols) resize_release_kernel(ResizeArgs a) {
    __shared__ int old[kRows], len[kRows], row[kRows];
    pdl_enter();
    resize_release(a, group_of_cta(), old, len, row);
}

constexpr int kScanThreads = 1024;  // at most; a CTA has as many as its pages or entries need
constexpr int kScanPages = 16;  // pages a thread looks at per step: four 16-byte loads in flight

// Exclusive prefix sum of v over the CTA's threads; *total gets the sum. `scratch`: 33 words. (A CTA of one
// warp meets no barrier.)
template <typename I>
__device__ __forceinline__ I block_scan(I v, I* scratch, I* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    I inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I t = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += t;
    }
    if (blockDim.x == 32) {
        *total = __shfl_sync(FULL, inc, 31);
        return inc - v;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        I w = lane < static_cast<int>(blockDim.x >> 5) ? scratch[lane] : 0;
        const I mine = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I t = __shfl_up_sync(FULL, w, o);
            if (lane >= o) w += t;
        }
        scratch[lane] = w - mine;
        if (lane == 31) scratch[32] = w;
    }
    __syncthreads();
    const I before = scratch[warp] + inc - v;
    *total = scratch[32];
    __syncthreads();
    return before;
}

// The counts of pages [p, p + kScanPages) as a mask of those that are live (past the end: 0).
__device__ __forceinline__ unsigned live_mask(const int32_t* ref, int64_t p, int64_t nb, bool vec) {
    unsigned m = 0;
    if (vec && p + kScanPages <= nb) {
        int4 v[kScanPages / 4];
#pragma unroll
        for (int u = 0; u < kScanPages / 4; ++u) v[u] = reinterpret_cast<const int4*>(ref + p)[u];
#pragma unroll
        for (int u = 0; u < kScanPages / 4; ++u)
            m |= (v[u].x > 0 ? 1u : 0u) << (4 * u) | (v[u].y > 0 ? 2u : 0u) << (4 * u) |
                 (v[u].z > 0 ? 4u : 0u) << (4 * u) | (v[u].w > 0 ? 8u : 0u) << (4 * u);
    } else {
        for (int u = 0; u < kScanPages; ++u)
            if (p + u < nb && ref[p + u] > 0) m |= 1u << u;
    }
    return m;
}

// One CTA: how many pages each growing entry needs and where its pages start in the list of
// free pages, then that list, lowest page first, as far as it is needed.
__device__ __forceinline__ void resize_plan(const ResizeArgs& a, int64_t* scratch) {
    int64_t total = 0;
    for (int64_t base = 0; base < a.n; base += blockDim.x) {
        const int64_t i = base + threadIdx.x;
        int64_t need = 0;
        int32_t from = -1;
        if (i < a.n) {
            const int64_t old = a.ws_old[i], len = old >= 0 ? a.lens[i] : 0;
            if (old >= 0 && len > old) {
                const int64_t had = pages_of(old, a.block_size);
                need = pages_of(len, a.block_size) - had;
                if (old % a.block_size != 0) {
                    // a partly filled last page that other rows hold too is copied before it is written
                    const int32_t last = a.table[a.row_idx[i] * a.max_blocks + had - 1];
                    if (last < 0 || last >= a.num_blocks) {
                        need = 0;
                        a.ws_old[i] = -1;
                        count_error(a.err);
                    } else if (a.ref[last] > 1) {
                        from = last;
                        ++need;
                    }
                }
            }
        }
        int64_t sum;
        const int64_t before = block_scan(need, scratch, &sum);
        if (i < a.n) {
            a.ws_first[i] = total + before;
            a.ws_need[i] = static_cast<int32_t>(need);
            a.ws_from[i] = from;
        }
        total += sum;
    }
    const bool vec = (reinterpret_cast<uintptr_t>(a.ref) & 15u) == 0;
    int64_t found = 0;
    for (int64_t base = 0; base < a.num_blocks && found < total; base += static_cast<int64_t>(blockDim.x) * kScanPages) {
        const int64_t p = base + static_cast<int64_t>(threadIdx.x) * kScanPages;
        const int64_t left = a.num_blocks - p;
        const unsigned in = left >= kScanPages ? (1u << kScanPages) - 1u : left > 0 ? (1u << left) - 1u : 0u;
        unsigned free = ~live_mask(a.ref, p, a.num_blocks, vec) & in;
        int sum;
        int64_t at = found + block_scan(__popc(free), reinterpret_cast<int*>(scratch), &sum);
        for (; free && at < total; free &= free - 1, ++at) a.ws_free[at] = static_cast<int32_t>(p + __ffs(free) - 1);
        found += sum;
    }
    if (threadIdx.x == 0) *a.ws_found = found;
}
__global__ void __launch_bounds__(kScanThreads) resize_plan_kernel(ResizeArgs a) {
    __shared__ int64_t scratch[33];
    pdl_enter();
    resize_plan(a, scratch);
}
__global__ void __launch_bounds__(kGroups * kCols) resize_small_kernel(ResizeArgs a) {
    __shared__ int s[3][kGroups][kRows];
    __shared__ int64_t scratch[33];
    const int g = threadIdx.x / kCols;
    pdl_enter();
    for (int64_t round = 0; round * kRows < a.n; round += kGroups) {
        resize_release(a, group_of_all(round), s[0][g], s[1][g], s[2][g]);
        __syncthreads();
    }
    resize_plan(a, scratch);
}

// The CTAs below a.copy_from hand out the pages and finish the rows; the others copy the pages
// that are shared (both read the plan only, and write different words).
template <typename V>
__global__ void __launch_bounds__(kCols) resize_assign_kernel(CacheList c, ResizeArgs a) {
    pdl_enter();
    const int64_t found = *a.ws_found;
    auto served = [&](int64_t i) { return a.ws_first[i] + a.ws_need[i] <= found || a.ws_need[i] == 0; };
    if (blockIdx.x >= a.copy_from) {
        const int64_t token_bytes = c.page_bytes / a.block_size;
        copy_items<V>(c, a.n, blockIdx.x - a.copy_from, gridDim.x - a.copy_from, [&](int64_t i, bool) {
            Pair p{a.ws_from[i], 0, 0};
            if (p.src >= 0 && served(i)) {
                p.dst = a.ws_free[a.ws_first[i]];
                p.bytes = a.ws_old[i] % a.block_size * token_bytes;
            }
            return p;
        });
        return;
    }
    if (!a.bookkeeping) return;
    for (int64_t i = blockIdx.x; i < a.n; i += a.copy_from) {
        const int64_t old = a.ws_old[i];
        int64_t len = old;
        const int32_t row = a.row_idx[i];
        int32_t* t = a.table + row * a.max_blocks;
        int32_t last = -1;  // the page of the row's last token
        if (old >= 0) {
            len = a.lens[i];
            if (len > old) {
                const int64_t had = pages_of(old, a.block_size), want = pages_of(len, a.block_size);
                const int32_t from = a.ws_from[i];
                if (served(i)) {
                    const int64_t begin = had - (from >= 0 ? 1 : 0);
                    const int32_t* pages = a.ws_free + a.ws_first[i];
                    for (int64_t j = begin + threadIdx.x; j < want; j += kCols) {
                        const int32_t page = pages[j - begin];
                        t[j] = page;
                        a.ref[page] = 1;
                    }
                    if (threadIdx.x == 0 && from >= 0) atomicSub(a.ref + from, 1);
                    last = begin < want ? pages[want - 1 - begin] : t[want - 1];
                } else {
                    if (threadIdx.x == 0) count_error(a.err);
                    len = old;
                }
            }
        }
        if (threadIdx.x == 0) {
            int64_t pos = -1, slot = -1;
            if (old >= 0) {
                a.seq_lens[row] = static_cast<int32_t>(len);
                if (len > 0) {
                    if (last < 0) last = t[(len - 1) / a.block_size];
                    pos = len - 1;
                    slot = last >= 0 && last < a.num_blocks
                               ? static_cast<int64_t>(last) * a.block_size + pos % a.block_size
                               : -1;
                }
            }
            if (a.pos) a.pos[i] = pos;
            if (a.slot) a.slot[i] = slot;
        }
    }
}

// ------------------------------------------------------------------ compact
// One CTA: N live pages; the free pages below N in order (ws_dst), and for every page its rank
// among the live ones, or -1 (ws_rank). Live page p >= N is the (rank - (N - moved))-th to move.
__global__ void __launch_bounds__(kScanThreads) compact_plan_kernel(CompactArgs a) {
    __shared__ int scratch[33];
    pdl_enter();
    const bool vec = (reinterpret_cast<uintptr_t>(a.ref) & 15u) == 0;
    const int64_t step = static_cast<int64_t>(blockDim.x) * kScanPages;
    int mine = 0, live = 0;  // (fewer than 2^31 pages)
    for (int64_t base = 0; base < a.num_blocks; base += step)
        mine += __popc(live_mask(a.ref, base + static_cast<int64_t>(threadIdx.x) * kScanPages, a.num_blocks, vec));
    block_scan(mine, scratch, &live);
    int seen = 0;  // live pages before this step's
    for (int64_t base = 0; base < a.num_blocks; base += step) {
        const int64_t p = base + static_cast<int64_t>(threadIdx.x) * kScanPages;
        const unsigned m = live_mask(a.ref, p, a.num_blocks, vec);
        int sum;
        int rank = seen + block_scan(__popc(m), scratch, &sum);
        for (int u = 0; u < kScanPages && p + u < a.num_blocks; ++u) {
            const bool on = (m >> u) & 1u;
            a.ws_rank[p + u] = on ? static_cast<int32_t>(rank) : -1;
            if (on) {
                if (p + u >= live) a.ws_src[rank] = static_cast<int32_t>(p + u);
                ++rank;
            } else if (p + u < live) {
                a.ws_dst[p + u - rank] = static_cast<int32_t>(p + u);
            }
            if (p + u == live - 1) *a.ws_moved = static_cast<int32_t>(live - rank);  // free pages below N
        }
        seen += sum;
    }
    if (threadIdx.x == 0) {
        if (live == 0) *a.ws_moved = 0;
        if (a.num_live) *a.num_live = static_cast<int32_t>(live);
        *a.ws_live = static_cast<int32_t>(live);
    }
}

template <typename V>
__global__ void __launch_bounds__(kCols) compact_move_kernel(CacheList c, CompactArgs a) {
    pdl_enter();
    const int64_t live = *a.ws_live, moved = *a.ws_moved, below = live - moved;
    if (blockIdx.x >= a.copy_from) {
        // Many pages are copied by five CTAs an SM, 6 MB in flight (measured at one size, 974 pages of 28 layers: 143
        // us; by four 154, by six 147, by all twelve 151); few by all, whose index reads then overlap (70 MB 15 us, by six an SM 21).
        const int64_t all = gridDim.x - a.copy_from, cta = blockIdx.x - a.copy_from;
        const int64_t ctas = moved * 2 * c.n >= 16 * all && a.few < all ? a.few : all;
        if (cta < ctas)
            copy_items<V>(c, moved, cta, ctas,
                          [&](int64_t i, bool) { return Pair{a.ws_src[below + i], a.ws_dst[i], c.page_bytes}; });
        return;
    }
    if (!a.bookkeeping) return;
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x, all = a.copy_from * kCols;
    for (int64_t i = tid; i < moved; i += all) {
        const int32_t s = a.ws_src[below + i];
        a.ref[a.ws_dst[i]] = a.ref[s];
        a.ref[s] = 0;
    }
    for (int64_t row = blockIdx.x; row < a.rows; row += a.copy_from) {
        const int64_t len = a.seq_lens[row];
        if (len < 0 || len > a.cap) {
            if (threadIdx.x == 0) count_error(a.err);
            continue;
        }
        int32_t* t = a.table + row * a.max_blocks;
        const int64_t used = pages_of(len, a.block_size);
        for (int64_t j = threadIdx.x; j < used; j += kCols) {
            const int32_t e = t[j];
            const int32_t rank = e >= 0 && e < a.num_blocks ? a.ws_rank[e] : -1;
            if (rank < 0)
                count_error(a.err);  // not a page, or one that no row is said to hold: left as it is
            else if (e >= live)
                t[j] = a.ws_dst[rank - below];
        }
    }
}

// ------------------------------------------------------------------ launches
template <typename F>
cudaError_t by_vec(int vec, F&& f) {
    switch (vec) {
        case 16: return f(uint4{});
        case 8: return f(uint2{});
        case 4: return f(static_cast<unsigned int>(0));
        default: return f(static_cast<unsigned short>(0));
    }
}

// CTAs that copy `items` (pair, cache, plane) spans: all resident at once at most, beside `others` CTAs of the
// launch (a copying CTA that starts when those are done ends late: the copies on write of 121 rows in 28 layers
// 16.8 us, beside them 15.3).
template <typename... KArgs>
int64_t copy_ctas(void (*kernel)(KArgs...), int num_sms, int64_t items, int64_t others = 0) {
    const int64_t all = persistent_grid(kernel, kCopyThreads, 0, num_sms, items + others);
    return all - others > all / 2 ? all - others : all / 2 + 1;
}

}  // namespace pages

cudaError_t launch_copy_pages(const CacheList& c, const PageCopyArgs& a, const PagePlan& p, cudaStream_t s) {
    return pages::by_vec(p.vec, [&](auto v) {
        auto kernel = pages::copy_kernel<decltype(v)>;
        const unsigned grid = static_cast<unsigned>(pages::copy_ctas(kernel, p.num_sms, a.n * c.n * 2));
        return launch_kernel(kernel, dim3(grid), dim3(pages::kCopyThreads), 0, s, p.pdl, 1, c, a);
    });
}

static dim3 table_grid(int64_t n, int64_t max_blocks) {
    const int64_t x = (max_blocks + pages::kCols - 1) / pages::kCols;
    return dim3(static_cast<unsigned>(x < 1 ? 1 : x > 1024 ? 1024 : x),
                static_cast<unsigned>((n + pages::kRows - 1) / pages::kRows));
}

// Threads of a CTA that scans `pages` pages and holds `entries` entries a thread each.
static dim3 scan_block(int64_t pages, int64_t entries) {
    int64_t t = (pages + pages::kScanPages - 1) / pages::kScanPages;
    t = ((t > entries ? t : entries) + 31) / 32 * 32;
    return dim3(static_cast<unsigned>(t < 32 ? 32 : t > pages::kScanThreads ? pages::kScanThreads : t));
}

// Calls whose groups all go into one CTA, and its threads.
static bool small_call(int64_t n, int64_t max_blocks) { return n * (max_blocks > 32 ? max_blocks : 32) <= pages::kSmallCall; }
static dim3 small_block(int64_t n) {
    const int64_t g = (n + pages::kRows - 1) / pages::kRows;
    return dim3(static_cast<unsigned>((g < pages::kGroups ? g : pages::kGroups) * pages::kCols));
}

cudaError_t launch_fork_rows(const ForkArgs& a, const PagePlan& p, cudaStream_t s) {
    if (small_call(a.n, a.max_blocks))
        return launch_kernel(pages::fork_small_kernel, dim3(1), small_block(a.n), 0, s, p.pdl, 1, a);
    const dim3 grid = table_grid(a.n, a.max_blocks), block(pages::kCols);
    const cudaError_t e = launch_kernel(pages::fork_take_kernel, grid, block, 0, s, p.pdl, 1, a);
    return e != cudaSuccess ? e : launch_kernel(pages::fork_give_kernel, grid, block, 0, s, true, 1, a);
}

cudaError_t launch_resize_plan(const ResizeArgs& a, const PagePlan& p, cudaStream_t s) {
    if (small_call(a.n, a.max_blocks))
        return launch_kernel(pages::resize_small_kernel, dim3(1), small_block(a.n), 0, s, p.pdl, 1, a);
    const cudaError_t e = launch_kernel(pages::resize_release_kernel, table_grid(a.n, a.max_blocks),
                                        dim3(pages::kCols), 0, s, p.pdl, 1, a);
    return e != cudaSuccess
               ? e
               : launch_kernel(pages::resize_plan_kernel, dim3(1), scan_block(a.num_blocks, a.n), 0, s, true, 1, a);
}

cudaError_t launch_resize_assign(const CacheList& c, const ResizeArgs& a, const PagePlan& p, cudaStream_t s) {
    return pages::by_vec(p.vec, [&](auto v) {
        auto kernel = pages::resize_assign_kernel<decltype(v)>;
        ResizeArgs b = a;
        b.copy_from = a.n < p.num_sms ? a.n : p.num_sms;
        const int64_t copy = pages::copy_ctas(kernel, p.num_sms, a.n * c.n * 2, b.copy_from);
        return launch_kernel(kernel, dim3(static_cast<unsigned>(b.copy_from + copy)), dim3(pages::kCols), 0, s, true, 1,
                             c, b);
    });
}

cudaError_t launch_compact_plan(const CompactArgs& a, const PagePlan& p, cudaStream_t s) {
    return launch_kernel(pages::compact_plan_kernel, dim3(1), scan_block(a.num_blocks, 0), 0, s, p.pdl, 1, a);
}

cudaError_t launch_compact_move(const CacheList& c, const CompactArgs& a, const PagePlan& p, cudaStream_t s) {
    return pages::by_vec(p.vec, [&](auto v) {
        auto kernel = pages::compact_move_kernel<decltype(v)>;
        CompactArgs b = a;
        b.copy_from = a.rows < p.num_sms && a.rows > 0 ? a.rows : p.num_sms;
        const int64_t copy = pages::copy_ctas(kernel, p.num_sms, a.num_blocks / 2 * c.n * 2 + 1, b.copy_from);
        b.few = 5 * static_cast<int64_t>(p.num_sms);
        return launch_kernel(kernel, dim3(static_cast<unsigned>(b.copy_from + copy)), dim3(pages::kCols), 0, s, true, 1,
                             c, b);
    });
}

}  // namespace sra

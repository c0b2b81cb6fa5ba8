// Pages of a cache: taking, sharing, giving back, copying and closing up the pages of pools that
// hold sequences' recurrent states, convolution histories or token rows.
//
// refs[p] counts the page table entries that hold page p; a page with none is free, and the lowest
// free pages are given out first, so every result is a function of the arguments alone.  The
// bookkeeping is integers: one read of refs and of the table rows concerned.  It is bound by
// latency, so each operation is one kernel of one cluster (eight blocks when there are many pages or forks,
// else one): the blocks count their share of refs, exchange the counts through distributed shared
// memory, and place their own pages, with hardware cluster barriers between and no waiting on
// memory.  The payload moves in kda_pages_copy, bound by HBM: 24 pages of 6.3 MB in 45 us.  Of the books, taking pages
// of 8192 takes 5 us, of a million 16; closing up 8192 pages 10, a million 108; 64 forks of rows of 64 entries 10.
#include <cooperative_groups.h>

#include "kda_layer.h"
#include "kda_segments.cuh"

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMostBlocks = 8;
// One block counts this many pages as fast as a cluster starts and meets: compaction of 8192 pages takes 10 us
// either way, 16384 take 14 in one block and 10 in a cluster, 32768 take 23 and 10.5.
constexpr int kPagesOfOneBlock = 8192;

// Sum of x over the block's threads before this one; *all: over all of them.  `tmp` holds
// kWarps + 1 ints; the block meets twice.
__device__ __forceinline__ int block_before(int x, int* tmp, int* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) tmp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int w = tmp[lane];
        int s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        tmp[lane] = s - w;
        if (lane == 31) tmp[kWarps] = s;
    }
    __syncthreads();
    *all = tmp[kWarps];
    return tmp[warp] + inc - x;
}

struct Shared {
    int tmp[kWarps + 1];
    int mine[2];  // this block's counts, read by the others
};

// Sums over the cluster's earlier blocks (base) and over all of them (all) of two counts.
__device__ __forceinline__ void cluster_sums(Shared& sh, int c0, int c1, int (&base)[2], int (&all)[2]) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) {
        sh.mine[0] = c0;
        sh.mine[1] = c1;
    }
    cl.sync();
    base[0] = base[1] = all[0] = all[1] = 0;
    const int rank = cl.block_rank(), blocks = cl.num_blocks();
    for (int r = 0; r < blocks; ++r) {
        const int* m = cl.map_shared_rank(sh.mine, r);
        const int a = m[0], b = m[1];
        if (r < rank) {
            base[0] += a;
            base[1] += b;
        }
        all[0] += a;
        all[1] += b;
    }
    cl.sync();  // before anyone writes `mine` again or leaves
}

constexpr int kEach = 4;                  // neighbouring things a thread looks at
constexpr int kTile = kThreads * kEach;

// The block's share [lo, hi) of n things, whole tiles.
__device__ __forceinline__ void share(int n, int& lo, int& hi) {
    cg::cluster_group cl = cg::this_cluster();
    const int blocks = cl.num_blocks(), tiles = n > 0 ? (n - 1) / kTile + 1 : 0;
    const int per = (tiles + blocks - 1) / blocks;
    const int64_t a = (int64_t)cl.block_rank() * per * kTile;
    lo = (int)min(a, (int64_t)n);
    hi = (int)min(a + (int64_t)per * kTile, (int64_t)n);
}

// Bit k: whether thing i + k of [lo, hi) satisfies f; the loads are independent of one another.
template <typename F>
__device__ __forceinline__ int which_of(int i, int hi, F f) {
    int bits = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) bits |= (i + k < hi && f(i + k) ? 1 : 0) << k;
    return bits;
}

// How many of [lo, hi) satisfy f (every thread gets the sum).
template <typename F>
__device__ __forceinline__ int count_if(Shared& sh, int lo, int hi, F f) {
    int c = 0;
#pragma unroll 4
    for (int64_t i = lo + (int)threadIdx.x * kEach; i < hi; i += kTile) c += __popc(which_of((int)i, hi, f));
    int all;
    block_before(c, sh.tmp, &all);
    __syncthreads();
    return all;
}

// put(rank, i) for every i of [lo, hi) with f(i), rank counting on from `base` in order of i;
// stops where the ranks reach `most`.
template <typename F, typename G>
__device__ __forceinline__ void place_if(Shared& sh, int lo, int hi, int base, int most, F f, G put) {
    for (int64_t i0 = lo; i0 < hi && base < most; i0 += kTile) {
        const int i = (int)i0 + (int)threadIdx.x * kEach;
        int bits = which_of(i, hi, f), all;
        int rank = base + block_before(__popc(bits), sh.tmp, &all);
        for (; bits && rank < most; bits &= bits - 1) put(rank++, i + __ffs(bits) - 1);
        base += all;
        __syncthreads();
    }
}

__device__ __forceinline__ void report(int32_t* status) {
    if (status) *status = KDA_ERR_RANGE;
}

// ---- taking and giving back ------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) pages_alloc_kernel(int32_t* refs, int P, int n, int32_t* out,
                                                               int32_t* status) {
    __shared__ Shared sh;
    int lo, hi, base[2], all[2];
    share(P, lo, hi);
    const auto is_free = [&](int i) { return refs[i] == 0; };
    cluster_sums(sh, count_if(sh, lo, hi, is_free), 0, base, all);
    place_if(sh, lo, hi, base[0], n, is_free, [&](int rank, int i) {
        out[rank] = i;
        refs[i] = 1;
    });
    if (all[0] < n) {
        cg::cluster_group cl = cg::this_cluster();
        for (int i = all[0] + cl.block_rank() * kThreads + threadIdx.x; i < n; i += cl.num_blocks() * kThreads) out[i] = -1;
        if (threadIdx.x == 0) report(status);
    }
}

__global__ void __launch_bounds__(256) pages_free_kernel(int32_t* refs, int P, const int32_t* pages, int64_t n,
                                                         int32_t* status) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int p = pages[i];
        if (p == -1) continue;
        bool ok = p >= 0 && p < P;
        if (ok) {
            // a count that is 0 already stays so
            int have = refs[p];
            for (;;) {
                if (have <= 0) {
                    ok = false;
                    break;
                }
                const int was = atomicCAS(refs + p, have, have - 1);
                if (was == have) break;
                have = was;
            }
        }
        if (!ok) report(status);
    }
}

// ---- forking ---------------------------------------------------------------------------------

// What becomes of request k, kept in dst_out[k] between the phases.
constexpr int kNeedsPage = 2, kSharesOnly = 1, kNothing = 0;
constexpr int kRefused = -2;
// One block writes this many children's rows as fast as a cluster: 64 rows of 16 to 256 entries take 9 to 16 us in one
// block and 10 to 16 in a cluster, 128 rows 14 to 22 and 11 to 15, 65536 rows of 64 entries 4000 and 670.
constexpr int kForksOfOneBlock = 64;
// Every pair of this many requests is compared (256 requests take 12 us, 13 by chains); more go by chains (1024 take
// 63 us by pairs, 23 by chains, 65536 114 ms and 0.7).
constexpr int kFewForks = 256;

// Sets kConflict in next[k] of every request k whose child is another request's child or any request's parent, in
// time linear in n: requests are chained by a hash of their child, head[n] holding the first of each chain and
// next[k] & kNext the one behind k, both plus one.  A look along a chain ends at the first request of the child it
// looks for, so that many requests of one child cost no more.
constexpr int kNext = 0xfffff, kConflict = 1 << 30;
__device__ __forceinline__ void find_conflicts(const int32_t* parents, const int32_t* children, int n, int32_t* head,
                                               int32_t* next) {
    cg::cluster_group cl = cg::this_cluster();
    const int first = cl.block_rank() * kThreads + threadIdx.x, step = cl.num_blocks() * kThreads;
    const auto chain = [&](int c) { return (int)__umulhi((unsigned)c * 2654435769u, (unsigned)n); };
    // the first request other than k whose child is c
    const auto other = [&](int c, int k) {
        int j = head[chain(c)] - 1;
        while (j >= 0 && (j == k || children[j] != c)) j = (next[j] & kNext) - 1;
        return j;
    };
    for (int i = first; i < n; i += step) head[i] = 0;
    cl.sync();
    for (int k = first; k < n; k += step) {
        const int c = children[k];
        next[k] = c != -1 && parents[k] != -1 ? atomicExch(head + chain(c), k + 1) : 0;
    }
    cl.sync();
    for (int k = first; k < n; k += step) {
        const int p = parents[k], c = children[k];
        if (p == -1 || c == -1) continue;
        if (other(c, k) >= 0) atomicOr(next + k, kConflict);
        const int j = other(p, -1);  // (if it is not the only one of its child, all of them have the flag)
        if (j >= 0) atomicOr(next + j, kConflict);
    }
    cl.sync();
}

__global__ void __launch_bounds__(kThreads) pages_fork_kernel(int32_t* tables, int32_t* lens, int S, int width,
                                                              int page_tokens, int32_t* refs, int P,
                                                              const int32_t* parents, const int32_t* children, int n,
                                                              int32_t* src_out, int32_t* dst_out, int32_t* status) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31;
    const int warp = cl.block_rank() * kWarps + (threadIdx.x >> 5), warps = cl.num_blocks() * kWarps;

    // 1. which requests stand: a warp looks each over
    const bool few = n <= kFewForks;
    if (!few) find_conflicts(parents, children, n, src_out, dst_out);
    for (int k = warp; k < n; k += warps) {
        const int p = parents[k], c = children[k];
        int what = kNothing;
        if (p != -1 && c != -1) {
            bool bad = p < 0 || p >= S || c < 0 || c >= S;
            if (few) {
                for (int j = lane; j < n && !bad; j += 32) {
                    const int pj = parents[j], cj = children[j];
                    if (pj != -1 && cj != -1 && (pj == c || (j != k && cj == c))) bad = true;
                }
                bad = __any_sync(0xffffffffu, bad);
            } else {
                bad |= (dst_out[k] & kConflict) != 0;
                __syncwarp();
            }
            int full = 0;
            bool part = false;
            if (!bad) {
                const int len = lens[p];
                if (len < 0 || len > (int64_t)width * page_tokens) {
                    bad = true;
                } else {
                    full = len / page_tokens;
                    part = len % page_tokens != 0;
                }
            }
            const int held = full + (part ? 1 : 0);
            for (int j = lane; j < held && !bad; j += 32) {
                const int page = tables[(int64_t)p * width + j];
                if (page < 0 || page >= P || refs[page] <= 0) bad = true;
            }
            bad = __any_sync(0xffffffffu, bad);
            what = bad ? kNothing : part ? kNeedsPage : kSharesOnly;
            if (bad && lane == 0) report(status);
        }
        if (lane == 0) dst_out[k] = what;
    }
    cl.sync();

    // 2. the free pages in order (in src_out, for now), and how many requests before each need one
    int lo, hi, klo, khi, base[2], all[2];
    share(P, lo, hi);
    share(n, klo, khi);
    const auto is_free = [&](int i) { return refs[i] == 0; };
    const auto needs = [&](int k) { return dst_out[k] == kNeedsPage; };
    const int free_here = count_if(sh, lo, hi, is_free);
    const int need_here = count_if(sh, klo, khi, needs);
    cluster_sums(sh, free_here, need_here, base, all);
    place_if(sh, lo, hi, base[0], all[1], is_free, [&](int rank, int i) { src_out[rank] = i; });
    cl.sync();

    // 3. the requests' pages, in order; those that find none are refused
    for (int k0 = klo, rank = base[1]; k0 < khi; k0 += kThreads) {
        const int k = k0 + threadIdx.x;
        const int what = k < khi ? dst_out[k] : kNothing;
        int here;
        const int before = block_before(what == kNeedsPage ? 1 : 0, sh.tmp, &here);
        if (k < khi) {
            int page = what == kSharesOnly ? -1 : kRefused;
            if (what == kNeedsPage) {
                if (rank + before < all[0]) page = src_out[rank + before];
                else report(status);
            }
            dst_out[k] = page;
        }
        rank += here;
        __syncthreads();
    }
    cl.sync();

    // 4. the children's rows
    for (int k = warp; k < n; k += warps) {
        const int page = dst_out[k];
        __syncwarp();
        if (page == kRefused) {
            if (lane == 0) src_out[k] = dst_out[k] = -1;
            continue;
        }
        const int p = parents[k], c = children[k], len = lens[p], full = len / page_tokens;
        const int32_t* from = tables + (int64_t)p * width;
        int32_t* to = tables + (int64_t)c * width;
        for (int j = lane; j < width; j += 32) {
            int e = -1;
            if (j < full) {
                e = from[j];
                atomicAdd(refs + e, 1);
            } else if (j == full && page >= 0) {
                e = page;
                refs[e] = 1;
            }
            to[j] = e;
        }
        if (lane == 0) {
            src_out[k] = page >= 0 ? from[full] : -1;
            lens[c] = len;
        }
    }
}

// ---- closing up ------------------------------------------------------------------------------

// remap[0] is the number of used pages; remap[1 + p] the new place of a used page p behind it, -1 of a free one.  Of a
// free page before it remap[1 + p] is the move that fills its place; of a used one it is whatever was there, so that only
// as many words are written as there are moves, and dst[] has to confirm it.
// The entries i, i + step, ... of four, their loads ahead of the looks at them (8192 pages with 65536 entries: 37 us one by
// one, 25 by fours).
__device__ __forceinline__ void remap_entries(int32_t* tables, int64_t i, int64_t step, int64_t entries, int live, int P,
                                              const int32_t* remap, const int32_t* dst, int32_t* status) {
    int e[kEach], to[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) e[k] = i + k * step < entries ? tables[i + k * step] : -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) to[k] = e[k] >= 0 && e[k] < P ? remap[1 + e[k]] : -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        if (e[k] == -1) continue;
        if (e[k] >= 0 && e[k] < live) {
            if (to[k] >= 0 && to[k] < P / 2 && dst[to[k]] == e[k]) report(status);  // it was free: another page lies there now
        } else if (to[k] >= 0) {
            tables[i + k * step] = to[k];
        } else {
            report(status);  // an entry that held no used page stays as it is
        }
    }
}

// Table entries that the cluster itself looks over; more are a launch of their own over the machine.
constexpr int64_t kEntriesOfCluster = 65536;

__global__ void __launch_bounds__(kThreads) pages_compact_kernel(int32_t* refs, int P, int32_t* src_out,
                                                                 int32_t* dst_out, int32_t* remap, int32_t* tables,
                                                                 int entries, int32_t* status) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    int lo, hi, base[2], all[2];
    share(P, lo, hi);
    const int used_here = count_if(sh, lo, hi, [&](int i) { return refs[i] != 0; });
    cluster_sums(sh, used_here, 0, base, all);
    const int live = all[0];
    const auto hole = [&](int i) { return i < live && refs[i] == 0; };
    const auto tail = [&](int i) { return i >= live && refs[i] != 0; };
    // a share on one side of `live` has been counted already
    int holes = hi <= live ? hi - lo - used_here : 0, tails = lo >= live ? used_here : 0;
    if (lo < live && live < hi) {
        holes = count_if(sh, lo, hi, hole);
        tails = count_if(sh, lo, hi, tail);
    }
    cluster_sums(sh, holes, tails, base, all);
    const int moves = all[0];  // as many used pages behind `live` as holes before it
    place_if(sh, lo, min(hi, live), base[0], moves, hole, [&](int rank, int i) { dst_out[rank] = i; });
    place_if(sh, max(lo, min(live, hi)), hi, base[1], moves, tail, [&](int rank, int i) { src_out[rank] = i; });
    if (remap) {
        for (int i = max(lo, live) + (int)threadIdx.x; i < hi; i += kThreads)
            if (refs[i] == 0) remap[1 + i] = -1;
        if (cl.block_rank() == 0 && threadIdx.x == 0) remap[0] = live;
    }
    cl.sync();
    const int first = cl.block_rank() * kThreads + threadIdx.x, step = cl.num_blocks() * kThreads;
    for (int m = first; m < P / 2; m += step) {
        if (m >= moves) {
            src_out[m] = dst_out[m] = -1;
            continue;
        }
        const int s = src_out[m], d = dst_out[m];
        if (remap) {
            remap[1 + s] = d;
            remap[1 + d] = m;
        }
        refs[d] = refs[s];
        refs[s] = 0;
    }
    if (entries == 0) return;
    cl.sync();
    for (int i = first; i < entries; i += kEach * step) remap_entries(tables, i, step, entries, live, P, remap, dst_out, status);
}

__global__ void __launch_bounds__(256) pages_remap_kernel(int32_t* tables, int64_t entries, int P, const int32_t* remap,
                                                          const int32_t* dst, int32_t* status) {
    const int live = remap[0];
    const int64_t step = gridDim.x * 256ll;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < entries; i += kEach * step)
        remap_entries(tables, i, step, entries, live, P, remap, dst, status);
}

// ---- copying ---------------------------------------------------------------------------------

constexpr int kCopyThreads = 256, kCopySms = 152;
constexpr int kCopyVec = 4;                                  // 16-byte pieces of a thread in one go
constexpr int kCopyPiece = kCopyThreads * kCopyVec * 16;     // bytes of a block in one go

// Piece `at` of page s onto page d.
__device__ __forceinline__ void copy_piece(char* pool, int64_t page_bytes, int s, int d, int64_t at) {
    const uint4* from = reinterpret_cast<const uint4*>(pool + s * page_bytes + at);
    uint4* to = reinterpret_cast<uint4*>(pool + d * page_bytes + at);
    const int left = (int)(min((int64_t)kCopyPiece, page_bytes - at) / 16);
    uint4 r[kCopyVec];
#pragma unroll
    for (int v = 0; v < kCopyVec; ++v)
        if (v * kCopyThreads + (int)threadIdx.x < left) r[v] = __ldcs(from + v * kCopyThreads + threadIdx.x);
#pragma unroll
    for (int v = 0; v < kCopyVec; ++v)
        if (v * kCopyThreads + (int)threadIdx.x < left) __stcs(to + v * kCopyThreads + threadIdx.x, r[v]);
}

// marks, all zero before: [0] pairs listed, [1, 1 + P) the last pair (+ 1) that writes a page,
// [1 + P, 1 + 2 P) whether a pair reads it, then the list.
__global__ void __launch_bounds__(256) pages_mark_kernel(const int32_t* src, const int32_t* dst, int n, int P,
                                                         int32_t* marks, int32_t* status) {
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int s = src[i], d = dst[i];
        if (s == -1 || d == -1) continue;
        if (s < 0 || s >= P || d < 0 || d >= P) {
            report(status);
            continue;
        }
        if (s == d) continue;
        atomicMax(marks + 1 + d, i + 1);
        marks[1 + (int64_t)P + s] = 1;
        marks[1 + 2 * (int64_t)P + atomicAdd(marks, 1)] = i;
    }
}

__global__ void __launch_bounds__(kCopyThreads, 8) pages_copy_kernel(char* pool, int64_t page_bytes, const int32_t* src,
                                                                     const int32_t* dst, int P, const int32_t* marks,
                                                                     int32_t* status) {
    const int pairs = marks[0];
    const int64_t pieces = (page_bytes + kCopyPiece - 1) / kCopyPiece, items = pairs * pieces;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int i = marks[1 + 2 * (int64_t)P + it / pieces];
        const int64_t at = it % pieces * kCopyPiece;
        const int s = src[i], d = dst[i];
        // a later pair writes this page, or a pair reads it: left alone
        if (marks[1 + d] != i + 1 || marks[1 + (int64_t)P + d] != 0) {
            if (threadIdx.x == 0 && at == 0) report(status);
            continue;
        }
        copy_piece(pool, page_bytes, s, d, at);
    }
}

// Up to kFewPairs pairs: every block looks all of them over by itself (two threads hold a pair against half of
// the others each) and needs no marks.  128 pairs take about 3 us this way and 5 with the marks, 256 took 7.
constexpr int kFewPairs = kCopyThreads / 2;
__global__ void __launch_bounds__(kCopyThreads, 8) pages_copy_few_kernel(char* pool, int64_t page_bytes, const int32_t* src,
                                                                         const int32_t* dst, int n, int P, int32_t* status) {
    __shared__ __align__(16) int2 pairs[kFewPairs];
    __shared__ int2 good[kFewPairs];
    __shared__ int counts[kFewPairs / 32], against_first[kFewPairs];
    const int i = threadIdx.x % kFewPairs, part = threadIdx.x / kFewPairs, lane = i & 31, warp = i >> 5;
    int2 me = i < n ? make_int2(src[i], dst[i]) : make_int2(-1, -1);
    bool bad = false;
    if (me.x == -1 || me.y == -1 || me.x == me.y) {
        bad = me.x == me.y && me.x != -1 && (me.x < 0 || me.x >= P);
        me = make_int2(-1, -1);
    } else if (me.x < 0 || me.x >= P || me.y < 0 || me.y >= P) {
        bad = true;
        me = make_int2(-1, -1);
    }
    if (part == 0) pairs[i] = me;
    __syncthreads();
    // a later pair writes this page, or a pair reads it: left alone
    int against = 0;
    const int4* two = reinterpret_cast<const int4*>(pairs);
#pragma unroll 4
    for (int j = part * kFewPairs / 4; j < (part + 1) * kFewPairs / 4; ++j) {
        const int4 o = two[j];
        against |= (o.x == me.y) | (o.z == me.y) | ((o.y == me.y) & (2 * j > i)) | ((o.w == me.y) & (2 * j + 1 > i));
    }
    if (part == 0) against_first[i] = against;
    __syncthreads();
    const bool ok = part == 1 && me.x != -1 && !(against | against_first[i]);
    if (me.x != -1 && !ok) bad = true;
    if (bad && part == 1 && blockIdx.x == 0) report(status);
    const unsigned votes = __ballot_sync(0xffffffffu, ok);
    if (part == 1 && lane == 0) counts[warp] = __popc(votes);
    __syncthreads();
    int before = __popc(votes & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < kFewPairs / 32; ++w) {
        if (w < warp) before += counts[w];
        all += counts[w];
    }
    if (ok) good[before] = me;
    __syncthreads();
    const int64_t pieces = (page_bytes + kCopyPiece - 1) / kCopyPiece, items = all * pieces;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int2 q = good[it / pieces];
        copy_piece(pool, page_bytes, q.x, q.y, it % pieces * kCopyPiece);
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), bool many, cudaStream_t st, Args... args) {
    if (!many) {  // a cluster of one, without the cost of asking for it
        kern<<<1, kThreads, 0, st>>>(static_cast<KArgs>(args)...);
        return cudaGetLastError();
    }
    constexpr int blocks = kMostBlocks;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace

cudaError_t pages_alloc(int32_t* refs, int P, int n, int32_t* out, int32_t* status, cudaStream_t st) {
    return launch_cluster(pages_alloc_kernel, P > kPagesOfOneBlock, st, refs, P, n, out, status);
}

cudaError_t pages_free(int32_t* refs, int P, const int32_t* pages, int64_t n, int32_t* status, cudaStream_t st) {
    const int64_t blocks = (n + 255) / 256;
    pages_free_kernel<<<(unsigned)(blocks < 1216 ? blocks : 1216), 256, 0, st>>>(refs, P, pages, n, status);
    return cudaGetLastError();
}

cudaError_t pages_fork(int32_t* tables, int32_t* lens, int S, int width, int page_tokens, int32_t* refs, int P,
                       const int32_t* parents, const int32_t* children, int n, int32_t* src, int32_t* dst,
                       int32_t* status, cudaStream_t st) {
    return launch_cluster(pages_fork_kernel, P > kPagesOfOneBlock || n > kForksOfOneBlock, st, tables, lens, S, width,
                          page_tokens, refs, P, parents, children, n, src, dst, status);
}

size_t pages_compact_workspace(int P) { return ((size_t)P + 1) * 4; }

cudaError_t pages_compact(int32_t* refs, int P, int32_t* tables, int64_t entries, int32_t* src, int32_t* dst, void* ws,
                          int32_t* status, cudaStream_t st) {
    int32_t* remap = entries > 0 ? static_cast<int32_t*>(ws) : nullptr;
    const bool one = entries <= kEntriesOfCluster;
    cudaError_t e = launch_cluster(pages_compact_kernel, P > kPagesOfOneBlock, st, refs, P, src, dst, remap, tables,
                                   one ? (int)entries : 0, status);
    if (e != cudaSuccess || one) return e;
    const int64_t blocks = (entries + 255) / 256;
    pages_remap_kernel<<<(unsigned)(blocks < 1216 ? blocks : 1216), 256, 0, st>>>(tables, entries, P, remap, dst, status);
    return cudaGetLastError();
}

size_t pages_copy_workspace(int P, int n) { return n <= kFewPairs ? 0 : (1 + 2 * (size_t)P + n) * 4; }

cudaError_t pages_copy(void* pool, int P, int64_t page_bytes, const int32_t* src, const int32_t* dst, int n, void* ws,
                       int32_t* status, cudaStream_t st) {
    const int64_t items = n * ((page_bytes + kCopyPiece - 1) / kCopyPiece);
    const unsigned grid = (unsigned)(items < kCopySms * 8 ? items : kCopySms * 8);
    if (n <= kFewPairs) {
        pages_copy_few_kernel<<<grid, kCopyThreads, 0, st>>>(static_cast<char*>(pool), page_bytes, src, dst, n, P, status);
        return cudaGetLastError();
    }
    int32_t* marks = static_cast<int32_t*>(ws);
    cudaError_t e = cudaMemsetAsync(marks, 0, (1 + 2 * (size_t)P) * 4, st);
    if (e != cudaSuccess) return e;
    const int blocks = (n + 255) / 256;
    pages_mark_kernel<<<blocks < 1216 ? blocks : 1216, 256, 0, st>>>(src, dst, n, P, marks, status);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    pages_copy_kernel<<<grid, kCopyThreads, 0, st>>>(
        static_cast<char*>(pool), page_bytes, src, dst, P, marks, status);
    return cudaGetLastError();
}

}  // namespace kda

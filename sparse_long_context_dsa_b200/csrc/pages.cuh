// Pages of a paged cache shared between requests: fork, release and compact, on the device.
//
// A page is free when its reference count is 0 (or less); an allocation takes the lowest free
// pages, so every result is a function of the arguments alone.  The calls read (ref_in, table_in) and
// leave their result in (ref_out, table_out), which may be the same arrays.
//
// scan_kernel finds the pages: one cluster of CTAs, each with a contiguous part of the counts,
// counts them, exchanges the totals through distributed shared memory and, in a second pass over its
// part (from L2), ranks every page.  Fork: the first n free pages.  Compact: n_live live pages;
// those behind the first n_live places (movers, from the last down) and the free places among
// them (holes, from the first up).  The clusters behind the first copy ref_in and table_in where the
// outputs are other arrays.  fork_kernel, move_kernel then move whole pages of every pool with
// 16-byte loads, four in flight per thread, and update the tables.
//
// Bound: HBM, every moved page read and written once; the counts and tables are small beside it.
#pragma once

#include <climits>

#include <cooperative_groups.h>

#include "common.cuh"

namespace dsa {
namespace pages {

namespace cg = cooperative_groups;

constexpr int kMaxPools = 8;
constexpr int kScanThreads = 1024;
constexpr int kPer = 4 * kScanThreads;                     // counts per CTA and step
constexpr int kThreads = 256;
constexpr int64_t kSegment = 16 * 1024;                    // bytes of a page that one CTA copies at a time

struct Pools {
    uint8_t *data[kMaxPools];
    int64_t bytes[kMaxPools];                              // of a page
    int first[kMaxPools + 1];                              // segments before the pool's, in a page of all pools
    int n;
};

// Exclusive prefix sum of v over the CTA (kScanThreads); total in `sum`.
__device__ __forceinline__ int block_prefix(int v, int *warp_sums, int &sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                                       // the previous step's sums are read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int w = warp_sums[lane];                               // 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return x - v + (warp ? before : 0);
}

struct Scan {
    const int32_t *ref_in;
    int32_t *ref_out;                                      // ref_in itself: not copied
    int64_t n_pages;
    const int32_t *table_in;
    int32_t *table_out;                                    // table_in itself: not copied
    int64_t table_n;
    int32_t *list;                                         // fork: first `want` free pages; compact: holes
    int want;
    int32_t *movers, *place, *new_index, *n_live, *n_moves;      // compact
};

template <bool kCompact>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const Scan a)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    __shared__ int warp_sums[32];
    __shared__ int totals[16];                             // live pages of every CTA of the cluster
    cg::cluster_group cluster = cg::this_cluster();
    const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x;
    if (blockIdx.x >= (unsigned)size) {
        // copies of the inputs
        const int64_t t = (int64_t)(blockIdx.x - size) * kScanThreads + tid;
        const int64_t nt = (int64_t)(gridDim.x - size) * kScanThreads;
        if (a.ref_out != a.ref_in)
            for (int64_t i = t; i < a.n_pages; i += nt) a.ref_out[i] = a.ref_in[i];
        if (a.table_out != a.table_in)
            for (int64_t i = t; i < a.table_n; i += nt) a.table_out[i] = a.table_in[i];
        return;
    }
    const int64_t steps = (a.n_pages + kPer - 1) / kPer, per = (steps + size - 1) / size;
    const int64_t s0 = min(steps, rank * per), s1 = min(steps, s0 + per);
    auto live4 = [&](int64_t s, bool (&v)[4]) {
        const int64_t i = s * kPer + 4 * tid;
        if (i + 4 <= a.n_pages && (reinterpret_cast<uintptr_t>(a.ref_in) & 15) == 0) {
            const int4 r = *reinterpret_cast<const int4 *>(a.ref_in + i);
            v[0] = r.x > 0;
            v[1] = r.y > 0;
            v[2] = r.z > 0;
            v[3] = r.w > 0;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = i + j < a.n_pages && a.ref_in[i + j] > 0;
        }
    };
    int mine = 0;
    for (int64_t s = s0; s < s1; ++s) {
        bool v[4];
        live4(s, v);
        mine += v[0] + v[1] + v[2] + v[3];
    }
    int total;
    block_prefix(mine, warp_sums, total);
    if (tid < size) cluster.map_shared_rank(totals, tid)[rank] = total;
    cluster.sync();
    int before = 0, n_live = 0;
    for (int i = 0; i < size; ++i) {
        before += i < rank ? totals[i] : 0;
        n_live += totals[i];
    }
    if (kCompact && rank == 0 && tid == 0) {
        *a.n_live = n_live;
        if (n_live == a.n_pages) *a.n_moves = 0;           // else the thread of page n_live writes it
    }
    for (int64_t s = s0; s < s1; ++s) {
        // free pages before this step: enough for a fork?
        if (!kCompact && s * kPer - before >= a.want) break;
        bool v[4];
        live4(s, v);
        const int cnt = v[0] + v[1] + v[2] + v[3];
        int sum;
        int rk = before + block_prefix(cnt, warp_sums, sum);
        before += sum;
        const int64_t i0 = s * kPer + 4 * tid;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t i = i0 + j;
            if (i >= a.n_pages) break;
            if (!kCompact) {
                if (!v[j] && i - rk < a.want) a.list[i - rk] = (int)i;
            } else {
                if (i == n_live) *a.n_moves = n_live - rk;
                int place = -1;
                if (v[j] && i < n_live) {
                    place = (int)i;
                } else if (v[j]) {
                    a.movers[n_live - 1 - rk] = (int)i;
                    place = -2 - (n_live - 1 - rk);
                } else if (i < n_live) {
                    a.list[i - rk] = (int)i;
                }
                a.place[i] = place;
                if (place >= -1) a.new_index[i] = place;
            }
            rk += v[j];
        }
    }
    if (!kCompact && rank == size - 1 && tid == 0) *a.n_live = n_live;
    cluster.sync();                                        // no CTA's shared memory goes away while it is written
}

// Segment `seg` (of all pools' segments of a page) of page src to page dst.
__device__ __forceinline__ void copy_segment(const Pools &p, int seg, int64_t src, int64_t dst)
{
    int k = 0;
    while (seg >= p.first[k + 1]) ++k;
    const int64_t at = (int64_t)(seg - p.first[k]) * kSegment, n = min(kSegment, p.bytes[k] - at) / 16;
    const uint4 *s = reinterpret_cast<const uint4 *>(p.data[k] + src * p.bytes[k] + at);
    uint4 *d = reinterpret_cast<uint4 *>(p.data[k] + dst * p.bytes[k] + at);
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (threadIdx.x + u * kThreads < n) v[u] = s[threadIdx.x + u * kThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (threadIdx.x + u * kThreads < n) d[threadIdx.x + u * kThreads] = v[u];
}

// One block row of the grid per fork; its CTAs share the copied page's segments and the child's
// table row with its counts (every entry is a chain of three dependent accesses: 939 entries in
// one CTA held a call of 64 forks up for 6 of its 12.7 us).
__global__ void __launch_bounds__(kThreads) fork_kernel(int32_t *ref_out, int64_t n_pages,
                                                        const int32_t *table_in, int32_t *table_out, int max_pages,
                                                        int n_req, const int32_t *parent, const int32_t *child,
                                                        const int32_t *length, int n, const int32_t *fresh,
                                                        const int32_t *n_live, const Pools pools)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    const int i = blockIdx.y, tid = threadIdx.x;
    auto in_range = [&](int j) {
        const int L = length[j];
        return (unsigned)parent[j] < (unsigned)n_req && (unsigned)child[j] < (unsigned)n_req && L >= 0 &&
               (int64_t)L <= (int64_t)max_pages * kPage;
    };
    // its fresh page is that of its rank among the forks that copy one; a child is nobody's parent
    // and no earlier fork's child
    const int c = child[i];
    int rank = 0, clash = 0;
    for (int j = tid; j < n; j += kThreads) {
        if (j < i && in_range(j) && length[j] % kPage) ++rank;
        if (parent[j] == c || (j < i && child[j] == c)) ++clash;
    }
    clash = __syncthreads_or(clash);
    __shared__ int sum;
    if (tid == 0) sum = 0;
    __syncthreads();
    rank = __reduce_add_sync(0xffffffffu, rank);
    if ((tid & 31) == 0 && rank) atomicAdd(&sum, rank);
    __syncthreads();
    rank = sum;
    const bool lead = blockIdx.x == 0 && tid == 0;
    if (!in_range(i) || clash) {
        if (lead) set_error(kErrPages);
        return;                                            // the child's row stays as it is
    }
    const int L = length[i], full = L / kPage;
    const int32_t *from = table_in + (int64_t)parent[i] * max_pages;
    int32_t *to = table_out + (int64_t)c * max_pages;
    // whether somebody held the page before the call: a count above 0 that no fork of this call set
    // (`fresh` ascends; most pages lie outside its range)
    const int n_fresh = (int)min((int64_t)n, n_pages - *n_live);
    const int fresh_lo = n_fresh > 0 ? fresh[0] : INT_MAX, fresh_hi = n_fresh > 0 ? fresh[n_fresh - 1] : -1;
    auto held = [&](int page) {
        if (page < 0 || page >= n_pages || ref_out[page] <= 0) return false;
        if (page < fresh_lo || page > fresh_hi) return true;
        int a = 0, b = n_fresh;
        while (a < b) {
            const int mid = (a + b) / 2;
            if (fresh[mid] < page) a = mid + 1;
            else b = mid;
        }
        return fresh[a] != page;                           // (a < n_fresh: page <= fresh_hi)
    };
    int src = -1, dst = -1;
    if (L % kPage) {
        src = from[full];
        if (rank < n_fresh && held(src)) dst = fresh[rank];
        if (dst < 0 && lead) set_error(kErrPages);         // a page that nobody holds, or none free
    }
    if (dst >= 0)
        for (int seg = blockIdx.x; seg < pools.first[pools.n]; seg += gridDim.x) copy_segment(pools, seg, src, dst);
    for (int v = blockIdx.x * kThreads + tid; v < max_pages; v += gridDim.x * kThreads) {
        int page = -1;
        if (v < full) {
            page = from[v];
            if (!held(page)) {                             // it cannot be shared
                set_error(kErrPages);
                page = -1;
            } else {
                atomicAdd(ref_out + page, 1);
            }
        } else if (v == full && dst >= 0) {
            page = dst;
            ref_out[page] = 1;
        }
        to[v] = page;
    }
}

// Rows req[i] cut to their first keep[i] tokens: their further pages are given back.  One cluster:
// it copies the inputs where the outputs are other arrays, meets, and walks the listed rows.
__global__ void __launch_bounds__(kScanThreads) release_kernel(const int32_t *ref_in, int32_t *ref_out, int64_t n_pages,
                                                               const int32_t *table_in, int32_t *table_out,
                                                               int max_pages, int n_req, const int32_t *req,
                                                               const int32_t *keep, int n)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    const int64_t t = (int64_t)blockIdx.x * kScanThreads + threadIdx.x, nt = (int64_t)gridDim.x * kScanThreads;
    if (ref_out != ref_in)
        for (int64_t i = t; i < n_pages; i += nt) ref_out[i] = ref_in[i];
    if (table_out != table_in)
        for (int64_t i = t; i < (int64_t)n_req * max_pages; i += nt) table_out[i] = table_in[i];
    __threadfence();
    cg::this_cluster().sync();
    // warps take the listed rows in pieces of 32 entries
    const int lane = threadIdx.x & 31;
    const int64_t pieces = (max_pages + 31) / 32;
    for (int64_t w = t >> 5; w < n * pieces; w += nt >> 5) {
        const int i = (int)(w / pieces), v = (int)(w % pieces) * 32 + lane;
        const int b = req[i], K = keep[i];
        bool twice = false;
        for (int j = lane; j < i; j += 32) twice |= req[j] == b;
        if (__any_sync(0xffffffffu, twice) || b < 0 || b >= n_req || K < 0) {
            if (v == 0) set_error(kErrPages);
            continue;
        }
        if (v >= max_pages || v < (K + (int64_t)kPage - 1) / kPage) continue;
        int32_t *e = table_out + (int64_t)b * max_pages + v;
        const int page = __ldcg(e);
        if (page == -1) continue;
        *e = -1;
        if (page < 0 || page >= n_pages) {
            set_error(kErrPages);
        } else if (atomicSub(ref_out + page, 1) <= 0) {    // was free already
            atomicAdd(ref_out + page, 1);
            set_error(kErrPages);
        }
    }
}

// Copies of the inputs of a call that changes nothing, where its outputs are other arrays.
__global__ void __launch_bounds__(kThreads) copy_tables_kernel(const int32_t *ref_in, int32_t *ref_out, int64_t n_pages,
                                                               const int32_t *table_in, int32_t *table_out, int64_t n)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x, nt = (int64_t)gridDim.x * kThreads;
    if (ref_out != ref_in)
        for (int64_t i = t; i < n_pages; i += nt) ref_out[i] = ref_in[i];
    if (table_out != table_in)
        for (int64_t i = t; i < n; i += nt) table_out[i] = table_in[i];
}

// The moves of a compaction (grid-strided over move and segment), the new places and the table.
__global__ void __launch_bounds__(kThreads) move_kernel(const int32_t *ref_in, int32_t *ref_out, int64_t n_pages,
                                                        const int32_t *table_in, int32_t *table_out, int64_t table_n,
                                                        const int32_t *holes, const int32_t *movers,
                                                        const int32_t *place, int32_t *new_index, const int32_t *n_moves,
                                                        const Pools pools)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x, nt = (int64_t)gridDim.x * kThreads;
    const int moves = *n_moves;
    for (int64_t j = t; j < moves; j += nt) {
        const int src = movers[j], dst = holes[j];
        const int count = ref_in[src];
        ref_out[dst] = count;
        ref_out[src] = 0;
        new_index[src] = dst;
    }
    for (int64_t i = t; i < table_n; i += nt) {
        const int page = table_in[i];
        int to = -1;
        if (page >= 0 && page < n_pages) {
            to = place[page];
            if (to <= -2) to = holes[-2 - to];
            else if (to < 0) set_error(kErrPages);         // the table names a free page
        } else if (page != -1) {
            set_error(kErrPages);
        }
        table_out[i] = to;
    }
    const int segs = pools.first[pools.n];
    for (int64_t u = blockIdx.x; u < (int64_t)moves * segs; u += gridDim.x) {
        const int j = (int)(u / segs);
        copy_segment(pools, (int)(u % segs), movers[j], holes[j]);
    }
}

}  // namespace pages
}  // namespace dsa

// New tokens' K and V rows quantised into the 8-bit paged cache.
//
// Cache: codes e4m3 [pages][4 groups][8 regions][K|V][8 tokens][192], scales fp32
// [pages][4][8][K|V]; value = code * scale.  A block (page, group, region, K or V) is 1,536
// contiguous bytes with one scale, the smallest power of two s in [2^-126, 2^120] with
// max|x| <= 448 s (0 for a block of zeros).  With a power of two x / s is exact, so a code is
// one e4m3 rounding of x (relative error <= 2^-4 above the e4m3 subnormals, whatever the
// scale), code * s is exactly a bf16 value, and raising a block's scale for a larger token
// only shifts exponents: exact but for codes that become e4m3 subnormals.
//
// The call's tokens that lie next to each other in the list, in one region of one request, are
// a run; one warp per (run, group, K or V) writes the run's rows.  A run that begins at row a > 0
// of its region keeps the rows before it: s' = max(s, scale of the new rows), and where s' > s
// their codes are rounded again, e4m3(code * s / s').  Rows behind the run stay as they are.
//
// Two runs of one region (a list ordered step by step over its requests, a ring that a chunk laps, a
// page that two requests append to) would write one block's codes and scale at once, in any order.
// Where the list names requests, CTAs before the others (one for 2,048 entries) look for one, beside
// them: each takes a share of the pages by their hash and enters their visits into a table in shared
// memory, then, only if a page is visited twice or out of order, those of the regions.  A chunk of 2,048
// tokens takes 3.7 us with it, 3.2 without (8,192: 10.3 / 9.4; 64: 2.5 / 2.4); a decode step's list names
// no requests and has no such CTA.
//
// Bound: HBM for bulk appends (two bytes read and one written per element), latency for a
// decode step's few tokens (position -> block table -> block).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace dsa {
namespace quant {

constexpr int kBlockBytes = kRegion * kD;          // one tensor's codes of a (page, group, region)
constexpr int kRegionBytesQ = 2 * kBlockBytes;     // K then V
constexpr int kRegionsPerPage = kPage / kRegion;

// The smallest power of two s in [2^-126, 2^120] with a <= 448 s; 0 for a = 0 (a >= 0).
// 448 = 1.75 * 2^8: for a = f 2^x, f in [1, 2), it is 2^(x - 8) when f <= 1.75, else 2^(x - 7).
__device__ __forceinline__ float block_scale(float a)
{
    if (a == 0.0f) return 0.0f;
    const uint32_t u = __float_as_uint(a);
    const int x = (int)(u >> 23) - 127;
    const int e = min(max(x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126), 120);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

constexpr int kThreads = 256;
constexpr int kSeenSlots = 4096;                   // of the table of pages or regions
constexpr int kSeenEntries = kSeenSlots / 2;       // list entries for each CTA that looks for two runs of a region

// Enters the list's visits of a page (2^kShift = 64 tokens) or of a region (8) that fall to part `part`
// of `parts` of the pages into a table.  True where one was there already or, for pages, a visit's
// regions descend.
template <int kShift>
__device__ __forceinline__ bool visits_twice(uint32_t (&seen)[kSeenSlots], int64_t n_pages,
                                             const int32_t *__restrict__ block_table, int max_pages,
                                             const int32_t *__restrict__ q_req, int n_req,
                                             const int32_t *__restrict__ q_pos, int n, unsigned part, unsigned parts)
{
    constexpr int kEach = 8;                       // entries of a thread whose loads are in flight at once
    for (int i = threadIdx.x; i < kSeenSlots; i += kThreads) seen[i] = 0u;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    bool twice = false;
    for (int64_t e0 = threadIdx.x; e0 - threadIdx.x < n; e0 += kEach * kThreads) {
        int pos[kEach], req[kEach], pos_p[kEach], req_p[kEach], page[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int64_t e = e0 + u * kThreads;
            pos[u] = e < n ? q_pos[e] : -1;
            req[u] = e < n ? q_req[e] : -1;
            const bool first = lane == 0 && e > 0 && e < n;              // (the other lanes' by shuffles)
            pos_p[u] = first ? q_pos[e - 1] : -1;
            req_p[u] = first ? q_req[e - 1] : -1;
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int x = __shfl_up_sync(0xffffffffu, pos[u], 1), y = __shfl_up_sync(0xffffffffu, req[u], 1);
            if (lane > 0) {
                pos_p[u] = x;
                req_p[u] = y;
            }
            const bool here = req[u] >= 0 && req[u] < n_req && pos[u] >= 0 && pos[u] / kPage < max_pages;
            const bool goes_on = req[u] == req_p[u] && (pos[u] >> kShift) == (pos_p[u] >> kShift);
            if (kShift == 6 && here && goes_on && (pos[u] >> 3) < (pos_p[u] >> 3)) twice = true;
            page[u] = here && !goes_on ? block_table[(int64_t)req[u] * max_pages + pos[u] / kPage] : -1;
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            if (page[u] < 0 || page[u] >= n_pages) continue;
            const uint32_t h = ((uint32_t)page[u] + 1u) * 0x9E3779B1u;   // multiplicative hash: its upper bits choose the part
            if (__umulhi(h, parts) != part) continue;
            const uint32_t key = kShift == 6 ? (uint32_t)page[u] + 1u
                                             : (uint32_t)page[u] * kRegionsPerPage + (uint32_t)(pos[u] % kPage / kRegion) + 1u;
            uint32_t slot = ((key * 0x9E3779B1u ^ (key >> 3)) * 0x85EBCA6Bu) >> 20;
            for (int probe = 0; probe < kSeenSlots; ++probe, slot = (slot + 1) % kSeenSlots) {
                const uint32_t there = atomicCAS(&seen[slot], 0u, key);
                twice |= there == key;
                if (there == 0u || there == key) break;
            }
        }
    }
    return twice;
}

// An error where a region has two runs.  Lists as they are (pages visited once, their regions in
// order) are done with after the first look.
__device__ __forceinline__ void find_second_runs(int64_t n_pages, const int32_t *block_table, int max_pages,
                                                 const int32_t *q_req, int n_req, const int32_t *q_pos, int n,
                                                 unsigned part, unsigned parts)
{
    __shared__ uint32_t seen[kSeenSlots];          // page or region of the cache, plus 1; 0: none
    if (!__syncthreads_or(visits_twice<6>(seen, n_pages, block_table, max_pages, q_req, n_req, q_pos, n, part, parts))) return;
    if (visits_twice<3>(seen, n_pages, block_table, max_pages, q_req, n_req, q_pos, n, part, parts)) set_error(kErrAppendTwice);
}

// Two bf16 (packed) times r -> two e4m3 codes (bits 15:0).
__device__ __forceinline__ uint32_t codes2(uint32_t v, float r) { return cvt_e4m3x2(bf16_lo(v) * r, bf16_hi(v) * r); }

// kTok list entries per CTA (8 warps: group w / 2, K or V w % 2): the runs that begin among them.
// The first `looks` CTAs look for regions with two runs.
template <int kTok>
__global__ void __launch_bounds__(kThreads) kv_append_quant_kernel(
    uint8_t *__restrict__ cache, float *__restrict__ scale, int64_t n_pages, const int32_t *__restrict__ block_table,
    int max_pages, const int32_t *__restrict__ q_req, int n_req, const int32_t *__restrict__ q_pos, int n,
    const __nv_bfloat16 *__restrict__ new_k, const __nv_bfloat16 *__restrict__ new_v, unsigned looks)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp >> 1, which = warp & 1;
    if (blockIdx.x < looks) {
        find_second_runs(n_pages, block_table, max_pages, q_req, n_req, q_pos, n, blockIdx.x, looks);
        return;
    }
    const int i0 = (int)(blockIdx.x - looks) * kTok;
    // lane l: list entry i0 - 1 + l (the entry before the CTA's, its own, and the 8 a run of the
    // last one can reach)
    const int e = i0 - 1 + lane;
    const bool have = lane < kTok + 9 && e >= 0 && e < n;
    const int pos = have ? q_pos[e] : -1;
    const int req = have ? (q_req ? q_req[e] : e) : -1;
    const int pos_p = __shfl_up_sync(0xffffffffu, pos, 1), req_p = __shfl_up_sync(0xffffffffu, req, 1);
    const unsigned have_m = __ballot_sync(0xffffffffu, have);
    const bool prev = lane > 0 && ((have_m >> (lane - 1)) & 1u);
    const unsigned cont_m = __ballot_sync(0xffffffffu, have && prev && req == req_p && (pos >> 3) == (pos_p >> 3));
    const unsigned desc_m = __ballot_sync(0xffffffffu, have && prev && pos <= pos_p);
    const __nv_bfloat16 *src = which ? new_v : new_k;
#pragma unroll 1
    for (int l0 = 1; l0 <= kTok; ++l0) {
        if (!((have_m >> l0) & 1u) || ((cont_m >> l0) & 1u)) continue;     // no entry, or not a run's first
        // the run: entries l0 .. l0 + len - 1, ascending positions of one region
        const unsigned after = cont_m >> (l0 + 1);
        const unsigned good = after & ~(desc_m >> (l0 + 1));
        const int len = 1 + __ffs(~good) - 1;
        if (((after >> (len - 1)) & 1u) && threadIdx.x == 0) set_error(kErrAppendOrder);
        const int p0 = __shfl_sync(0xffffffffu, pos, l0), b = __shfl_sync(0xffffffffu, req, l0);
        const unsigned rows = __reduce_or_sync(0xffffffffu, lane >= l0 && lane < l0 + len ? 1u << (pos & 7) : 0u);
        const bool in_table = b >= 0 && b < n_req && p0 >= 0 && p0 / kPage < max_pages;
        const int64_t page = in_table ? block_table[(int64_t)b * max_pages + p0 / kPage] : -1;
        // (the new rows travel while the page is looked up)
        // chunk c = lane + 32 u: row c / 24 of the region, its elements 8 (c % 24) .. + 7
        uint4 x[6];
#pragma unroll
        for (int u = 0; u < 6; ++u) {
            const int c = lane + 32 * u, r = c / 24, cc = c % 24;
            x[u] = make_uint4(0, 0, 0, 0);
            if ((rows >> r) & 1u) {
                const int64_t i = i0 - 1 + l0 + __popc(rows & ((1u << r) - 1u));
                x[u] = __ldg(reinterpret_cast<const uint4 *>(src + (i * kG + g) * kD + cc * 8));
            }
        }
        if (page < 0 || page >= n_pages) {
            if (threadIdx.x == 0) set_error(kErrAttnIndex);
            continue;
        }
        const int64_t rid = (page * kG + g) * kRegionsPerPage + (p0 % kPage) / kRegion;
        uint8_t *block = cache + rid * kRegionBytesQ + which * kBlockBytes;
        float *sp = scale + rid * 2 + which;
        const int first = __ffs(rows) - 1;                                  // rows below it are kept
        const float s_old = first > 0 ? *sp : 0.0f;
        uint2 old[6];
        __nv_bfloat162 mx2 = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < 6; ++u) {
            const int c = lane + 32 * u, r = c / 24, cc = c % 24;
            old[u] = make_uint2(0, 0);
            if (r < first) old[u] = *reinterpret_cast<const uint2 *>(block + r * kD + cc * 8);
        }
#pragma unroll
        for (int u = 0; u < 6; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mx2 = __hmax2(mx2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j])));
        }
        float mx = fmaxf(__low2float(mx2), __high2float(mx2));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float s = fmaxf(s_old, block_scale(mx));
        const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;                   // exact for a power of two
        const float ratio = s_old * inv;
#pragma unroll
        for (int u = 0; u < 6; ++u) {
            const int c = lane + 32 * u, r = c / 24, cc = c % 24;
            uint2 *dst = reinterpret_cast<uint2 *>(block + r * kD + cc * 8);
            if ((rows >> r) & 1u) {
                *dst = make_uint2(codes2(x[u].x, inv) | (codes2(x[u].y, inv) << 16),
                                  codes2(x[u].z, inv) | (codes2(x[u].w, inv) << 16));
            } else if (r < first && s > s_old) {
                uint32_t w[2] = {old[u].x, old[u].y};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t lo = cvt_e4m3x2(e4m3_to_f32(w[j]) * ratio, e4m3_to_f32(w[j] >> 8) * ratio);
                    const uint32_t hi = cvt_e4m3x2(e4m3_to_f32(w[j] >> 16) * ratio, e4m3_to_f32(w[j] >> 24) * ratio);
                    w[j] = lo | (hi << 16);
                }
                *dst = make_uint2(w[0], w[1]);
            }
        }
        if (lane == 0) *sp = s;
    }
}

}  // namespace quant
}  // namespace dsa

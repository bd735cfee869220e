// Window GQA of many queries of a request over the 8-bit paged cache (layout and scales:
// append_quant.cuh): neighbouring queries' windows are almost the same tokens.
//
// A CTA takes 8 queries of the list and one KV group: 128 rows (query, head), the MMA's M.  It
// handles them in runs: queries of one request whose positions lie within 56 of one another share
// one stream of their windows' pages (64 tokens, 24 KiB, a ring of 4); rows of the
// other runs are masked.  A prefill chunk's 8 queries are one run.
//  * S = q K^T: tcgen05.mma kind::f8f6f4 straight from the codes (K-major, 64-byte swizzle), q as
//    two e4m3 terms of 2^-e q that accumulate into the same S.  The largest of 2^-e q is above 224
//    and the terms end at the subnormal step 2^-9, so q is off by at most 2^-10 / 224 < 2^-17 of the
//    head's largest element (the row kernel's second term, 16 times finer, needs a product of its own);
//  * softmax: thread = row (TMEM lane), fp32, log2 units, no exchange between threads.  As in the
//    row kernel, the sum l has a reference m and the weights P' = 2^(s - m) sV 2^(m - M) one of
//    their own, both moved only when a tile passes them by 2^10 (O is then rescaled in TMEM);
//  * O += P' V: P' as three e5m2 terms (cut off, cut off, rounded: 2^-9 relative, ending at 2^-22
//    of a row's largest) in shared memory, V's codes MN-major, N = 192.
// V rows that no query of the run attends are zeroed in shared memory.  A NaN code at a token that
// only some of them attend would reach the others (their P' is 0, but 0 * NaN is not): such
// tokens are looked at, and a run that has one is done again, query by query.
// Bound: neither the tensor pipe (22 % busy with its 12 + 6 instructions per 64 tokens and 8 queries) nor
// memory (L2 7 %), but a CTA's chain, set-up and q's conversion - S - softmax of 128 rows - P' V, with
// one CTA per SM: 512 queries, a window of 512, are 256 CTAs, two rounds, 42.7 us (SMs 78 % active).
#pragma once

#include "attention_quant_tc.cuh"

namespace dsa {
namespace attnqb {

using attnq::ex2;
using attnq::kRegBytes;
using attnq::Params;
using attnqt::desc_hi;
using attnqt::desc_lo;
using attnqt::hsub2;
using attnqt::mma_f8;

constexpr int kQueries = 8;
constexpr int kTileBytes = quant::kRegionsPerPage * kRegBytes;   // a page of one group: 24 KiB
constexpr int kStages = 4;
constexpr int kThreads = 352;                                    // warps 0-3, 4-7 softmax of even and odd tiles, 8 S, 9 loads, 10 P' V
constexpr int kSpan = 56;                                        // positions of a run lie this close to its first
constexpr int kOCol = 128;                                       // TMEM: S 0, 64; O 128 .. 319, 320 .. 511 (even and odd tiles)
constexpr int kTmemCols = 512;
constexpr float kBase = 5.0f;                                    // log2 of a weight at its reference
constexpr float kSlack = 10.0f;                                  // log2 units a reference may lag behind

struct Smem {
    uint8_t q[2][3 * 128 * 64];                                  // hi, lo: [64-dim block][row][64], 64-byte swizzle
    uint8_t p[2][3][128 * 64];                                   // [buffer][term][row][64 tokens], 64-byte swizzle
    float4 scale[kStages][8];                                    // K's, V's, log2 of V's
    int there[kStages];                                          // the page is there
    float qscale[128];
    float4 merge[2][128];                                        // m, M, l of a row's even and odd tiles
    int pos[kQueries], req[kQueries];
    int run_end[kQueries];                                       // first query behind the run that begins here
    int nan[2];                                                  // run n (by parity) met a NaN code at a partly attended token: n + 1
    uint64_t full[kStages], empty[kStages], s_full[2], s_read[2], p_ready[2], pv_done[2], merged, run_done;
    uint32_t tmem;
};
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kTileBytes + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");

constexpr uint32_t kIdescS = umma_idesc_e4m3(128, kPage);
constexpr uint32_t kIdescO = umma_idesc_e4m3(128, kD) | (1u << 7) | (1u << 16);    // P' e5m2 K-major, V MN-major

// 32 consecutive fp32 columns of this warp's 32 TMEM lanes written from registers (not waited for).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
          "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
          "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
          "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}

// The next run of a CTA's queries: [u0, u1), request b, tokens lo .. hi of its windows.
struct Run {
    int u0, u1, b, lo, hi, tiles;
};

__device__ __forceinline__ Run run_at(const Smem &sm, const Params &p, int u0, bool single)
{
    Run r;
    r.u0 = u0;
    r.u1 = single ? u0 + 1 : sm.run_end[u0];
    r.b = sm.req[u0];
    r.lo = INT_MAX;
    r.hi = -1;
    for (int u = u0; u < r.u1; ++u) {
        r.lo = min(r.lo, max(0, sm.pos[u] - p.window + 1));
        r.hi = max(r.hi, sm.pos[u]);
    }
    r.tiles = r.hi < 0 ? 0 : r.hi / kPage - r.lo / kPage + 1;
    return r;
}

__global__ void __launch_bounds__(kThreads, 1)
    window_attn_band_kernel(const __grid_constant__ CUtensorMap tmap, const Params p)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    if (threadIdx.x == 0) prefetch_tensormap(&tmap);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem &sm = *reinterpret_cast<Smem *>(ring + kStages * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.full[i], 2);                           // the load is announced; the scales are there
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_read[i], 4);
            mbar_init(&sm.p_ready[i], 4);
            mbar_init(&sm.pv_done[i], 1);
        }
        mbar_init(&sm.merged, 8);
        mbar_init(&sm.run_done, 11);                             // every role: none is two runs behind another
        sm.nan[0] = sm.nan[1] = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(&sm.tmem, kTmemCols);
    pdl_wait();      // the previous kernel's results are visible from here on
    const int blocks = (p.nq + kQueries - 1) / kQueries;
    const int g = (int)blockIdx.x / blocks, q0 = ((int)blockIdx.x % blocks) * kQueries;
    const int n_q = min(kQueries, p.nq - q0);
    if (tid < kQueries) {
        int pos = -1, req = -1;
        if (tid < n_q) {
            pos = p.q_pos[q0 + tid];
            req = p.q_req ? p.q_req[q0 + tid] : q0 + tid;
            if (pos >= 0 && (req < 0 || req >= p.n_req)) {
                set_error(kErrAttnIndex);
                pos = -1;
            }
        }
        sm.pos[tid] = pos;                                       // -1: attends nothing
        sm.req[tid] = req;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9 && lane < kQueries) {
        const int p0 = sm.pos[lane];
        int e = lane + 1;
        while (p0 >= 0 && e < kQueries && sm.pos[e] >= 0 && sm.req[e] == sm.req[lane] && abs(sm.pos[e] - p0) <= kSpan) ++e;
        sm.run_end[lane] = e;
    }
    const uint32_t tmem = sm.tmem;
    // q of every query: 2^-e q = hi + lo in e4m3; 8 threads share a head, thread c of them holds dims
    // 8 c .. 8 c + 7 of every 64-dim block
    if (warp < 8) {
        const int h = (tid >> 3) & 15, c = tid & 7, even = tid >> 7;     // queries even, even + 2, ..
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q + ((int64_t)q0 * kHQ + g * kHeadsPerGroup + h) * kD + 8 * c);
        constexpr int kNext = kHQ * kD / 8;                      // 16-byte pieces from one query to the next
        uint4 ahead[2][3];                                       // the next two queries' pieces, in flight
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 3; ++j)
                ahead[u][j] = even + 2 * u < n_q ? __ldg(src + (even + 2 * u) * kNext + 8 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
        for (int u = even; u < n_q; u += 2) {
            uint4 qv[3];
            __nv_bfloat162 a2 = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                qv[j] = ahead[0][j];
                ahead[0][j] = ahead[1][j];
                if (u + 4 < n_q) ahead[1][j] = __ldg(src + (u + 4) * kNext + 8 * j);
                const uint32_t w[4] = {qv[j].x, qv[j].y, qv[j].z, qv[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) a2 = __hmax2(a2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
            }
            float a = fmaxf(__low2float(a2), __high2float(a2));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
            const float s = quant::block_scale(a), inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
            const int r = 16 * u + h;
            if (c == 0) sm.qscale[r] = s * p.scale_log2;
            const int at = r * 64 + ((((c >> 1) ^ ((r >> 1) & 3)) << 4) | ((c & 1) << 3));
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const uint32_t w[4] = {qv[j].x, qv[j].y, qv[j].z, qv[j].w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = bf16_lo(w[i]) * inv, y = bf16_hi(w[i]) * inv;
                    hi[i] = cvt_e4m3x2(x, y);
                    const uint32_t back = attnq::e4m3x2_to_f16x2((uint16_t)hi[i]);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&back));
                    lo[i] = cvt_e4m3x2(x - f.x, y - f.y);
                }
                *reinterpret_cast<uint2 *>(sm.q[0] + j * 8192 + at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                *reinterpret_cast<uint2 *>(sm.q[1] + j * 8192 + at) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            }
        }
        fence_proxy_async();
    }
    // q, the runs; the loads' warp does not wait for q
    __syncwarp();
    if (warp == 9) asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
    else asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");

    // Every role walks the same runs: after a run that met a NaN (read behind the run's barrier), its
    // queries one by one.
    int n_run = 0, u0 = 0, single_until = 0;
    bool ok = true;
    auto next = [&](const Run &r) {                              // the run is done: where the next one begins
        const int met = *reinterpret_cast<volatile int *>(&sm.nan[n_run & 1]);
        ++n_run;
        if (u0 >= single_until && r.u1 - r.u0 > 1 && met == n_run) {
            single_until = r.u1;
        } else {
            u0 = r.u1;
        }
    };
    int tg = 0;                                                  // tiles before this one, over all runs

    if (warp == 9) {
        // ---- loads: a page of the group at a time
        while (u0 < n_q && ok) {
            const Run r = run_at(sm, p, u0, u0 < single_until);
            for (int ti = 0; ti < r.tiles; ++ti, ++tg) {
                const int st = tg % kStages, v = r.lo / kPage + ti;
                int page = -1;
                if (v < p.max_pages) page = p.block_table[(int64_t)r.b * p.max_pages + v];
                const bool there = page >= 0 && page < p.n_pages;
                if (!there && lane == 0) set_error(kErrAttnIndex);
                const int block = there ? (page * kG + g) * quant::kRegionsPerPage : 0;
                // the regions that hold a token of the windows (lane l: region l), each in a box of its
                // own: one box of the page's 8 takes 6,000 cycles to land, 8 boxes 1,600
                const int tok = v * kPage + 8 * lane;
                const bool held = there && lane < 8 && tok <= r.hi && tok + 7 >= r.lo;
                const unsigned boxes = __popc(__ballot_sync(0xffffffffu, held));
                const float2 sc = held ? __ldg(p.scale + block + lane) : make_float2(0.0f, 0.0f);
                if (tg >= kStages) ok = __all_sync(0xffffffffu, mbar_wait_sleep(&sm.empty[st], (unsigned)(tg / kStages - 1) & 1u));
                if (!ok) break;
                if (lane == 0) {
                    if (boxes) mbar_arrive_expect_tx(&sm.full[st], boxes * kRegBytes);
                    else mbar_arrive(&sm.full[st]);
                    sm.there[st] = there;
                }
                __syncwarp();
                if (held) tma_load_3d(ring + st * kTileBytes + lane * kRegBytes, &tmap, 0, (block + lane) * 16, 0, &sm.full[st]);
                if (lane < 8) sm.scale[st][lane] = make_float4(sc.x, sc.y, log2f(sc.y), 0.0f);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.full[st]);
            }
            if (ok && lane == 0) mbar_arrive(&sm.run_done);
            ok = __all_sync(0xffffffffu, ok && mbar_wait_sleep(&sm.run_done, (unsigned)n_run & 1u));
            next(r);
        }
        // none of this warp's loads is in flight when the CTA ends, after a wait that gave up as well
        __syncwarp();
        if (lane == 0)
            for (int s = 0; s < kStages && s < tg; ++s) {
                const int last = tg - 1 - (tg - 1 - s) % kStages;
                mbar_wait(&sm.full[s], (unsigned)(last / kStages) & 1u);
            }
        __syncwarp();
    } else if (warp == 8) {
        // ---- S, at most two tiles ahead of the weights (one elected lane).  K: rows of 64 bytes, 8 of a region
        // 512 bytes, regions 3 KiB apart; q: rows of 64 bytes
        if (elect_one()) {
            const uint32_t k_lo = desc_lo(smem_u32(ring), 16);
            constexpr uint32_t kKvHi = desc_hi(kRegBytes, 4), kRowsHi = desc_hi(512, 4);
            while (u0 < n_q && ok) {
                const Run r = run_at(sm, p, u0, u0 < single_until);
                for (int ti = 0; ti < r.tiles && ok; ++ti, ++tg) {
                    const int st = tg % kStages;
                    ok = mbar_wait(&sm.full[st], (unsigned)(tg / kStages) & 1u) &&
                         (ti < 2 || mbar_wait(&sm.s_read[tg & 1], (unsigned)((tg - 2) >> 1) & 1u));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t b = k_lo + (uint32_t)st * (kTileBytes >> 4), d = tmem + 64 * (tg & 1);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int ks = 0; ks < 6; ++ks) {
                            const uint32_t a = desc_lo(smem_u32(sm.q[term]) + (ks >> 1) * 8192 + (ks & 1) * 32, 16);
                            const uint32_t bk = b + (((ks >> 1) * 1024 + (ks & 1) * 32) >> 4);
                            if (term == 0 && ks == 0) mma_f8<false>(d, a, kRowsHi, bk, kKvHi, kIdescS);
                            else mma_f8<true>(d, a, kRowsHi, bk, kKvHi, kIdescS);
                        }
                    umma_commit(&sm.s_full[tg & 1]);
                }
                if (ok) mbar_arrive(&sm.run_done);
                ok = ok && mbar_wait(&sm.run_done, (unsigned)n_run & 1u);
                next(r);
            }
            // every commit has arrived when TMEM is released, after a wait that gave up as well (umma_commit)
            for (int b = 0; b < 2; ++b) commits_done(&sm.s_full[b], (tg + 1 - b) / 2);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ---- O += P' V as the weights are there (one elected lane).  V^T: 64-dim blocks 1 KiB apart, 8-token
        // groups 3 KiB apart; P': rows of 64 bytes
        if (elect_one()) {
            const uint32_t v_lo = desc_lo(smem_u32(ring) + 512, 1024);
            constexpr uint32_t kKvHi = desc_hi(kRegBytes, 4), kRowsHi = desc_hi(512, 4);
            while (u0 < n_q && ok) {
                const Run r = run_at(sm, p, u0, u0 < single_until);
                for (int ti = 0; ti < r.tiles && ok; ++ti, ++tg) {
                    ok = mbar_wait(&sm.p_ready[tg & 1], (unsigned)(tg >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t b = v_lo + (uint32_t)(tg % kStages) * (kTileBytes >> 4), d = tmem + kOCol + kD * (tg & 1);
#pragma unroll
                    for (int term = 0; term < 3; ++term) {
                        const uint32_t a = desc_lo(smem_u32(sm.p[tg & 1][term]), 16);
                        if (term == 0 && ti < 2) mma_f8<false>(d, a, kRowsHi, b, kKvHi, kIdescO);
                        else mma_f8<true>(d, a, kRowsHi, b, kKvHi, kIdescO);
                        mma_f8<true>(d, a + (32 >> 4), kRowsHi, b + (4 * kRegBytes >> 4), kKvHi, kIdescO);
                    }
                    umma_commit(&sm.empty[tg % kStages]);
                    umma_commit(&sm.pv_done[tg & 1]);
                }
                if (ok) mbar_arrive(&sm.run_done);
                ok = ok && mbar_wait(&sm.run_done, (unsigned)n_run & 1u);
                next(r);
            }
            for (int b = 0; b < 2; ++b) commits_done(&sm.pv_done[b], (tg + 1 - b) / 2);
            for (int s = 0; s < kStages; ++s) commits_done(&sm.empty[s], (tg + kStages - 1 - s) / kStages);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = row 16 u + h, the tiles of its group's parity
        const int grp = tid >> 7, row = tid & 127, wg = warp & 3, u = row >> 4;
        const uint32_t trow = tmem + ((uint32_t)(32 * wg) << 16), tcol_o = trow + kOCol + kD * grp;
        const float qf = sm.qscale[row];
        const int64_t head = (int64_t)(q0 + u) * kHQ + g * kHeadsPerGroup + (row & 15);
        bool landed = true;
        // a wait that gives up leaves the error flag and garbage; the later ones are then short
        auto wait = [&](uint64_t *bar, unsigned parity) {
            if (!mbar_wait(bar, parity, landed ? kWaitLimitCycles : 1ll << 22)) landed = false;
        };
        while (u0 < n_q) {
            const Run r = run_at(sm, p, u0, u0 < single_until);
            const bool mine = u >= r.u0 && u < r.u1;
            const int pos = mine ? sm.pos[u] : -1, t_lo = mine ? max(0, pos - p.window + 1) : 0;
            // tokens that every query of the run attends: all_lo .. all_hi
            int all_lo = 0, all_hi = INT_MAX;
            for (int i = r.u0; i < r.u1; ++i) {
                all_lo = max(all_lo, max(0, sm.pos[i] - p.window + 1));
                all_hi = min(all_hi, sm.pos[i]);
            }
            float m = -INFINITY, M = -INFINITY, mref = 0.0f, c = 0.0f, l = 0.0f;
            for (int ti = 0; ti < r.tiles; ++ti, ++tg) {
                if ((tg & 1) != grp) continue;
                const int st = tg % kStages, t0 = (r.lo / kPage + ti) * kPage;
                wait(&sm.full[st], (unsigned)(tg / kStages) & 1u);
                const bool there = sm.there[st] != 0;
                const bool whole = there && t0 >= all_lo && t0 + kPage - 1 <= all_hi;
                if (!whole && row < kPage) {
                    // V rows that nobody attends: zero; that some attend: looked at for NaN
                    const int t = t0 + row;
                    const bool none = !there || t < r.lo || t > r.hi;
                    if (none || t < all_lo || t > all_hi) {
                        uint8_t *v = ring + st * kTileBytes + (row >> 3) * kRegBytes + 512 + (row & 7) * 64;
                        bool bad = false;
#pragma unroll 4
                        for (int i = 0; i < 12; ++i) {
                            uint4 *x = reinterpret_cast<uint4 *>(v + (i >> 2) * 1024 + (i & 3) * 16);
                            if (none) {
                                *x = make_uint4(0, 0, 0, 0);
                            } else {
                                const uint4 y = *x;
                                bad |= (__vcmpeq4(y.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(y.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu) |
                                        __vcmpeq4(y.z & 0x7F7F7F7Fu, 0x7F7F7F7Fu) | __vcmpeq4(y.w & 0x7F7F7F7Fu, 0x7F7F7F7Fu)) != 0u;
                            }
                        }
                        if (bad) sm.nan[n_run & 1] = n_run + 1;
                    }
                }
                wait(&sm.s_full[grp], (unsigned)(tg >> 1) & 1u);
                __syncwarp();
                tc_fence_after();
                float s[64];
                {
                    float a[32], b[32];
                    tmem_ld32x2(trow + 64 * grp, trow + 64 * grp + 32, a, b);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        s[i] = a[i];
                        s[32 + i] = b[i];
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.s_read[grp]);
                // a score is s[i] fr, fr = qf times K's scale where the whole warp attends the whole tile; else
                // the scores themselves (-inf: not attended) take the place of s and fr is 1
                const bool plain = whole && __all_sync(0xffffffffu, mine);
                if (!plain) {
#pragma unroll
                    for (int rg = 0; rg < 8; ++rg) {
                        const float f = qf * sm.scale[st][rg].x;
#pragma unroll
                        for (int i = 8 * rg; i < 8 * rg + 8; ++i) {
                            const int t = t0 + i;
                            s[i] = there && t >= t_lo && t <= pos ? s[i] * f : -INFINITY;
                        }
                    }
                }
                float mx = -INFINITY, mv = -INFINITY;
#pragma unroll
                for (int rg = 0; rg < 8; ++rg) {
                    const float4 sc = sm.scale[st][rg];
                    const float *x = s + 8 * rg;
                    float y = fmaxf(fmaxf(x[0], x[1]), x[2]);
                    y = fmaxf(fmaxf(y, x[3]), x[4]);
                    y = fmaxf(fmaxf(y, x[5]), x[6]);
                    y = fmaxf(y, x[7]) * (plain ? qf * sc.x : 1.0f);
                    mx = fmaxf(mx, y);
                    mv = fmaxf(mv, y + sc.z);
                }
                // this group's tile before (tg - 2) is in O, and its P' has been read
                if (ti >= 2) wait(&sm.pv_done[grp], (unsigned)((tg - 2) >> 1) & 1u);
                __syncwarp();
                // the references move where a token passes one by more than the slack, or there is none
                const bool move = mx > m + kSlack || mv > M + kSlack || (M == -INFINITY && mx > -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                    float al = 1.0f, ao = 1.0f;
                    if (move) {
                        const float a = fmaxf(m, mx), d = fmaxf(M, mv);
                        if (a != m) al = exp2f(m - a);
                        if (d != M) ao = exp2f(M - d);
                        m = a;
                        M = d;
                        mref = a == -INFINITY ? 0.0f : a - kBase;
                        c = d == -INFINITY ? 0.0f : exp2f(fminf(a - d, 126.0f));
                        l *= al;
                    }
                    if (ti >= 2 && __any_sync(0xffffffffu, ao != 1.0f)) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < kD; c0 += 32) {
                            float o[32];
                            tmem_ld32(tcol_o + c0, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= ao;
                            tmem_st32(tcol_o + c0, o);
                        }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        tc_fence_before();
                    }
                }
                // P' in three e5m2 terms: the upper bytes of w, of what they leave, and of the rest,
                // rounded; 16 tokens at a time
                uint8_t *dst = sm.p[grp][0] + row * 64;
                float2 add2 = make_float2(0.0f, 0.0f);
                const float2 mr2 = make_float2(-mref, -mref), one2 = make_float2(1.0f, 1.0f);
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t w[8];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float4 sc = sm.scale[st][2 * ch + hf];
                        const float fr = plain ? qf * sc.x : 1.0f, f = fminf(sc.y * c, 8.5070592e37f);     // 2^126
                        const float2 fr2 = make_float2(fr, fr), f2 = make_float2(f, f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = 16 * ch + 8 * hf + 2 * i;
                            const float2 x = ffma2(make_float2(s[e], s[e + 1]), fr2, mr2);
                            const float2 p2 = make_float2(ex2(x.x), ex2(x.y));
                            add2 = ffma2(p2, one2, add2);
                            const float2 y = fmul2(p2, f2);
                            w[4 * hf + i] = attnq::pack_f16x2(y.x, y.y);
                        }
                    }
                    const int at = (ch ^ ((row >> 1) & 3)) << 4;
#pragma unroll
                    for (int term = 0; term < 3; ++term) {
                        if (term == 2) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] += 0x00800080u;
                        }
                        *reinterpret_cast<uint4 *>(dst + term * (128 * 64) + at) =
                            make_uint4(__byte_perm(w[0], w[1], 0x7531), __byte_perm(w[2], w[3], 0x7531),
                                       __byte_perm(w[4], w[5], 0x7531), __byte_perm(w[6], w[7], 0x7531));
                        if (term < 2) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = hsub2(w[i], w[i] & 0xFF00FF00u);
                        }
                    }
                }
                l += add2.x + add2.y;
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_ready[grp]);
            }
            // ---- the run's rows: the two groups' sums and references meet, each group writes half of the dims
            sm.merge[grp][row] = make_float4(m, M, l, 0.0f);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.merged);
            for (int x = max(tg - 2, tg - r.tiles); x < tg; ++x) wait(&sm.pv_done[x & 1], (unsigned)(x >> 1) & 1u);
            wait(&sm.merged, (unsigned)n_run & 1u);
            __syncwarp();
            tc_fence_after();
            float w[2] = {0.0f, 0.0f}, e2;                       // of each group's O, then of their sum
            {
                const float4 a = sm.merge[0][row], b = sm.merge[1][row];
                m = fmaxf(a.x, b.x);
                M = fmaxf(a.y, b.y);
                // (a sum without a reference is 0 or NaN)
                l = (a.x == -INFINITY ? a.z : a.z * exp2f(a.x - m)) + (b.x == -INFINITY ? b.z : b.z * exp2f(b.x - m));
                // 1 / l, then 2^(M - m) (their product may be below fp32's range); 0 for a row with no token or no
                // V; a NaN sum stays NaN (no comparison holds for it)
                const float f = l > 0.0f ? 1.0f / l : l;
                e2 = M > -INFINITY ? exp2f(M - m) : 0.0f;
                w[0] = a.y == -INFINITY ? 0.0f : exp2f(a.y - M);
                w[1] = b.y == -INFINITY ? 0.0f : exp2f(b.y - M);
                w[0] *= f;
                w[1] *= f;
            }
            const bool has[2] = {r.tiles >= 2 || (r.tiles == 1 && ((tg - 1) & 1) == 0), r.tiles >= 2 || (r.tiles == 1 && ((tg - 1) & 1) == 1)};
            // through shared memory (this warp's share of the P' tiles, which the last MMAs have read), so that
            // a warp writes whole lines of the output: 32 rows of 192 B, 16-byte pieces XORed by the row
            uint8_t *rows = sm.p[0][0] + warp * (32 * kD);
#pragma unroll 1
            for (int c0 = 0; c0 < kD / 2; c0 += 32) {
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (has[b]) {
                        float x[32];
                        tmem_ld32(trow + kOCol + kD * b + (kD / 2) * grp + c0, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(x[i], w[b], o[i]);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(rows + lane * kD + (((c0 / 8 + i) ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(pack_bf16x2(o[8 * i] * e2, o[8 * i + 1] * e2), pack_bf16x2(o[8 * i + 2] * e2, o[8 * i + 3] * e2),
                                   pack_bf16x2(o[8 * i + 4] * e2, o[8 * i + 5] * e2),
                                   pack_bf16x2(o[8 * i + 6] * e2, o[8 * i + 7] * e2));
            }
            __syncwarp();
            // (out is 8-byte aligned: two stores of 8 bytes where it is not 16-byte aligned)
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
#pragma unroll 2
            for (int i = 0; i < 12; ++i) {                       // 12 pieces of 16 bytes a row, 32 at a time
                const int e = lane + 32 * i, rw = e / 12, piece = e % 12;
                const uint4 x = *reinterpret_cast<const uint4 *>(rows + rw * kD + ((piece ^ ((rw >> 1) & 3)) << 4));
                const int v = 2 * wg + (rw >> 4);
                __nv_bfloat16 *dst = p.out + ((int64_t)(q0 + v) * kHQ + g * kHeadsPerGroup + (rw & 15)) * kD + (kD / 2) * grp + 8 * piece;
                if (v >= r.u0 && v < r.u1) {
                    if (wide) {
                        *reinterpret_cast<uint4 *>(dst) = x;
                    } else {
                        reinterpret_cast<uint2 *>(dst)[0] = make_uint2(x.x, x.y);
                        reinterpret_cast<uint2 *>(dst)[1] = make_uint2(x.z, x.w);
                    }
                }
            }
            __syncwarp();
            if (mine && grp == 0 && p.lse) p.lse[head] = l == 0.0f ? -INFINITY : (m - kBase + log2f(l)) * 0.69314718055994531f;
            tc_fence_before();
            fence_proxy_async();
            // every warp has looked at the run's tokens (sm.nan) before any role goes on
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.run_done);
            wait(&sm.run_done, (unsigned)n_run & 1u);
            __syncwarp();
            next(r);
        }
    }
    tc_fence_before();
    __syncthreads();                                             // every role is done (or gave up)
    tc_fence_after();
    if (warp == 8) tmem_free(tmem, kTmemCols);
}

}  // namespace attnqb
}  // namespace dsa

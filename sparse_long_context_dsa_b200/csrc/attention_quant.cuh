// Sparse and window GQA over the 8-bit paged cache (layout and scales: append_quant.cuh).
//
// A row is (query, KV group): 16 query heads over the tokens of its regions (the selection, or
// the window's regions), t <= p and inside the window.  A cluster of S CTAs (S = 1, 2, .. 16:
// more while there are few rows) shares a row, each a contiguous part of its regions, in tiles of
// 8 regions (64 tokens):
//  * a producer warp resolves the regions (sel_idx -> block_table -> block, scales; a region's
//    lookups are spread over the tiles before it) and loads each with one TMA box (K and V rows
//    lie side by side: 3 KiB) into a ring of kStages tiles; 4 warps compute:
//  * S = q K^T on mma.sync m16n8k16 fp16 (fp32 accumulate).  K's codes convert to fp16 exactly, and
//    so does 2^-e q (e per head, the largest element in [2^14, 2^15)) but for elements below
//    2^-32 of the head's largest, off by 2^-40 of it at most.  (The e4m3 mma.sync of this GPU runs
//    as two fp16 ones and their conversions: 21 cycles a k-step of 32 for q in two e4m3 terms
//    against 8 for each k-step of 16 here.)  Warp w takes regions 2w and 2w + 1 of the tile.  The K
//    scale multiplies the finished dot product.
//  * softmax in fp32, log2 units, with a running reference m per head for the sum l.  The P that
//    meets V carries the V scale, so it has a reference of its own: P' = 2^(s - m) * sV * 2^(m -
//    M), M the running maximum of s + log2 sV.  P' is rounded to fp16 (2^-12 relative, and no
//    token within 2^-24 of the largest contribution is lost); l sums the unrounded fp32 P.
//  * O += P' V with V's codes converted to fp16 (exact) on mma.sync m16n8k16, fp32 accumulate;
//    warp w owns output dims [48w, 48w + 48), so no warp merges another's O.
//    One barrier per tile: the references move (and a second one is taken) only when some token
//    passes one by more than 2^8; until then P' stays below 2^8.
//  * out = O / l * 2^(M - m), lse = ln 2 (m + log2 l); an empty row gives 0 and -inf.  With S > 1
//    the CTA's (O, m, M, l) of head h goes to CTA h mod S as one bulk copy that completes on that
//    CTA's inbox barrier, and CTA r merges heads r, r + S, ... and writes them.
// Rows of V that no token attends (behind the query, before the window, regions that are not
// there) are zeroed in shared memory: their P' is 0, but 0 * NaN is not.
#pragma once

#include <cuda_fp16.h>

#include "append_quant.cuh"
#include "common.cuh"

namespace dsa {
namespace attnq {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);                      // and the producer warp
constexpr int kStages = 2;
constexpr int kCtasPerSm = 3;
constexpr int kTileRegions = 8;                                  // 64 tokens
constexpr int kRegBytes = quant::kRegionBytesQ;                  // 3 KiB: K rows, then V rows
constexpr int kTileBytes = kTileRegions * kRegBytes;
constexpr int kQRow = 2 * kD + 16;                               // fp16 q rows (bytes), padded against bank conflicts
constexpr int kPRow = 2 * 64 + 16;                               // P' tile row (bytes), padded
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kInRow = kD + 4;                                   // inbox row: O, m, M, l, pad

// Dynamic shared memory, after the ring (which begins on a 1,024-byte boundary).
struct Smem {
    union {
        float inbox[kHeadsPerGroup * kInRow];                    // S > 1: (source CTA, its head slot)
        uint8_t q[16 * kQRow];                                   // before the cluster's first barrier
    };
    uint8_t ptile[2][16 * kPRow];
    float qscale[16];
    float mx[kWarps][16][2];
    float l[kWarps][16];
    uint64_t full[kStages], empty[kStages], inbox_bar;
    int region[kStages][kTileRegions];                           // -1: none
    float4 scale[kStages][kTileRegions];                         // K's, V's, log2 of V's
};
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kTileBytes + sizeof(Smem);

struct Params {
    const __nv_bfloat16 *q;      // [nq][64][192]
    const float2 *scale;         // [pages][4][8]: K's and V's
    const int32_t *block_table;
    const int32_t *q_req;        // nullptr: identity
    const int32_t *q_pos;
    const int32_t *sel_idx;
    const int32_t *sel_count;
    __nv_bfloat16 *out;
    float *lse;                  // may be null
    int64_t n_pages;
    int max_pages, n_req, nq, k;
    int window;                  // 0: the selection
    float scale_log2;            // log2(e) / sqrt(192)
    int splits;                  // CTAs (the cluster) per row: 1, 2, 4, 8 or 16
    int per;                     // regions of a row for each of them
};

// Byte offset of (row, col) in a region's [16 rows: 8 K, 8 V][192 B]: 64-byte lines with the
// 16-byte chunks XORed by bits 1-2 of the line index, so that 8 rows of one column fall in
// distinct 16-byte bank groups.
__device__ __forceinline__ uint32_t swz(int row, int col)
{
    const int line = row * 3 + (col >> 6);
    return (uint32_t)(line * 64 + ((((col >> 4) & 3) ^ ((line >> 1) & 3)) << 4) + (col & 15));
}

// e4m3 pairs in the low / high 16 bits of v -> fp16 pairs (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// 2^x to 2 ulp; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// D (16x8 fp32) += A (16x16 fp16, row) * B (16x8 fp16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b)
{
    const __half2 r = __hmax2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Either of two fp16 weights (>= 0, or NaN) above 2^8.
__device__ __forceinline__ bool any_above_256(uint32_t v)
{
    return __hgt2_mask(*reinterpret_cast<const __half2 *>(&v), __half2half2(__ushort_as_half(0x5C00))) != 0u;
}

// Barrier of the 4 computing warps; _or: true when `pred` holds for one of their threads.
__device__ __forceinline__ void warps_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool warps_sync_or(bool pred)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((int)pred)
        : "memory");
    return r != 0;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    sparse_attn_quant_kernel(const __grid_constant__ CUtensorMap tmap, const Params p)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    if (threadIdx.x == 0) prefetch_tensormap(&tmap);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem &sm = *reinterpret_cast<Smem *>(ring + kStages * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
    const int S = p.splits;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.full[i], 2);                           // the loads are announced; the scales are there
            mbar_init(&sm.empty[i], kWarps);
        }
        mbar_init(&sm.inbox_bar, 1);
        mbar_arrive_expect_tx(&sm.inbox_bar, (unsigned)(kHeadsPerGroup * kInRow * 4));
        fence_mbar_init();
    }
    pdl_wait();      // the previous kernel's results are visible from here on

    // rows in group-major order: the CTAs resident together gather from one group's share
    const unsigned rid_row = blockIdx.x / (unsigned)S;
    const int rank = (int)(blockIdx.x % (unsigned)S);
    const int g = (int)(rid_row / (unsigned)p.nq), qi = (int)(rid_row % (unsigned)p.nq);
    const int b = p.q_req ? p.q_req[qi] : qi;
    const int pos = p.q_pos[qi];
    const int row = qi * kG + g;
    const bool bad = pos >= 0 && (b < 0 || b >= p.n_req);
    const int t_lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    int cnt = 0;                                                 // a query before position 0 attends nothing
    if (bad) {
        if (tid == 0) set_error(kErrAttnIndex);
    } else if (pos >= 0 && p.window > 0) {
        cnt = (pos >> 3) - (t_lo >> 3) + 1;
    } else if (pos >= 0) {
        const int raw = p.sel_count[row];
        cnt = min(max(raw, 0), p.k);
        if (tid == 0 && cnt != raw) set_error(kErrAttnIndex);
    }
    // this CTA's regions: [j_lo, j_lo + n_reg) of the row's
    const int per = (cnt + S - 1) / S;
    const int j_lo = min(cnt, rank * per), n_reg = min(cnt - j_lo, per);
    const int n_tiles = (n_reg + kTileRegions - 1) / kTileRegions;
    __syncthreads();                                             // the barriers are set up

    if (warp == kWarps) {
        if (S > 1) cluster_arrive();
        // ---- producer: lane l holds region 32 n + l of the CTA (n: the batch of 4 tiles)
        auto region_of = [&](int j) -> int {
            if (j >= n_reg) return -1;
            return p.window > 0 ? (t_lo >> 3) + j_lo + j : p.sel_idx[(int64_t)row * p.k + j_lo + j];
        };
        auto page_of = [&](int j, int r) -> int {
            if (j >= n_reg) return -1;
            if (r >= 0 && r / 8 < p.max_pages) {
                const int page = p.block_table[(int64_t)b * p.max_pages + r / 8];
                if (page >= 0 && page < p.n_pages) return page;
            }
            set_error(kErrAttnIndex);
            return -1;
        };
        int r = region_of(lane), page = page_of(lane, r);
        int block = page < 0 ? -1 : (page * kG + g) * quant::kRegionsPerPage + r % 8;
        float2 sc = block < 0 ? make_float2(0.0f, 0.0f) : __ldg(p.scale + block);
        int r_n = -1, block_n = -1;                              // the next batch's
        float2 sc_n = make_float2(0.0f, 0.0f);
        bool ok = true;
        for (int ti = 0; ti < n_tiles; ++ti) {
            const int st = ti % kStages, sub = ti & 3;
            if (ti >= kStages) ok = __all_sync(0xffffffffu, mbar_wait_sleep(&sm.empty[st], (unsigned)(ti / kStages - 1) & 1u));
            if (!ok) break;
            const bool mine = (lane >> 3) == sub;
            const unsigned there = __ballot_sync(0xffffffffu, mine && block >= 0);
            if (lane == 0) {
                if (there) mbar_arrive_expect_tx(&sm.full[st], (unsigned)(__popc(there) * kRegBytes));
                else mbar_arrive(&sm.full[st]);
            }
            __syncwarp();
            if (mine) {
                if (block >= 0)
                    tma_load_3d(ring + st * kTileBytes + (lane & 7) * kRegBytes, &tmap, 0, 0, block * 16, &sm.full[st]);
                sm.region[st][lane & 7] = block < 0 ? -1 : r;
                sm.scale[st][lane & 7] = make_float4(sc.x, sc.y, log2f(sc.y), 0.0f);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[st]);
            // the next batch's lookups, one dependent load per tile of this batch
            const int jn = (ti & ~3) * kTileRegions + 32 + lane;
            if (sub == 0) {
                r_n = region_of(jn);
            } else if (sub == 1) {
                const int pg = page_of(jn, r_n);
                block_n = pg < 0 ? -1 : (pg * kG + g) * quant::kRegionsPerPage + r_n % 8;
            } else if (sub == 2) {
                sc_n = block_n < 0 ? make_float2(0.0f, 0.0f) : __ldg(p.scale + block_n);
            } else {
                r = r_n;
                block = block_n;
                sc = sc_n;
            }
        }
        __syncwarp();
        if (S > 1) cluster_wait();
        return;
    }

    // 2^-e q of head h in fp16 (warp w: heads 4w .. 4w + 3; lane: 6 elements)
    {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(
            p.q + ((int64_t)qi * kHQ + g * kHeadsPerGroup + 4 * warp) * kD) + lane;
        uint32_t w[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 3; ++j) w[i][j] = __ldg(src + i * (kD / 2) + 32 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = 4 * warp + i;
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < 3; ++j) a = fmaxf(a, fmaxf(fabsf(bf16_lo(w[i][j])), fabsf(bf16_hi(w[i][j]))));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            // block_scale puts the largest element in [224, 448]; 2^6 more, into [2^13, 2^15)
            const float s = quant::block_scale(a), inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
            if (lane == 0) sm.qscale[h] = s * (p.scale_log2 * 0.015625f);
#pragma unroll
            for (int j = 0; j < 3; ++j)
                *reinterpret_cast<uint32_t *>(sm.q + h * kQRow + 4 * (lane + 32 * j)) =
                    pack_f16x2(bf16_lo(w[i][j]) * inv * 64.0f, bf16_hi(w[i][j]) * inv * 64.0f);
        }
    }
    warps_sync();
    // A fragments of q, rows gq and gq + 8.  A k-step is a 16-byte chunk of K's codes: a thread's 4
    // codes 4t .. 4t + 3 of it are k = 2t, 2t + 1, 2t + 8, 2t + 9, for q as for K.
    uint32_t qa[12][4];
#pragma unroll
    for (int ks = 0; ks < 12; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint2 v = *reinterpret_cast<const uint2 *>(sm.q + (gq + 8 * h) * kQRow + 32 * ks + 8 * t);
            qa[ks][h] = v.x;
            qa[ks][2 + h] = v.y;
        }
    const float qf[2] = {sm.qscale[gq], sm.qscale[gq + 8]};
    if (S > 1) {
        // every CTA's inbox barrier is set up, and its q read, before any CTA copies into its inbox
        __syncwarp();
        cluster_arrive();
    }

    float o[3][2][4];                                            // 16-dim block, even / odd dims
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) o[j][s][0] = o[j][s][1] = o[j][s][2] = o[j][s][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY};      // references (rows gq, gq + 8)
    float c[2] = {0.0f, 0.0f};                                   // 2^(m - M)
    float l[2] = {0.0f, 0.0f};                                   // this thread's part of the sum
    float mref[2] = {0.0f, 0.0f};                                // m, or 0 for -inf
    bool landed = true;
    // the lane's ldmatrix offsets: K chunks 4 kb .. + 3 of row lane % 8 (region 2 warp), V chunk
    // 3 warp + j (row lane % 8 of region lane / 8), P' rows
    uint32_t koff[3], voff[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        koff[j] = smem_u32(ring) + 2 * warp * kRegBytes + swz(lane & 7, j * 64 + 16 * (lane >> 3));
        voff[j] = smem_u32(ring) + (lane >> 3) * kRegBytes + swz(8 + (lane & 7), 48 * warp + 16 * j);
    }
    const uint32_t poff = smem_u32(sm.ptile[0]) + (lane & 15) * kPRow + 16 * (lane >> 4);
    uint8_t *pw = sm.ptile[0] + gq * kPRow + 2 * (16 * warp + 2 * t);

    for (int ti = 0; ti < n_tiles; ++ti) {
        const int st = ti % kStages;
        // a wait that gives up leaves the error flag and garbage; the others are then short, and
        // every barrier is still met
        if (!mbar_wait(&sm.full[st], (unsigned)(ti / kStages) & 1u, landed ? kWaitLimitCycles : 1ll << 24)) landed = false;
        uint8_t *tile = ring + st * kTileBytes;

        // ---- S of regions 2w, 2w + 1
        float s[2][4];
        float4 sc[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const int j = 2 * warp + nt;
            const int r = sm.region[st][j];
            sc[nt] = sm.scale[st][j];
            float acc[2][4] = {};                                // even and odd chunks: two chains
#pragma unroll
            for (int kb = 0; kb < 3; ++kb) {
                uint32_t v[4];
                ldmatrix_x4(koff[kb] + st * kTileBytes + nt * kRegBytes, v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mma_f16_16816(acc[x & 1], qa[4 * kb + x], e4m3x2_to_f16x2((uint16_t)v[x]),
                                  e4m3x2_to_f16x2((uint16_t)(v[x] >> 16)));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = (acc[0][e] + acc[1][e]) * (qf[e >> 1] * sc[nt].x);
            if (r < 0 || 8 * r < t_lo || 8 * r + 7 > pos) {
                // some rows are attended by no token (the own region, the window's first, none there):
                // their scores are -inf and their V rows zero, whatever they hold
                const int u0 = r < 0 ? 8 : t_lo - 8 * r, u1 = pos - 8 * r;       // attended: u0 <= row <= u1
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int u = 2 * t + (e & 1);
                    if (u < u0 || u > u1) s[nt][e] = -INFINITY;
                }
                for (int i = lane; i < 8 * (kD / 16); i += 32) {
                    const int rr = i / (kD / 16);
                    if (rr < u0 || rr > u1)
                        *reinterpret_cast<uint4 *>(tile + j * kRegBytes + swz(8 + rr, (i % (kD / 16)) * 16)) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();                             // before the ring's next load of these bytes
            }
        }
        // ---- P' of regions 2w, 2w + 1, for the references as they are
        uint32_t pp[2][2];
        float add[2];
        auto weights = [&]() {
            add[0] = add[1] = 0.0f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = ex2(s[nt][2 * h] - mref[h]), p1 = ex2(s[nt][2 * h + 1] - mref[h]);
                    add[h] += p0 + p1;
                    const float f = fminf(sc[nt].y * c[h], 8.5070592e37f);         // 2^126
                    pp[nt][h] = pack_f16x2(p0 * f, p1 * f);
                    *reinterpret_cast<uint32_t *>(pw + (ti & 1) * (16 * kPRow) + 8 * h * kPRow + 16 * nt) = pp[nt][h];
                }
        };
        weights();
        // a reference has to move when a weight passes 2^8 (a thread's four of l: 2^10), or when
        // there is none yet; a NaN moves nothing
        const uint32_t top = max_f16x2(max_f16x2(pp[0][0], pp[0][1]), max_f16x2(pp[1][0], pp[1][1]));
        const bool grow = fmaxf(add[0], add[1]) > 1024.0f || any_above_256(top) || fminf(M[0], M[1]) == -INFINITY;
        if (warps_sync_or(grow)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float x = fmaxf(s[0][2 * h], s[0][2 * h + 1]), y = fmaxf(s[1][2 * h], s[1][2 * h + 1]);
                float mxs = fmaxf(x, y), mxv = fmaxf(x + sc[0].z, y + sc[1].z);
                mxs = fmaxf(mxs, __shfl_xor_sync(0xffffffffu, mxs, 1));
                mxs = fmaxf(mxs, __shfl_xor_sync(0xffffffffu, mxs, 2));
                mxv = fmaxf(mxv, __shfl_xor_sync(0xffffffffu, mxv, 1));
                mxv = fmaxf(mxv, __shfl_xor_sync(0xffffffffu, mxv, 2));
                if (t == 0) {
                    sm.mx[warp][gq + 8 * h][0] = mxs;
                    sm.mx[warp][gq + 8 * h][1] = mxv;
                }
            }
            warps_sync();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float a = m[h], d = M[h];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    a = fmaxf(a, sm.mx[w][gq + 8 * h][0]);
                    d = fmaxf(d, sm.mx[w][gq + 8 * h][1]);
                }
                const float al = m[h] == a ? 1.0f : exp2f(m[h] - a), ao = M[h] == d ? 1.0f : exp2f(M[h] - d);
                l[h] *= al;
#pragma unroll
                for (int j = 0; j < 3; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        o[j][x][2 * h] *= ao;
                        o[j][x][2 * h + 1] *= ao;
                    }
                m[h] = a;
                M[h] = d;
                mref[h] = a == -INFINITY ? 0.0f : a;
                c[h] = d == -INFINITY ? 0.0f : exp2f(fminf(a - d, 126.0f));
            }
            weights();
            warps_sync();
        }
        l[0] += add[0];
        l[1] += add[1];
        // ---- O[:, 48w .. 48w + 47] += P' V, two k-steps (4 regions) at a time
        const uint32_t pt = poff + (ti & 1) * (16 * kPRow);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            if (kk == 1 && n_reg - ti * kTileRegions <= 4) break;
            uint32_t pa[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                ldmatrix_x4(pt + 64 * kk + 32 * x, pa[x][0], pa[x][1], pa[x][2], pa[x][3]);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                uint32_t v[4];
                ldmatrix_x4_trans(voff[j] + st * kTileBytes + 4 * kk * kRegBytes, v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // (token 2t: dims d, d + 1)(token 2t + 1: dims d, d + 1) -> pairs of tokens per dim
                    const uint32_t a = __byte_perm(v[2 * x], 0, 0x3120), bb = __byte_perm(v[2 * x + 1], 0, 0x3120);
                    mma_f16_16816(o[j][0], pa[x], e4m3x2_to_f16x2((uint16_t)a), e4m3x2_to_f16x2((uint16_t)bb));
                    mma_f16_16816(o[j][1], pa[x], e4m3x2_to_f16x2((uint16_t)(a >> 16)),
                                  e4m3x2_to_f16x2((uint16_t)(bb >> 16)));
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);
    }

    // ---- the CTA's sums
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) sm.l[warp][gq + 8 * h] = l[h];
    }
    warps_sync();
    const int64_t head0 = (int64_t)qi * kHQ + g * kHeadsPerGroup;
    float L[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        L[h] = (sm.l[0][gq + 8 * h] + sm.l[1][gq + 8 * h]) + (sm.l[2][gq + 8 * h] + sm.l[3][gq + 8 * h]);
    if (S == 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // 0 for a row with no token or no V; a NaN sum stays NaN (no comparison holds for it)
            const float f = L[h] > 0.0f ? (M[h] > -INFINITY ? exp2f(M[h] - m[h]) / L[h] : 0.0f) : L[h];
#pragma unroll
            for (int j = 0; j < 3; ++j)
                *reinterpret_cast<uint2 *>(p.out + (head0 + gq + 8 * h) * kD + 48 * warp + 16 * j + 4 * t) =
                    make_uint2(pack_bf16x2(o[j][0][2 * h] * f, o[j][1][2 * h] * f),
                               pack_bf16x2(o[j][0][2 * h + 1] * f, o[j][1][2 * h + 1] * f));
            if (p.lse && warp == 0 && t == 0)
                p.lse[head0 + gq + 8 * h] = L[h] == 0.0f ? -INFINITY : (m[h] + log2f(L[h])) * 0.69314718055994531f;
        }
        return;
    }
    // ---- (O, m, M, l) of head h to CTA h % S, inbox row (rank, h / S); staged in the ring, whose
    // loads have all been waited for
    float *stage = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float *in = stage + (gq + 8 * h) * kInRow;
#pragma unroll
        for (int j = 0; j < 3; ++j)
            *reinterpret_cast<float4 *>(in + 48 * warp + 16 * j + 4 * t) =
                make_float4(o[j][0][2 * h], o[j][1][2 * h], o[j][0][2 * h + 1], o[j][1][2 * h + 1]);
        if (warp == 0 && t == 0) *reinterpret_cast<float4 *>(in + kD) = make_float4(m[h], M[h], L[h], 0.0f);
    }
    fence_proxy_async();                                         // the rows, to the copy engine
    __syncwarp();
    cluster_wait();
    warps_sync();
    const int per_cta = kHeadsPerGroup / S;                      // heads this CTA merges
    if (warp == 0 && lane < kHeadsPerGroup) {
        bulk_copy_to_cta(sm.inbox + (rank * per_cta + lane / S) * kInRow, stage + lane * kInRow,
                         (unsigned)(kInRow * 4), &sm.inbox_bar, (unsigned)(lane % S));
        bulk_commit();
    }
    const bool inbox_ok = mbar_wait(&sm.inbox_bar, 0u);          // false: error set
    for (int e = tid; inbox_ok && e < per_cta * (kD / 2); e += 32 * kWarps) {
        const int j = e / (kD / 2), d = 2 * (e % (kD / 2));
        float mm = -INFINITY, MM = -INFINITY;
        for (int cc = 0; cc < S; ++cc) {
            const float *in = sm.inbox + (cc * per_cta + j) * kInRow;
            mm = fmaxf(mm, in[kD]);
            MM = fmaxf(MM, in[kD + 1]);
        }
        const float mref = mm == -INFINITY ? 0.0f : mm, Mref = MM == -INFINITY ? 0.0f : MM;
        float Ls = 0.0f, x = 0.0f, y = 0.0f;
        for (int cc = 0; cc < S; ++cc) {
            const float *in = sm.inbox + (cc * per_cta + j) * kInRow;
            const float2 v = *reinterpret_cast<const float2 *>(in + d);
            const float wt = exp2f(in[kD + 1] - Mref);
            Ls += exp2f(in[kD] - mref) * in[kD + 2];
            x += wt * v.x;
            y += wt * v.y;
        }
        const float f = Ls > 0.0f ? (MM > -INFINITY ? exp2f(MM - mm) / Ls : 0.0f) : Ls;
        const int64_t head = head0 + rank + S * j;
        *reinterpret_cast<uint32_t *>(p.out + head * kD + d) = pack_bf16x2(x * f, y * f);
        if (p.lse && d == 0) p.lse[head] = Ls == 0.0f ? -INFINITY : (mm + log2f(Ls)) * 0.69314718055994531f;
    }
    // this CTA's copies have read their rows before its shared memory goes away
    if (warp == 0 && lane < kHeadsPerGroup) bulk_wait_read_all();
}

}  // namespace attnq
}  // namespace dsa

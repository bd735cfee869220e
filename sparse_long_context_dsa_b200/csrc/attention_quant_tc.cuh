// GQA of a (query, KV group) row over the 8-bit paged cache (layout and scales: append_quant.cuh):
// its selected regions, or its window's.  With q, k, v the row's 16 queries and its tokens' values,
//   s_t = q . k_t / sqrt(192),   out = sum_t e^(s_t) v_t / sum_t e^(s_t).
//
// Tiles of 16 regions (128 tokens, 48 KiB: a box {64 dims, 16 rows, 3 blocks} per region lands K's
// and V's 8 rows as the MMAs take them).  tokens (S) and dims (O) are the MMA's M, the 16 heads
// its N: a row has no more of them.
//  * S^T = K q^T: kind::f8f6f4 straight from the codes, 6 steps of K = 32.  2^-e q = hi + lo / 16 in
//    e4m3 side by side in N (off by at most 2^-14 / 224 < 2^-21 of the head's largest element, which is
//    above 224 there); the codes' scale and q's multiply the fp32 sums.
//  * softmax: thread = token, fp32, log2 units, against references m (of s) and M (of s + log2 of V's
//    scale) of each head that move only where a weight passes 2^15 (then O is rescaled in TMEM).
//  * O^T += V^T P'^T: V's codes MN-major, P' = 2^(s - m) sV 2^(m - M) as three e5m2 terms (cut off, cut
//    off, rounded) of its fp16 value, side by side in N; the terms are added at the end.
// Rows of few queries are split over a cluster, whose CTAs' (O, m, M, l) meet in distributed shared
// memory; many rows run through one CTA after another without draining the ring.
// Warps: 0-3 softmax, 4 loads (the lookups of the next 32 regions run ahead), 5 the MMAs' issuer.
//
// Bound: a row's chain load - S - softmax - P' V - the next weights, with two CTAs per SM and two tiles
// each in flight: of ~3,000 cycles a tile the weights take 900 and the P' V behind them 1,000.  k = 512,
// a call from Python (in a graph): one decode at 16,384 tokens 11.7 us (9.9; latency: 64 CTAs of two tiles;
// the bf16 kernel, twice the bytes, 8.6), 8 at 131,072 19.3 us (17.0; 2.6 TB/s), 32 of 4,096 .. 262,144
// 47.5 us (4.3 TB/s, 0.66 of the copy rate), a chunk of 256 queries at 32,768 212 us (184; 1.6 GB of gathers
// from L2, 7.7 TB/s; tensor pipe 18 %, issue slots 39 %).  Tried and not faster (the chunk, us against 229 with the
// issuer as lane 0 in place of an elected lane): regions as boxes of 128 and 64 dims, two rows of a token
// in place of three 243; K's and V's places released apart 236; eight softmax warps of 8 heads 238.
#pragma once

#include <type_traits>

#include "attention_quant.cuh"

namespace dsa {
namespace attnqt {

using attnq::ex2;
using attnq::kRegBytes;
using attnq::Params;

constexpr int kTileRegions = 16;                                 // 128 tokens: the MMA's M
constexpr int kTileBytes = kTileRegions * kRegBytes;             // 48 KiB
constexpr int kStages = 2;
constexpr int kInRow = kD + 4;                                   // inbox row: O, m, M, l, pad
constexpr int kThreads = 192;                                    // warps 0-3 softmax, 4 loads, 5 MMA
constexpr int kCtasPerSm = 2;
constexpr int kN = 32;                                           // S: 16 heads x (hi, lo) of q
constexpr int kNp = 48;                                          // O: 16 heads x three terms of P'
constexpr int kOCol = 64;                                        // TMEM: S 0, 32 (two buffers); O 64 (dims 0-127), 112 (64-191)
constexpr int kTmemCols = 256;
constexpr float kBase = 5.0f;                                    // log2 of a weight at its reference
constexpr float kTop = 32768.0f;                                 // 2^15: the largest P' before the references move

struct Smem {
    uint8_t p[3][128 * 16];                                      // P': [term][token][16 heads], e5m2
    uint8_t q[3 * kN * 64];                                      // q: [64-dim block][hi of 16 heads, lo][64], 64-byte swizzle
    float4 scale[kStages][kTileRegions];                         // K's, V's, log2 of V's
    int region[kStages][kTileRegions];                           // -1: none
    float qscale[16], mref[16], c[16], al[16], ao[16], m[16], M[16], f[16];
    float red[4][32];
    uint64_t full[kStages], empty[kStages], s_full[2], p_ready, pv_done, q_ready, inbox_bar;
    uint32_t tmem;
    int state;                                                   // 1: some head has no V yet; 2: O is rescaled
};
constexpr size_t kSmemBytes = 1024 + (size_t)kStages * kTileBytes + sizeof(Smem);
constexpr int kInboxOffset = 16 * 1024;                          // in the ring, behind the staged rows
static_assert(16 * kInRow * 4 <= kInboxOffset && kInboxOffset + 16 * kInRow * 4 <= kTileBytes, "staging and inbox");
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");

// Shared-memory matrix descriptors in halves: lo = start address and LBO, hi = SBO, version (sm_100)
// and swizzle (4: 64 bytes, 0: none).  A later tile's lo is lo + byte offset / 16.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) { return (sbo >> 4) | (1u << 14) | (swizzle << 29); }

// D[tmem] (+)= A[smem] B[smem]^T, kind::f8f6f4, the accumulate flag an immediate.
template <bool kAccumulate>
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .b64 a, b;\n\t.reg .pred p;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.eq.u32 p, %6, 1;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}"
        ::"r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"((int)kAccumulate)
        : "memory");
}
constexpr uint32_t kIdescS = umma_idesc_e4m3(128, kN);
// V^T (A, e4m3) and P'^T (B, e5m2) MN-major
constexpr uint32_t kIdescO = umma_idesc_e4m3(128, kNp) | (1u << 10) | (1u << 15) | (1u << 16);

// Whether the phase of `bar` with the given parity is complete; never suspends.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, unsigned parity)
{
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b)
{
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Either of two fp16 weights (>= 0, or NaN) above 2^15.
__device__ __forceinline__ bool any_above_top(uint32_t v)
{
    return __hgt2_mask(*reinterpret_cast<const __half2 *>(&v), __half2half2(__ushort_as_half(0x7800))) != 0u;
}

// 16 consecutive fp32 columns of this warp's 32 TMEM lanes (one row per lane).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
          "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Lane l of the warp gets the maximum over the lanes of v[l], 31 shuffles.
__device__ __forceinline__ float reduce_scatter_max32(float (&v)[32])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
            v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, w));
        }
    }
    return v[0];
}

// Lane l gets the sum over the lanes of v[l / 2], 16 shuffles.
__device__ __forceinline__ float reduce_scatter_add16(float (&v)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 8; w > 0; w >>= 1) {
        const bool up = (lane & (2 * w)) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * w);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// A row (query, group) as the CTA `rank` of its cluster sees it.
struct Row {
    int g, qi, b, pos, t_lo, row;
    int j_lo, n_reg, n_tiles;                                    // its regions of the row's, in tiles
};

// Rows in group-major order: the CTAs at work together gather from one group's share.
__device__ __forceinline__ Row row_of(const Params &p, unsigned r, int rank, bool report)
{
    Row x;
    x.g = (int)(r / (unsigned)p.nq);
    x.qi = (int)(r % (unsigned)p.nq);
    x.row = x.qi * kG + x.g;
    x.pos = p.q_pos[x.qi];
    x.b = p.q_req ? p.q_req[x.qi] : x.qi;
    const int raw = p.window > 0 ? 0 : p.sel_count[x.row];
    x.t_lo = p.window > 0 ? max(0, x.pos - p.window + 1) : 0;
    int cnt = 0;                                                 // a query before position 0 attends nothing
    if (x.pos >= 0) {
        if (x.b < 0 || x.b >= p.n_req) {
            if (report) set_error(kErrAttnIndex);
        } else if (p.window > 0) {
            cnt = (x.pos >> 3) - (x.t_lo >> 3) + 1;
        } else {
            cnt = min(max(raw, 0), p.k);
            if (report && cnt != raw) set_error(kErrAttnIndex);
        }
    }
    x.j_lo = rank * p.per;
    x.n_reg = max(0, min(cnt - x.j_lo, p.per));
    x.n_tiles = (x.n_reg + kTileRegions - 1) / kTileRegions;
    return x;
}

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    sparse_attn_quant_tc_kernel(const __grid_constant__ CUtensorMap tmap, const Params p)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    if (threadIdx.x == 0) prefetch_tensormap(&tmap);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Smem &sm = *reinterpret_cast<Smem *>(ring + kStages * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.splits;
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.full[i], 2);                           // the loads are announced; the scales are there
            mbar_init(&sm.empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
        }
        mbar_init(&sm.p_ready, 1);
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.q_ready, 4);
        mbar_init(&sm.inbox_bar, 1);
        mbar_arrive_expect_tx(&sm.inbox_bar, (unsigned)(kHeadsPerGroup * kInRow * 4));
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc(&sm.tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();                                             // the barriers are set up, TMEM is there
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    pdl_wait();      // the previous kernel's results are visible from here on

    // This CTA's rows: with S = 1 every gridDim.x-th one (the ring, the barriers' phases and the
    // tiles' count `base` run through them all), else the cluster's one.
    const unsigned rows = p.row_end;
    const unsigned first = p.row0 + blockIdx.x / (unsigned)S, step = gridDim.x / (unsigned)S;
    const int rank = (int)(blockIdx.x % (unsigned)S);

    if (warp == 4) {
        // ---- loads: lane l holds region 32 n + l of the row (n: the batch of 2 tiles)
        int tg = 0;                                              // tiles before this one, over all rows
        bool ok = true;
        for (unsigned rr = first; rr < rows && ok; rr += step) {
            // (the selection is read beside its count: entries within k lie in the row)
            auto raw_region = [&](int row, int j_lo, int j) -> int {
                return p.window > 0 || j_lo + j >= p.k || j >= p.per ? -1 : p.sel_idx[(int64_t)row * p.k + j_lo + j];
            };
            const int row = (int)(rr % (unsigned)p.nq) * kG + (int)(rr / (unsigned)p.nq);
            int r = raw_region(row, rank * p.per, lane), r_n = raw_region(row, rank * p.per, 32 + lane);
            const Row x = row_of(p, rr, rank, lane == 0 && rank == 0);
            // the page of region j, and (once it is there) its block
            auto page_of = [&](int j, int &reg) -> int {
                if (j >= x.n_reg) return -1;
                if (p.window > 0) reg = (x.t_lo >> 3) + x.j_lo + j;
                return reg >= 0 && reg / 8 < p.max_pages ? p.block_table[(int64_t)x.b * p.max_pages + reg / 8] : -1;
            };
            auto block_of = [&](int j, int reg, int page) -> int {
                if (j >= x.n_reg) return -1;
                if (page >= 0 && page < p.n_pages) return (page * kG + x.g) * quant::kRegionsPerPage + reg % 8;
                set_error(kErrAttnIndex);
                return -1;
            };
            int page_n = page_of(lane, r);
            int block = block_of(lane, r, page_n);
            float2 sc = block < 0 ? make_float2(0.0f, 0.0f) : __ldg(p.scale + block);
            for (int ti = 0; ti < x.n_tiles; ++ti, ++tg) {
                const int st = tg % kStages, sub = ti & 1;
                if (tg >= kStages) ok = __all_sync(0xffffffffu, mbar_wait_sleep(&sm.empty[st], (unsigned)(tg / kStages - 1) & 1u));
                if (!ok) break;
                const bool mine = (lane >> 4) == sub;
                const unsigned there = __ballot_sync(0xffffffffu, mine && block >= 0);
                if (lane == 0) {
                    if (there) mbar_arrive_expect_tx(&sm.full[st], (unsigned)(__popc(there) * kRegBytes));
                    else mbar_arrive(&sm.full[st]);
                }
                __syncwarp();
                if (mine) {
                    if (block >= 0)
                        tma_load_3d(ring + st * kTileBytes + (lane & 15) * kRegBytes, &tmap, 0, block * 16, 0, &sm.full[st]);
                    sm.region[st][lane & 15] = block < 0 ? -1 : r;
                    sm.scale[st][lane & 15] = make_float4(sc.x, sc.y, log2f(sc.y), 0.0f);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.full[st]);
                // the next batch's lookups: no load is waited for in the tile that issues it
                const int jn = (ti & ~1) * kTileRegions + 32 + lane;
                if (sub == 0) {
                    page_n = page_of(jn, r_n);
                } else {
                    r = r_n;
                    block = block_of(jn, r, page_n);
                    sc = block < 0 ? make_float2(0.0f, 0.0f) : __ldg(p.scale + block);
                    r_n = raw_region(row, x.j_lo, jn + 32);
                }
            }
        }
        // none of this warp's loads is in flight when the CTA ends, after a wait that gave up as well
        __syncwarp();
        if (lane == 0)
            for (int s = 0; s < kStages && s < tg; ++s) {
                const int last = tg - 1 - (tg - 1 - s) % kStages;
                mbar_wait(&sm.full[s], (unsigned)(last / kStages) & 1u);
            }
        __syncwarp();
    } else if (warp == 5) {
        // ---- MMA issuer (one elected lane): S(i) as its codes land, O += P'(j) V(j) as the weights are
        // there, whichever is ready; at most two S are ahead of the weights
        if (elect_one()) {
            // K: rows of 64 bytes, a region's 8 rows 512 bytes, regions 3 KiB apart; V^T: 64-dim blocks
            // 1 KiB apart, 8-token groups 3 KiB apart; P'^T: 8 tokens x 16 heads 128 bytes, terms 2 KiB apart
            const uint32_t k_lo = desc_lo(smem_u32(ring), 16), v_lo = desc_lo(smem_u32(ring) + 512, 1024);
            const uint32_t q_lo = desc_lo(smem_u32(sm.q), 16), p_lo = desc_lo(smem_u32(sm.p), 128);
            constexpr uint32_t kKvHi = desc_hi(kRegBytes, 4), kQHi = desc_hi(512, 4), kPHi = desc_hi(2048, 0);
            // the rows of the next S (r_s: i_s of n_s tiles issued) and of the next P' V (r_p)
            unsigned r_s = first, r_p = first, rows_s = 0;
            int i_s = 0, i_p = 0, i = 0, j = 0;
            int n_s = r_s < rows ? row_of(p, r_s, rank, false).n_tiles : 0;
            int reg_p = r_p < rows ? row_of(p, r_p, rank, false).n_reg : 0;
            bool ok = true;
            long long since = clock64();
            while (ok) {
                // (q_ready's phases count the rows with tiles: after one of them the softmax waits for its
                // S before it puts the next q, so a parity is never one phase off)
                while (r_s < rows && i_s == n_s) {
                    r_s += step;
                    if (n_s > 0) ++rows_s;
                    i_s = 0;
                    n_s = r_s < rows ? row_of(p, r_s, rank, false).n_tiles : 0;
                }
                while (r_p < rows && i_p * kTileRegions >= reg_p) {
                    r_p += step;
                    i_p = 0;
                    reg_p = r_p < rows ? row_of(p, r_p, rank, false).n_reg : 0;
                }
                if (r_p >= rows) break;
                if (j < i && mbar_test(&sm.p_ready, (unsigned)j & 1u)) {
                    tc_fence_after();
                    const uint32_t a = v_lo + (uint32_t)(j % kStages) * (kTileBytes >> 4);
                    const int steps = min(4, (reg_p - i_p * kTileRegions + 3) / 4);        // 32 tokens each
                    auto mma = [&](auto acc, int kk) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mma_f8<decltype(acc)::value>(tmem + kOCol + kNp * h, a + kk * (4 * kRegBytes >> 4) + h * (1024 >> 4),
                                                         kKvHi, p_lo + kk * (512 >> 4), kPHi, kIdescO);
                    };
                    if (i_p > 0) mma(std::true_type{}, 0);
                    else mma(std::false_type{}, 0);
#pragma unroll 1
                    for (int kk = 1; kk < steps; ++kk) mma(std::true_type{}, kk);
                    umma_commit(&sm.empty[j % kStages]);
                    umma_commit(&sm.pv_done);
                    ++j;
                    ++i_p;
                    since = clock64();
                } else if (r_s < rows && i < j + 2 && mbar_test(&sm.full[i % kStages], (unsigned)(i / kStages) & 1u) &&
                           (i_s > 0 || mbar_test(&sm.q_ready, rows_s & 1u))) {
                    tc_fence_after();
                    const uint32_t a = k_lo + (uint32_t)(i % kStages) * (kTileBytes >> 4), d = tmem + 32 * (i & 1);
                    mma_f8<false>(d, a, kKvHi, q_lo, kQHi, kIdescS);
#pragma unroll
                    for (int ks = 1; ks < 6; ++ks)
                        mma_f8<true>(d, a + (((ks >> 1) * 1024 + (ks & 1) * 32) >> 4), kKvHi,
                                     q_lo + (((ks >> 1) * (kN * 64) + (ks & 1) * 32) >> 4), kQHi, kIdescS);
                    umma_commit(&sm.s_full[i & 1]);
                    ++i;
                    ++i_s;
                    since = clock64();
                } else if (clock64() - since > kWaitLimitCycles) {
                    set_error(kErrWaitTimeout);
                    ok = false;
                }
            }
            // every commit has arrived when TMEM is released, after a wait that gave up as well (umma_commit)
            commits_done(&sm.pv_done, j);
            for (int s = 0; s < 2; ++s) commits_done(&sm.s_full[s], (i + 1 - s) / 2);
            for (int s = 0; s < kStages; ++s) commits_done(&sm.empty[s], (j + kStages - 1 - s) / kStages);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = token (TMEM lane) 32 warp + lane of the tile
        const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16);
        bool landed = true;
        // a wait that gives up leaves the error flag and garbage; the later ones are then short, and
        // every barrier is still met
        auto wait = [&](uint64_t *bar, unsigned parity) {
            if (!mbar_wait(bar, parity, landed ? kWaitLimitCycles : 1ll << 22)) landed = false;
        };
        // 2^-e q = hi + lo / 16 in e4m3, for row r: threads 8 h .. 8 h + 7 share head h, thread c
        // of them holds dims 8 c .. 8 c + 7 of every 64-dim block
        uint4 qv[3];
        auto load_q = [&](unsigned r) {
            const int g = (int)(r / (unsigned)p.nq), qi = (int)(r % (unsigned)p.nq);
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.q + ((int64_t)qi * kHQ + g * kHeadsPerGroup + (tid >> 3)) * kD + 8 * (tid & 7));
#pragma unroll
            for (int j = 0; j < 3; ++j) qv[j] = __ldg(src + 8 * j);
        };
        auto put_q = [&](bool tiles) {                           // (no S waits for the q of a row without tiles)
            const int h = tid >> 3, c = tid & 7;
            __nv_bfloat162 a2 = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const uint32_t w[4] = {qv[j].x, qv[j].y, qv[j].z, qv[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) a2 = __hmax2(a2, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
            }
            float a = fmaxf(__low2float(a2), __high2float(a2));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
            const float s = quant::block_scale(a), inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
            if (c == 0) sm.qscale[h] = s * p.scale_log2;
            uint8_t *dst = sm.q + h * 64 + ((((c >> 1) ^ ((h >> 1) & 3)) << 4) | ((c & 1) << 3));
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
                    lo[i] = cvt_e4m3x2((x - f.x) * 16.0f, (y - f.y) * 16.0f);
                }
                *reinterpret_cast<uint2 *>(dst + j * (kN * 64)) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                *reinterpret_cast<uint2 *>(dst + j * (kN * 64) + 16 * 64) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && tiles) mbar_arrive(&sm.q_ready);
        };
        int tg = 0;                                              // tiles before this one, over all rows
        Row x{}, x_next{};
        if (first < rows) {
            load_q(first);
            x_next = row_of(p, first, rank, false);
            put_q(x_next.n_tiles > 0);
        }
        for (unsigned rr = first; rr < rows; rr += step) {
            x = x_next;
            if (tid < 16) {
                sm.m[tid] = sm.M[tid] = -INFINITY;
                sm.mref[tid] = sm.c[tid] = 0.0f;
            }
            attnq::warps_sync();                                 // the references, qscale
            float2 l[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) l[h] = make_float2(0.0f, 0.0f);
            bool unset = true;
            if (rr + step < rows) {                              // for the row after this one
                load_q(rr + step);
                x_next = row_of(p, rr + step, rank, false);
            }
            for (int ti = 0; ti < x.n_tiles; ++ti, ++tg) {
                const int st = tg % kStages;
                wait(&sm.full[st], (unsigned)(tg / kStages) & 1u);                         // the scales
                const int j = 4 * warp + (lane >> 3);
                const float4 sc = sm.scale[st][j];
                const int r = sm.region[st][j], tok = 8 * r + (lane & 7);
                const bool ok = r >= 0 && tok <= x.pos && tok >= x.t_lo;
                const bool all_ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    // a V row that no token attends: zero, whatever it holds
                    uint8_t *v = ring + st * kTileBytes + j * kRegBytes + 512 + (lane & 7) * 64;
#pragma unroll 1
                    for (int i = 0; i < 12; ++i)
                        *reinterpret_cast<uint4 *>(v + (i >> 2) * 1024 + (i & 3) * 16) = make_uint4(0, 0, 0, 0);
                }
                wait(&sm.s_full[tg & 1], (unsigned)(tg >> 1) & 1u);
                __syncwarp();
                tc_fence_after();
                float xs[32];
                tmem_ld32(trow + 32 * (tg & 1), xs);
                float2 s[8], pr[8];                              // scores, weights
                const float2 ks2 = make_float2(sc.x, sc.x), vs2 = make_float2(sc.y, sc.y), one2 = make_float2(1.0f, 1.0f);
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float2 q2 = *reinterpret_cast<const float2 *>(&sm.qscale[2 * h]);
                    const float2 y = ffma2(make_float2(xs[16 + 2 * h], xs[17 + 2 * h]), make_float2(0.0625f, 0.0625f),
                                           make_float2(xs[2 * h], xs[2 * h + 1]));
                    s[h] = fmul2(y, fmul2(ks2, q2));             // (the scales first: y times one of them may overflow)
                }
                if (!all_ok) {
#pragma unroll
                    for (int h = 0; h < 8; ++h)
                        if (!ok) s[h] = make_float2(-INFINITY, -INFINITY);
                }
                // P' of the tile before has been read
                if (tg > 0) wait(&sm.pv_done, (unsigned)(tg - 1) & 1u);
                __syncwarp();
#pragma unroll 1
                for (int pass = unset ? 1 : 0;; pass = 2) {
                    bool grow = pass == 1;
                    if (pass != 1) {
                        // the weights for the references as they are (pass 2: as they have moved)
                        uint32_t w[8], top = 0u;
                        float2 add = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int h = 0; h < 8; ++h) {
                            const float2 mr = *reinterpret_cast<const float2 *>(&sm.mref[2 * h]);
                            const float2 cc = *reinterpret_cast<const float2 *>(&sm.c[2 * h]);
                            const float2 e = ffma2(s[h], one2, make_float2(-mr.x, -mr.y));
                            pr[h] = make_float2(ex2(e.x), ex2(e.y));
                            add = ffma2(pr[h], one2, add);
                            float2 f = fmul2(vs2, cc);
                            f = make_float2(fminf(f.x, 8.5070592e37f), fminf(f.y, 8.5070592e37f));         // 2^126
                            const float2 x2 = fmul2(pr[h], f);
                            w[h] = attnq::pack_f16x2(x2.x, x2.y);
                            top = attnq::max_f16x2(top, w[h]);
                        }
                        grow = pass == 0 && (add.x + add.y > kTop || any_above_top(top));
                        // three e5m2 terms: the upper bytes of w, of what they leave, and of the rest, rounded
                        uint8_t *dst = sm.p[0] + (32 * warp + lane) * 16;
#pragma unroll
                        for (int term = 0; term < 3; ++term) {
                            if (term == 2) {
#pragma unroll
                                for (int h = 0; h < 8; ++h) w[h] += 0x00800080u;
                            }
                            *reinterpret_cast<uint4 *>(dst + term * 2048) =
                                make_uint4(__byte_perm(w[0], w[1], 0x7531), __byte_perm(w[2], w[3], 0x7531),
                                           __byte_perm(w[4], w[5], 0x7531), __byte_perm(w[6], w[7], 0x7531));
                            if (term < 2) {
#pragma unroll
                                for (int h = 0; h < 8; ++h) w[h] = hsub2(w[h], w[h] & 0xFF00FF00u);
                            }
                        }
                        fence_proxy_async();
                        tc_fence_before();
                    }
                    if (!attnq::warps_sync_or(grow)) break;
                    // ---- the references move: the tile's maxima of s and s + log2 sV of every head
                    float v[32];
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        v[2 * h] = s[h].x;
                        v[2 * h + 1] = s[h].y;
                        v[16 + 2 * h] = s[h].x + sc.z;
                        v[17 + 2 * h] = s[h].y + sc.z;
                    }
                    sm.red[warp][lane] = reduce_scatter_max32(v);
                    attnq::warps_sync();
                    if (warp == 0) {
                        float *ref = lane < 16 ? &sm.m[lane] : &sm.M[lane - 16];
                        const float old = *ref;
                        const float a = fmaxf(fmaxf(fmaxf(sm.red[0][lane], sm.red[1][lane]), fmaxf(sm.red[2][lane], sm.red[3][lane])), old);
                        const float scale = old == a ? 1.0f : exp2f(old - a);
                        const float d = __shfl_xor_sync(0xffffffffu, a, 16);
                        *ref = a;
                        const unsigned none = __ballot_sync(0xffffffffu, lane >= 16 && a == -INFINITY);
                        const unsigned moved = __ballot_sync(0xffffffffu, lane >= 16 && scale != 1.0f);
                        if (lane < 16) {
                            sm.mref[lane] = a == -INFINITY ? 0.0f : a - kBase;
                            sm.c[lane] = d == -INFINITY ? 0.0f : exp2f(fminf(a - d, 126.0f));
                            sm.al[lane] = scale;
                        } else {
                            sm.ao[lane - 16] = scale;
                        }
                        if (lane == 0) sm.state = (none ? 1 : 0) | (moved ? 2 : 0);
                    }
                    attnq::warps_sync();
                    unset = (sm.state & 1) != 0;
                    if (ti > 0) {
#pragma unroll
                        for (int h = 0; h < 8; ++h) l[h] = fmul2(l[h], *reinterpret_cast<const float2 *>(&sm.al[2 * h]));
                        if (sm.state & 2) {
                            // O holds the tiles before this one (their MMAs are done)
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < 2 * kNp; c0 += 16) {
                                float o[16];
                                tmem_ld16(trow + kOCol + c0, o);
#pragma unroll
                                for (int h = 0; h < 16; ++h) o[h] *= sm.ao[h];
                                tmem_st16(trow + kOCol + c0, o);
                            }
                            tc_fence_before();
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 8; ++h) l[h] = ffma2(pr[h], one2, l[h]);
                if (tid == 0) mbar_arrive(&sm.p_ready);
            }
            // every S of this row is done with its q: the next row's
            if (rr + step < rows) put_q(x_next.n_tiles > 0);
            // ---- the CTA's sums and factors
            {
                float v[16];
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    v[2 * h] = l[h].x;
                    v[2 * h + 1] = l[h].y;
                }
                const float sum = reduce_scatter_add16(v);
                if ((lane & 1) == 0) sm.red[warp][lane >> 1] = sum;
            }
            attnq::warps_sync();
            const int64_t head0 = (int64_t)x.qi * kHQ + x.g * kHeadsPerGroup;
            if (warp == 0 && lane < 16) {
                const float L = (sm.red[0][lane] + sm.red[1][lane]) + (sm.red[2][lane] + sm.red[3][lane]);
                const float m = sm.m[lane], M = sm.M[lane];
                // O times 1 / L, then 2^(M - m) (their product may be below fp32's range); 0 for a row with no
                // token or no V; a NaN sum stays NaN (no comparison holds for it)
                sm.f[lane] = S > 1 ? L : L > 0.0f ? 1.0f / L : L;
                sm.ao[lane] = M > -INFINITY ? exp2f(M - m) : 0.0f;
                if (S == 1 && p.lse) p.lse[head0 + lane] = L == 0.0f ? -INFINITY : (m - kBase + log2f(L)) * 0.69314718055994531f;
            }
            if (x.n_tiles > 0) wait(&sm.pv_done, (unsigned)(tg - 1) & 1u);
            attnq::warps_sync();                                 // the factors; every warp is past the ring (S > 1)
            tc_fence_after();
            float *stage = reinterpret_cast<float *>(ring);
#pragma unroll 1
            for (int h2 = 0; h2 < 2; ++h2) {
                if (h2 == 1 && warp < 2) break;                  // dims 64-127 again
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0.0f;
                __syncwarp();
                if (x.n_tiles > 0) {
#pragma unroll 1
                    for (int c0 = 0; c0 < kNp; c0 += 16) {
                        float o1[16];
                        tmem_ld16(trow + kOCol + kNp * h2 + c0, o1);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] += o1[i];
                    }
                }
                const int d = 64 * h2 + 32 * warp + lane;
                if (S == 1) {
#pragma unroll
                    for (int h = 0; h < 16; ++h) p.out[(head0 + h) * kD + d] = __float2bfloat16_rn(o[h] * sm.f[h] * sm.ao[h]);
                } else {
#pragma unroll
                    for (int h = 0; h < 16; ++h) stage[h * kInRow + d] = o[h];
                }
            }
            if (S > 1) {
                if (warp == 0 && lane < 16)
                    *reinterpret_cast<float4 *>(stage + lane * kInRow + kD) = make_float4(sm.m[lane], sm.M[lane], sm.f[lane], 0.0f);
                fence_proxy_async();                             // the rows, to the copy engine
            }
            tc_fence_before();
            attnq::warps_sync();                                 // before the references are set again
        }
    }
    tc_fence_before();
    __syncthreads();                                             // every role is done (or gave up)
    tc_fence_after();
    if (warp == 5) tmem_free(tmem, kTmemCols);
    if (S == 1) return;
    // ---- (O, m, M, l) of head h to CTA h % S, inbox row (rank, h / S), both in the ring, which every
    // CTA of the cluster has finished with
    float *stage = reinterpret_cast<float *>(ring);
    float *inbox = reinterpret_cast<float *>(ring + kInboxOffset);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    const int per_cta = kHeadsPerGroup / S;                      // heads this CTA merges
    if (warp == 0 && lane < kHeadsPerGroup) {
        bulk_copy_to_cta(inbox + (rank * per_cta + lane / S) * kInRow, stage + lane * kInRow, (unsigned)(kInRow * 4),
                         &sm.inbox_bar, (unsigned)(lane % S));
        bulk_commit();
    }
    const bool inbox_ok = mbar_wait(&sm.inbox_bar, 0u);          // false: error set
    const int64_t head0 = (int64_t)(first % (unsigned)p.nq) * kHQ + (int)(first / (unsigned)p.nq) * kHeadsPerGroup;
    for (int e = tid; inbox_ok && e < per_cta * (kD / 2); e += kThreads) {
        const int j = e / (kD / 2), d = 2 * (e % (kD / 2));
        float mm = -INFINITY, MM = -INFINITY;
#pragma unroll 4
        for (int cc = 0; cc < S; ++cc) {
            const float *in = inbox + (cc * per_cta + j) * kInRow;
            mm = fmaxf(mm, in[kD]);
            MM = fmaxf(MM, in[kD + 1]);
        }
        const float mref = mm == -INFINITY ? 0.0f : mm, Mref = MM == -INFINITY ? 0.0f : MM;
        float Ls = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll 4
        for (int cc = 0; cc < S; ++cc) {
            const float *in = inbox + (cc * per_cta + j) * kInRow;
            const float2 v = *reinterpret_cast<const float2 *>(in + d);
            const float wt = ex2(in[kD + 1] - Mref);
            Ls += ex2(in[kD] - mref) * in[kD + 2];
            x += wt * v.x;
            y += wt * v.y;
        }
        const float f = Ls > 0.0f ? 1.0f / Ls : Ls, e2 = MM > -INFINITY ? exp2f(MM - mm) : 0.0f;
        const int64_t head = head0 + rank + S * j;
        *reinterpret_cast<uint32_t *>(p.out + head * kD + d) = pack_bf16x2(x * f * e2, y * f * e2);
        if (p.lse && d == 0) p.lse[head] = Ls == 0.0f ? -INFINITY : (mm - kBase + log2f(Ls)) * 0.69314718055994531f;
    }
    // this CTA's copies have read their rows before its shared memory goes away
    if (warp == 0 && lane < kHeadsPerGroup) bulk_wait_read_all();
}

}  // namespace attnqt
}  // namespace dsa

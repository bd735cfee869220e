// (header comment written once the kernel is settled)
#pragma once

#include <type_traits>

#include "attention_quant.cuh"

namespace dsa {
namespace attnqt {

using attnq::ex2;
using attnq::kInRow;
using attnq::kRegBytes;
using attnq::Params;

constexpr int kTileRegions = 16;                                 // 128 tokens: the MMA's M
constexpr int kTileBytes = kTileRegions * kRegBytes;             // 48 KiB
constexpr int kStages = 2;
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
    uint64_t full[kStages], empty[kStages], s_full[2], p_ready, pv_done, q_ready, drain, inbox_bar;
    uint32_t tmem;
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

// Lane l of the warp gets f(over the lanes) of v[l] (f: max), 31 shuffles.
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
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.inbox_bar, 1);
        mbar_arrive_expect_tx(&sm.inbox_bar, (unsigned)(kHeadsPerGroup * kInRow * 4));
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc(&sm.tmem, kTmemCols);
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
    tc_fence_before();
    __syncthreads();                                             // the barriers are set up, TMEM is there
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int64_t head0 = (int64_t)qi * kHQ + g * kHeadsPerGroup;

    if (warp == 4) {
        // ---- loads: lane l holds region 32 n + l of the CTA (n: the batch of 2 tiles)
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
        auto block_of = [&](int page, int r) { return page < 0 ? -1 : (page * kG + g) * quant::kRegionsPerPage + r % 8; };
        int r = region_of(lane), block = block_of(page_of(lane, r), r);
        float2 sc = block < 0 ? make_float2(0.0f, 0.0f) : __ldg(p.scale + block);
        int r_n = region_of(32 + lane), block_n = -1;            // the next batch's
        float2 sc_n = make_float2(0.0f, 0.0f);
        int issued = 0;
        for (int ti = 0; ti < n_tiles; ++ti) {
            const int st = ti % kStages, sub = ti & 1;
            if (ti >= kStages &&
                !__all_sync(0xffffffffu, mbar_wait_sleep(&sm.empty[st], (unsigned)(ti / kStages - 1) & 1u)))
                break;
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
            issued = ti + 1;
            // the next batch's lookups, one dependent load per tile of this batch
            if (sub == 0) {
                block_n = block_of(page_of((ti & ~1) * kTileRegions + 32 + lane, r_n), r_n);
            } else {
                r = r_n;
                block = block_n;
                sc_n = block < 0 ? make_float2(0.0f, 0.0f) : __ldg(p.scale + block);
                sc = sc_n;
                r_n = region_of((ti & ~1) * kTileRegions + 64 + lane);
            }
        }
        // none of this warp's loads is in flight when the CTA ends, after a wait that gave up as well
        __syncwarp();
        if (lane == 0)
            for (int s = 0; s < kStages && s < issued; ++s) {
                const int last = issued - 1 - (issued - 1 - s) % kStages;
                mbar_wait(&sm.full[s], (unsigned)(last / kStages) & 1u);
            }
        __syncwarp();
    } else if (warp == 5) {
        // ---- MMA issuer (one lane): S(i) as its codes land, O += P'(j) V(j) as the weights are
        // there, whichever is ready; at most two S are ahead of the weights
        if (lane == 0) {
            bool ok = mbar_wait(&sm.q_ready, 0u);
            // K: rows of 64 bytes, a region's 8 rows 512 bytes, regions 3 KiB apart; V^T: 64-dim blocks
            // 1 KiB apart, 8-token groups 3 KiB apart; P'^T: 8 tokens x 16 heads 128 bytes, terms 2 KiB apart
            const uint32_t k_lo = desc_lo(smem_u32(ring), 16), v_lo = desc_lo(smem_u32(ring) + 512, 1024);
            const uint32_t q_lo = desc_lo(smem_u32(sm.q), 16), p_lo = desc_lo(smem_u32(sm.p), 128);
            constexpr uint32_t kKvHi = desc_hi(kRegBytes, 4), kQHi = desc_hi(512, 4), kPHi = desc_hi(2048, 0);
            int i = 0, j = 0;
            long long since = clock64();
            while (j < n_tiles && ok) {
                if (j < i && mbar_test(&sm.p_ready, (unsigned)j & 1u)) {
                    tc_fence_after();
                    const uint32_t a = v_lo + (uint32_t)(j % kStages) * (kTileBytes >> 4);
                    const int steps = min(4, (n_reg - j * kTileRegions + 3) / 4);          // 32 tokens each
                    auto step = [&](auto acc, int kk) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            mma_f8<decltype(acc)::value>(tmem + kOCol + kNp * h, a + kk * (4 * kRegBytes >> 4) + h * (1024 >> 4),
                                                         kKvHi, p_lo + kk * (512 >> 4), kPHi, kIdescO);
                    };
                    if (j > 0) step(std::true_type{}, 0);
                    else step(std::false_type{}, 0);
                    if (steps > 1) step(std::true_type{}, 1);
                    if (steps > 2) step(std::true_type{}, 2);
                    if (steps > 3) step(std::true_type{}, 3);
                    umma_commit(&sm.empty[j % kStages]);
                    umma_commit(&sm.pv_done);
                    ++j;
                    since = clock64();
                } else if (i < n_tiles && i < j + 2 && mbar_test(&sm.full[i % kStages], (unsigned)(i / kStages) & 1u)) {
                    tc_fence_after();
                    const uint32_t a = k_lo + (uint32_t)(i % kStages) * (kTileBytes >> 4), d = tmem + 32 * (i & 1);
                    mma_f8<false>(d, a, kKvHi, q_lo, kQHi, kIdescS);
#pragma unroll
                    for (int ks = 1; ks < 6; ++ks)
                        mma_f8<true>(d, a + (((ks >> 1) * 1024 + (ks & 1) * 32) >> 4), kKvHi,
                                     q_lo + (((ks >> 1) * (kN * 64) + (ks & 1) * 32) >> 4), kQHi, kIdescS);
                    umma_commit(&sm.s_full[i & 1]);
                    ++i;
                    since = clock64();
                } else if (clock64() - since > kWaitLimitCycles) {
                    set_error(kErrWaitTimeout);
                    ok = false;
                }
            }
            // no MMA is in flight when TMEM is released, after a wait that gave up as well
            umma_commit(&sm.drain);
            mbar_wait(&sm.drain, 0u);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = token (TMEM lane) 32 warp + lane of the tile
        // q of head h: 2^-e q = hi + lo / 16 in e4m3 (warp w: heads 4w .. 4w + 3; lane: 6 elements)
        {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q + (head0 + 4 * warp) * kD) + lane;
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
                const float s = quant::block_scale(a), inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
                if (lane == 0) {
                    sm.qscale[h] = s * p.scale_log2;
                    sm.m[h] = sm.M[h] = -INFINITY;
                    sm.mref[h] = sm.c[h] = 0.0f;
                }
                // dims 2 lane, 2 lane + 1 of block j
                const int at = ((((2 * lane) >> 4) ^ ((h >> 1) & 3)) << 4) + ((2 * lane) & 15);
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const float x = bf16_lo(w[i][j]) * inv, y = bf16_hi(w[i][j]) * inv;
                    const uint32_t hi = cvt_e4m3x2(x, y);
                    const uint32_t lo = cvt_e4m3x2((x - e4m3_to_f32(hi)) * 16.0f, (y - e4m3_to_f32(hi >> 8)) * 16.0f);
                    *reinterpret_cast<uint16_t *>(sm.q + j * (kN * 64) + h * 64 + at) = (uint16_t)hi;
                    *reinterpret_cast<uint16_t *>(sm.q + j * (kN * 64) + (16 + h) * 64 + at) = (uint16_t)lo;
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_ready);
        }
        attnq::warps_sync();                                     // qscale and the references
        const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16);
        float2 l[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) l[h] = make_float2(0.0f, 0.0f);
        bool unset = true, landed = true;
        for (int ti = 0; ti < n_tiles; ++ti) {
            const int st = ti % kStages;
            // a wait that gives up leaves the error flag and garbage; the later ones are then short,
            // and every barrier is still met
            auto wait = [&](uint64_t *bar, unsigned parity) {
                if (!mbar_wait(bar, parity, landed ? kWaitLimitCycles : 1ll << 22)) landed = false;
            };
            wait(&sm.full[st], (unsigned)(ti / kStages) & 1u);   // (the scales; long there)
            const int j = 4 * warp + (lane >> 3);
            const float4 sc = sm.scale[st][j];
            const int r = sm.region[st][j], tok = 8 * r + (lane & 7);
            const bool ok = r >= 0 && tok <= pos && tok >= t_lo;
            const bool all_ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                // a V row that no token attends: zero, whatever it holds
                uint8_t *v = ring + st * kTileBytes + j * kRegBytes + 512 + (lane & 7) * 64;
#pragma unroll
                for (int i = 0; i < 12; ++i) *reinterpret_cast<uint4 *>(v + (i >> 2) * 1024 + (i & 3) * 16) = make_uint4(0, 0, 0, 0);
            }
            wait(&sm.s_full[ti & 1], (unsigned)(ti >> 1) & 1u);
            __syncwarp();
            tc_fence_after();
            float x[32];
            tmem_ld32(trow + 32 * (ti & 1), x);
            float2 s[8], pr[8];                                  // scores, weights
            const float2 ks2 = make_float2(sc.x, sc.x), vs2 = make_float2(sc.y, sc.y);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float2 q2 = *reinterpret_cast<const float2 *>(&sm.qscale[2 * h]);
                const float2 y = ffma2(make_float2(x[16 + 2 * h], x[17 + 2 * h]), make_float2(0.0625f, 0.0625f),
                                       make_float2(x[2 * h], x[2 * h + 1]));
                s[h] = fmul2(fmul2(y, ks2), q2);
            }
            if (!all_ok) {
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (!ok) s[h] = make_float2(-INFINITY, -INFINITY);
            }
            bool grow = false;
            auto weights = [&]() {
                uint32_t w[8], top = 0u;
                float2 add = make_float2(0.0f, 0.0f);
                const float2 one2 = make_float2(1.0f, 1.0f);
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float2 mr = *reinterpret_cast<const float2 *>(&sm.mref[2 * h]);
                    const float2 cc = *reinterpret_cast<const float2 *>(&sm.c[2 * h]);
                    const float2 e = ffma2(s[h], one2, make_float2(-mr.x, -mr.y));
                    pr[h] = make_float2(ex2(e.x), ex2(e.y));
                    add = ffma2(pr[h], one2, add);
                    float2 f = fmul2(vs2, cc);
                    f = make_float2(fminf(f.x, 8.5070592e37f), fminf(f.y, 8.5070592e37f));     // 2^126
                    const float2 x2 = fmul2(pr[h], f);
                    w[h] = attnq::pack_f16x2(x2.x, x2.y);
                    top = attnq::max_f16x2(top, w[h]);
                }
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
                grow = add.x + add.y > kTop || any_above_top(top);
            };
            // P' of the tile before has been read
            if (ti > 0) wait(&sm.pv_done, (unsigned)(ti - 1) & 1u);
            __syncwarp();
            if (!unset) weights();
            tc_fence_before();
            if (attnq::warps_sync_or(grow || unset)) {
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
                    float a = lane < 16 ? sm.m[lane] : sm.M[lane - 16];
                    const float old = a;
#pragma unroll
                    for (int w = 0; w < 4; ++w) a = fmaxf(a, sm.red[w][lane]);
                    const float scale = old == a ? 1.0f : exp2f(old - a);
                    const float d = __shfl_xor_sync(0xffffffffu, a, 16);
                    if (lane < 16) {
                        sm.m[lane] = a;
                        sm.mref[lane] = a == -INFINITY ? 0.0f : a - kBase;
                        sm.c[lane] = d == -INFINITY ? 0.0f : exp2f(fminf(a - d, 126.0f));
                        sm.al[lane] = scale;
                    } else {
                        sm.M[lane - 16] = a;
                        sm.ao[lane - 16] = scale;
                    }
                }
                attnq::warps_sync();
                unset = false;
                bool rescale = false;
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    l[h] = fmul2(l[h], *reinterpret_cast<const float2 *>(&sm.al[2 * h]));
                    unset |= fminf(sm.M[2 * h], sm.M[2 * h + 1]) == -INFINITY;
                    rescale |= sm.ao[2 * h] != 1.0f || sm.ao[2 * h + 1] != 1.0f;
                }
                if (ti > 0 && rescale) {
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
                weights();
                attnq::warps_sync();
            }
#pragma unroll
            for (int h = 0; h < 8; ++h) l[h] = ffma2(pr[h], make_float2(1.0f, 1.0f), l[h]);
            if (tid == 0) mbar_arrive(&sm.p_ready);
        }
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
        if (warp == 0 && lane < 16) {
            const float L = (sm.red[0][lane] + sm.red[1][lane]) + (sm.red[2][lane] + sm.red[3][lane]);
            const float m = sm.m[lane], M = sm.M[lane];
            // 0 for a row with no token or no V; a NaN sum stays NaN (no comparison holds for it)
            sm.f[lane] = S > 1 ? L : L > 0.0f ? (M > -INFINITY ? exp2f(M - m) / L : 0.0f) : L;
            if (S == 1 && p.lse) p.lse[head0 + lane] = L == 0.0f ? -INFINITY : (m - kBase + log2f(L)) * 0.69314718055994531f;
        }
        if (n_tiles > 0) {
            if (!mbar_wait(&sm.pv_done, (unsigned)(n_tiles - 1) & 1u, landed ? kWaitLimitCycles : 1ll << 22)) landed = false;
        }
        attnq::warps_sync();                                     // the factors; every warp is past the ring
        tc_fence_after();
        float *stage = reinterpret_cast<float *>(ring);
#pragma unroll 1
        for (int h2 = 0; h2 < 2; ++h2) {
            if (h2 == 1 && warp < 2) break;                      // dims 64-127 again
            float o[16], o1[16], o2[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = o1[i] = o2[i] = 0.0f;
            if (n_tiles > 0) {
                __syncwarp();
                tmem_ld16(trow + kOCol + kNp * h2, o);
                tmem_ld16(trow + kOCol + kNp * h2 + 16, o1);
                tmem_ld16(trow + kOCol + kNp * h2 + 32, o2);
            }
            const int d = 64 * h2 + 32 * warp + lane;
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                const float y = o[h] + (o1[h] + o2[h]);
                if (S == 1) p.out[(head0 + h) * kD + d] = __float2bfloat16_rn(y * sm.f[h]);
                else stage[h * kInRow + d] = y;
            }
        }
        if (S > 1) {
            if (warp == 0 && lane < 16)
                *reinterpret_cast<float4 *>(stage + lane * kInRow + kD) = make_float4(sm.m[lane], sm.M[lane], sm.f[lane], 0.0f);
            fence_proxy_async();                                 // the rows, to the copy engine
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
    for (int e = tid; inbox_ok && e < per_cta * (kD / 2); e += kThreads) {
        const int j = e / (kD / 2), d = 2 * (e % (kD / 2));
        float mm = -INFINITY, MM = -INFINITY;
        for (int cc = 0; cc < S; ++cc) {
            const float *in = inbox + (cc * per_cta + j) * kInRow;
            mm = fmaxf(mm, in[kD]);
            MM = fmaxf(MM, in[kD + 1]);
        }
        const float mref = mm == -INFINITY ? 0.0f : mm, Mref = MM == -INFINITY ? 0.0f : MM;
        float Ls = 0.0f, x = 0.0f, y = 0.0f;
        for (int cc = 0; cc < S; ++cc) {
            const float *in = inbox + (cc * per_cta + j) * kInRow;
            const float2 v = *reinterpret_cast<const float2 *>(in + d);
            const float wt = exp2f(in[kD + 1] - Mref);
            Ls += exp2f(in[kD] - mref) * in[kD + 2];
            x += wt * v.x;
            y += wt * v.y;
        }
        const float f = Ls > 0.0f ? (MM > -INFINITY ? exp2f(MM - mm) / Ls : 0.0f) : Ls;
        const int64_t head = head0 + rank + S * j;
        *reinterpret_cast<uint32_t *>(p.out + head * kD + d) = pack_bf16x2(x * f, y * f);
        if (p.lse && d == 0) p.lse[head] = Ls == 0.0f ? -INFINITY : (mm - kBase + log2f(Ls)) * 0.69314718055994531f;
    }
    // this CTA's copies have read their rows before its shared memory goes away
    if (warp == 0 && lane < kHeadsPerGroup) bulk_wait_read_all();
}

}  // namespace attnqt
}  // namespace dsa

// Sparse and window GQA over the 8-bit paged cache (layout and scales: append_quant.cuh).
//
// A row is (query, KV group): 16 query heads over the tokens of its regions (the selection, or
// the window's regions), t <= p and inside the window.  One CTA of 4 warps per row streams the
// regions in tiles of 8 (64 tokens):
//  * S = q K^T on e4m3 tensor cores (mma.sync m16n8k32, fp32 accumulate) straight from the
//    codes; a head's q is split into two e4m3 terms, q / 2^e = hi + lo, which is exact for
//    elements above 2^-10 of the head's largest and off by at most 2^-18 of it below.  Warp w
//    takes regions 2w and 2w + 1 of the tile.  The K scale multiplies the finished dot product.
//  * softmax in fp32, log2 units, with a running reference m per head for the sum l.  The P that
//    meets V carries the V scale, so it has a reference of its own: P' = 2^(s - m) * sV * 2^(m -
//    M), M the running maximum of s + log2 sV.  P' is rounded to fp16 (2^-12 relative, and no
//    token within 2^-24 of the largest contribution is lost); l sums the unrounded fp32 P.
//  * O += P' V with V's codes converted to fp16 (exact) on mma.sync m16n8k16, fp32 accumulate;
//    warp w owns output dims [48w, 48w + 48), so no warp merges another's O.
//  * out = O / l * 2^(M - m), lse = ln 2 (m + log2 l); an empty row gives 0 and -inf.
// Rows of V that no token attends (behind the query, before the window, regions that are not
// there) are zeroed in shared memory: their P' is 0, but 0 * NaN is not.
#pragma once

#include <cuda_fp16.h>

#include "append_quant.cuh"
#include "common.cuh"

namespace dsa {
namespace attnq {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTileRegions = 8;                                  // 64 tokens
constexpr int kRegBytes = quant::kRegionBytesQ;                  // 3 KiB: K rows, then V rows
constexpr int kTileBytes = kTileRegions * kRegBytes;
constexpr int kQRow = kD + 16;                                   // q code rows, padded against bank conflicts
constexpr int kPRow = 2 * 64 + 16;                               // P' tile row (bytes), padded
constexpr float kSlack = 8.0f;                                   // log2 units a reference may lag behind
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    const __nv_bfloat16 *q;      // [nq][64][192]
    const uint8_t *cache;
    const float *scale;
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

__global__ void __launch_bounds__(kThreads) sparse_attn_quant_kernel(const Params p)
{
    pdl_trigger();   // the next kernel may launch; it waits for this one itself
    pdl_wait();      // the previous kernel's results are visible from here on
    __shared__ __align__(128) uint8_t tile[kTileBytes];
    __shared__ __align__(16) uint8_t qcodes[2][16 * kQRow];      // hi, lo
    __shared__ float qscale[16];
    __shared__ __align__(16) uint8_t ptile[2][16 * kPRow];
    __shared__ float mx_sh[kWarps][16][2];
    __shared__ float l_sh[kWarps][16];
    __shared__ int r_sh[kTileRegions];                           // region (-1: none)
    __shared__ float ks_sh[kTileRegions], vs_sh[kTileRegions];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, t = lane & 3;
    const int g = (int)(blockIdx.x / (unsigned)p.nq), qi = (int)(blockIdx.x % (unsigned)p.nq);
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

    // q of head h, 2^-e q = hi + lo in e4m3 (warp w: heads 4w .. 4w + 3; lane: 6 elements)
    for (int h = 4 * warp; h < 4 * warp + 4; ++h) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q + ((int64_t)qi * kHQ + g * kHeadsPerGroup + h) * kD);
        float v[6], a = 0.0f;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const uint32_t w = __ldg(src + lane + 32 * j);
            v[2 * j] = bf16_lo(w);
            v[2 * j + 1] = bf16_hi(w);
            a = fmaxf(a, fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const float s = quant::block_scale(a), inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
        if (lane == 0) qscale[h] = s * p.scale_log2;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const float x = v[2 * j] * inv, y = v[2 * j + 1] * inv;
            const uint32_t hi = cvt_e4m3x2(x, y);
            const uint32_t lo = cvt_e4m3x2(x - e4m3_to_f32(hi), y - e4m3_to_f32(hi >> 8));
            *reinterpret_cast<uint16_t *>(qcodes[0] + h * kQRow + 2 * (lane + 32 * j)) = (uint16_t)hi;
            *reinterpret_cast<uint16_t *>(qcodes[1] + h * kQRow + 2 * (lane + 32 * j)) = (uint16_t)lo;
        }
    }
    __syncthreads();
    // A fragments of q: rows gq, gq + 8; k = 32 ks + 4t .. + 3 and + 16
    uint32_t qa[2][6][4];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int ks = 0; ks < 6; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qa[s][ks][i] = *reinterpret_cast<const uint32_t *>(qcodes[s] + (gq + 8 * (i & 1)) * kQRow + 32 * ks +
                                                                  16 * (i >> 1) + 4 * t);
    const float qf[2] = {qscale[gq], qscale[gq + 8]};

    float o[3][2][4];                                            // 16-dim block, even / odd dims
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) o[j][s][0] = o[j][s][1] = o[j][s][2] = o[j][s][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, M[2] = {-INFINITY, -INFINITY};      // references (rows gq, gq + 8)
    float c[2] = {0.0f, 0.0f};                                   // 2^(m - M)
    float l[2] = {0.0f, 0.0f};                                   // this thread's part of the sum

    const int n_tiles = (cnt + kTileRegions - 1) / kTileRegions;
    for (int ti = 0; ti < n_tiles; ++ti) {
        const int j0 = ti * kTileRegions, nr = min(kTileRegions, cnt - j0);
        __syncthreads();                                         // the previous tile is done with
        if (tid < kTileRegions) {
            int r = -1;
            float ks = 0.0f, vs = 0.0f;
            int64_t rid = 0;
            if (tid < nr) {
                r = p.window > 0 ? (t_lo >> 3) + j0 + tid : p.sel_idx[(int64_t)row * p.k + j0 + tid];
                const int64_t page = (r < 0 || r / 8 >= p.max_pages) ? -1 : p.block_table[(int64_t)b * p.max_pages + r / 8];
                if (page < 0 || page >= p.n_pages) {
                    set_error(kErrAttnIndex);
                    r = -1;
                } else {
                    rid = (page * kG + g) * quant::kRegionsPerPage + r % 8;
                    ks = p.scale[2 * rid];
                    vs = p.scale[2 * rid + 1];
                }
            }
            r_sh[tid] = r;
            ks_sh[tid] = ks;
            vs_sh[tid] = vs;
            // the region's address travels through the tile's first bytes of its slot
            *reinterpret_cast<int64_t *>(tile + tid * kRegBytes) = rid;
        }
        __syncthreads();
        int64_t rid[kTileRegions];
#pragma unroll
        for (int j = 0; j < kTileRegions; ++j) rid[j] = *reinterpret_cast<const int64_t *>(tile + j * kRegBytes);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kTileRegions; ++j) {
            const bool there = r_sh[j] >= 0;
            for (int i = tid; i < kRegBytes / 16; i += kThreads) {
                const int rr = i / (kD / 16), cc = i % (kD / 16);
                uint4 v = make_uint4(0, 0, 0, 0);
                // rows of V that no token attends stay zero
                const int tok = 8 * r_sh[j] + (rr & 7);
                if (there && (rr < 8 || (tok <= pos && tok >= t_lo)))
                    v = __ldg(reinterpret_cast<const uint4 *>(p.cache + rid[j] * kRegBytes) + i);
                *reinterpret_cast<uint4 *>(tile + j * kRegBytes + swz(rr, cc * 16)) = v;
            }
        }
        __syncthreads();

        // ---- S of regions 2w, 2w + 1
        float s[2][4];
        float mxs[2] = {-INFINITY, -INFINITY}, mxv[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const int j = 2 * warp + nt;
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const uint32_t base = smem_u32(tile + j * kRegBytes);
#pragma unroll
            for (int kb = 0; kb < 3; ++kb) {
                uint32_t b0, b1, b2, b3;
                ldmatrix_x4(base + swz(lane & 7, kb * 64 + 16 * (lane >> 3)), b0, b1, b2, b3);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mma_e4m3_16832(acc, qa[x][2 * kb], b0, b1);
                    mma_e4m3_16832(acc, qa[x][2 * kb + 1], b2, b3);
                }
            }
            const int r = r_sh[j];
            const float ks = ks_sh[j], lv = log2f(vs_sh[j]);
            float mr[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int tok = 8 * r + 2 * t + (e & 1);
                const bool ok = r >= 0 && tok <= pos && tok >= t_lo;
                s[nt][e] = ok ? acc[e] * (qf[e >> 1] * ks) : -INFINITY;
                mr[e >> 1] = fmaxf(mr[e >> 1], s[nt][e]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mxs[h] = fmaxf(mxs[h], mr[h]);
                mxv[h] = fmaxf(mxv[h], mr[h] + lv);
            }
        }
        // ---- move the references where a token passes them by more than the slack
        const bool grow = mxs[0] > m[0] + kSlack || mxs[1] > m[1] + kSlack || mxv[0] > M[0] + kSlack ||
                          mxv[1] > M[1] + kSlack;
        if (__syncthreads_or(grow)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mxs[h] = fmaxf(mxs[h], __shfl_xor_sync(0xffffffffu, mxs[h], 1));
                mxs[h] = fmaxf(mxs[h], __shfl_xor_sync(0xffffffffu, mxs[h], 2));
                mxv[h] = fmaxf(mxv[h], __shfl_xor_sync(0xffffffffu, mxv[h], 1));
                mxv[h] = fmaxf(mxv[h], __shfl_xor_sync(0xffffffffu, mxv[h], 2));
                if (t == 0) {
                    mx_sh[warp][gq + 8 * h][0] = mxs[h];
                    mx_sh[warp][gq + 8 * h][1] = mxv[h];
                }
            }
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float a = m[h], d = M[h];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    a = fmaxf(a, mx_sh[w][gq + 8 * h][0]);
                    d = fmaxf(d, mx_sh[w][gq + 8 * h][1]);
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
                c[h] = d == -INFINITY ? 0.0f : exp2f(fminf(a - d, 126.0f));
            }
        }
        // ---- P' of regions 2w, 2w + 1
        const float mref[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
        uint8_t *pt = ptile[ti & 1];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const float vs = vs_sh[2 * warp + nt];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float p0 = exp2f(s[nt][2 * h] - mref[h]), p1 = exp2f(s[nt][2 * h + 1] - mref[h]);
                l[h] += p0 + p1;
                const float f = fminf(vs * c[h], 8.5070592e37f);                   // 2^126
                *reinterpret_cast<uint32_t *>(pt + (gq + 8 * h) * kPRow + 2 * (16 * warp + 8 * nt + 2 * t)) =
                    pack_f16x2(p0 * f, p1 * f);
            }
        }
        __syncthreads();
        // ---- O[:, 48w .. 48w + 47] += P' V, two k-steps (4 regions) at a time
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t pa[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                ldmatrix_x4(smem_u32(pt) + (lane & 15) * kPRow + 64 * kk + 32 * x + 16 * (lane >> 4), pa[x][0], pa[x][1],
                            pa[x][2], pa[x][3]);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                uint32_t v[4];
                ldmatrix_x4_trans(smem_u32(tile + (4 * kk + (lane >> 3)) * kRegBytes) +
                                      swz(8 + (lane & 7), 48 * warp + 16 * j), v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    // (token 2t: dims d, d + 1)(token 2t + 1: dims d, d + 1) -> pairs of tokens per dim
                    const uint32_t a = __byte_perm(v[2 * x], 0, 0x3120), bb = __byte_perm(v[2 * x + 1], 0, 0x3120);
                    mma_f16_16816(o[j][0], pa[x], e4m3x2_to_f16x2((uint16_t)a), e4m3x2_to_f16x2((uint16_t)bb));
                    mma_f16_16816(o[j][1], pa[x], e4m3x2_to_f16x2((uint16_t)(a >> 16)), e4m3x2_to_f16x2((uint16_t)(bb >> 16)));
                }
            }
        }
    }

    // ---- the row's sums, then the outputs of this warp's dims
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (t == 0) l_sh[warp][gq + 8 * h] = l[h];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int hr = gq + 8 * h;
        const float L = (l_sh[0][hr] + l_sh[1][hr]) + (l_sh[2][hr] + l_sh[3][hr]);
        const int64_t head = (int64_t)qi * kHQ + g * kHeadsPerGroup + hr;
        const float f = L > 0.0f && M[h] > -INFINITY ? exp2f(M[h] - m[h]) / L : 0.0f;
        // NaN stays NaN: L is then NaN too, and no comparison holds
        const float z = L == L ? f : L;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int d = 48 * warp + 16 * j + 4 * t;
            const uint2 v = make_uint2(pack_bf16x2(o[j][0][2 * h] * z, o[j][1][2 * h] * z),
                                       pack_bf16x2(o[j][0][2 * h + 1] * z, o[j][1][2 * h + 1] * z));
            *reinterpret_cast<uint2 *>(p.out + head * kD + d) = v;
        }
        if (p.lse && warp == 0 && t == 0)
            p.lse[head] = L == 0.0f ? -INFINITY : (m[h] + log2f(L)) * 0.69314718055994531f;
    }
}

}  // namespace attnq
}  // namespace dsa

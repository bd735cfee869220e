// What the two attention kernels over the 8-bit paged cache share (layout and scales of the cache:
// append_quant.cuh; one cluster or CTA per row: attention_quant_tc.cuh; windows of chunks:
// attention_quant_band.cuh).
#pragma once

#include <cuda_fp16.h>

#include "append_quant.cuh"
#include "common.cuh"

namespace dsa {
namespace attnq {

constexpr int kRegBytes = quant::kRegionBytesQ;                  // 3 KiB: K rows, then V rows
constexpr float kLog2e = 1.4426950408889634f;

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
    int splits;                  // row kernel: CTAs (the cluster) per row: 1, 2, 4, 8 or 16
    int per;                     // regions of a row for each of them
    unsigned row0, row_end;      // row kernel: the launch's rows, of nq * 4
};

// A pair of e4m3 codes -> fp16 (exact).
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

}  // namespace attnq
}  // namespace dsa

// zccl_fp8.cuh -- device helpers of the block-scaled e4m3 products: the scale
// of a block, the conversion to e4m3, and the table of the groups' tiles.
#pragma once

#include "zccl_fp8.h"
#include "zccl_ops.cuh"

namespace zccl {

// A block's largest magnitude counts as at least 2^-100, so that neither the
// scale nor its inverse leaves the normal range (an all-zero block gets a
// scale, too, and codes of zero).
constexpr float kAmaxMin = 7.888609052210118e-31f;
constexpr float kE4m3Max = 448.0f;

// scale = amax / 448 and the factor 448 * (1 / amax), every operation rounded
// in fp32.
__device__ __forceinline__ void block_scale(float amax, float* scale, float* factor)
{
    const float a = fmaxf(amax, kAmaxMin);
    *scale = a / kE4m3Max;
    *factor = kE4m3Max * (1.0f / a);
}

// Two values as e4m3 (nearest even, saturating, NaN kept): lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Sizes of the groups from the table of their first rows, which is not
// trusted: every row index stays within 0..rows whatever it holds.
__device__ __forceinline__ void group_rows(const int32_t* offsets, uint32_t rows, uint32_t g, uint32_t* lo, uint32_t* hi)
{
    if (offsets == nullptr) {
        *lo = 0;
        *hi = rows;
        return;
    }
    const int32_t a = ld_l2(offsets + g), b = ld_l2(offsets + g + 1);
    *lo = a < 0 ? 0u : min((uint32_t)a, rows);
    *hi = b < 0 ? 0u : min((uint32_t)b, rows);
    if (*hi < *lo) *hi = *lo;
}

// Exclusive prefix sum, by warp 0, of each group's blocks of `unit` rows:
// prefix[0..G] (shared memory).  G <= 512.  With `limit` a table that claims
// more blocks than that is cut off there.
__device__ __forceinline__ void group_prefix(const int32_t* offsets, uint32_t rows, uint32_t G, uint32_t unit,
                                             uint32_t limit, uint32_t* prefix)
{
    if (threadIdx.x >= 32) return;
    const uint32_t per = (G + 31) / 32, first = min(G, threadIdx.x * per), last = min(G, first + per);
    uint32_t sum = 0;
    for (uint32_t g = first; g < last; ++g) {
        uint32_t lo, hi;
        group_rows(offsets, rows, g, &lo, &hi);
        const uint32_t n = (hi - lo + unit - 1) / unit;
        prefix[g] = n;
        sum += n;
    }
    uint32_t run = (uint32_t)warp_scan(sum) - sum;
    for (uint32_t g = first; g < last; ++g) {
        const uint32_t n = prefix[g];
        prefix[g] = min(run, limit);
        run += n;
    }
    const uint32_t total = __shfl_sync(0xFFFFFFFFu, run, 31);
    if (threadIdx.x == 0) prefix[G] = min(total, limit);
}

// The group whose range of prefix holds i (i < prefix[G]).
__device__ __forceinline__ uint32_t group_at(const uint32_t* prefix, uint32_t G, uint32_t i)
{
    uint32_t lo = 0, hi = G;  // prefix[lo] <= i < prefix[hi]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (prefix[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

}  // namespace zccl

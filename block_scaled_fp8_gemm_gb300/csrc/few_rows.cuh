// few_rows.cuh -- what the kernels for few rows of activations share: the weights are the MMA's M
// operand, a pair of 128-row tiles per stage, and the activations' rows its N columns.  Eight
// promotion warps keep one weight row of one tile per thread, for all columns.
#pragma once

#include <atomic>

#include "kernels.h"

namespace gemmar {

constexpr int kThreads = 384;
constexpr int kEpiThreads = 256;
constexpr int kTileBytes = 128 * 128;
constexpr int kRegsLow = 56;     // warps 0-3 after setmaxnreg.dec
constexpr int kRegsHigh = 224;   // promotion warps after setmaxnreg.inc
constexpr uint32_t kAbortGraceNs = 200000;   // let copies in flight land before an aborting CTA exits

// The kernel was built with registers enough for that split (setmaxnreg would wait forever).  known: that
// it was; a query that failed is made again by the next call.
inline bool few_rows_split_ok(std::atomic<bool> &known, const void *kernel, int low = kRegsLow, int high = kRegsHigh)
{
    if (!known) {
        cudaFuncAttributes f;
        known = cudaFuncGetAttributes(&f, kernel) == cudaSuccess && f.numRegs * kThreads >= 128 * low + kEpiThreads * high;
    }
    return known;
}

// acc[j] += (sum of column j) * (weight scale * token scale j) for 8 columns
__device__ __forceinline__ void promote8(float *acc, const uint32_t (&d)[8], const float *ts)
{
    const float4 a = *reinterpret_cast<const float4 *>(ts), b = *reinterpret_cast<const float4 *>(ts + 4);
    ptx::fma2(acc[0], acc[1], __uint_as_float(d[0]), __uint_as_float(d[1]), a.x, a.y);
    ptx::fma2(acc[2], acc[3], __uint_as_float(d[2]), __uint_as_float(d[3]), a.z, a.w);
    ptx::fma2(acc[4], acc[5], __uint_as_float(d[4]), __uint_as_float(d[5]), b.x, b.y);
    ptx::fma2(acc[6], acc[7], __uint_as_float(d[6]), __uint_as_float(d[7]), b.z, b.w);
}

}  // namespace gemmar

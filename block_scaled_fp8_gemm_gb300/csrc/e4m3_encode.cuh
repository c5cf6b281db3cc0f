// e4m3_encode.cuh -- the e4m3 encoder of the quantisers: codes = e4m3_rn_sat(x / s)
// with the IEEE quotient, mostly without dividing.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace gemmar {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t enc4(float a, float b, float c, float d, float s)
{
    if (s == 0.0f)
        return 0u;
    uint32_t lo = ptx::e4m3x2_from_f32(__fdiv_rn(a, s), __fdiv_rn(b, s));
    uint32_t hi = ptx::e4m3x2_from_f32(__fdiv_rn(c, s), __fdiv_rn(d, s));
    return lo | (hi << 16);
}

// e4m3 codes of RN(a/s) and RN(b/s) without dividing, given yl = RN(y(1 - 2^-21))
// and yh = RN(y(1 + 2^-21)) for y = RN(1/s) (s > 0, y a normal number).  The
// products l = RN(a yl) and h = RN(a yh) are a/s times (1 -+ 2^-21) and three
// rounding factors, each within 2^-24 of 1; (1 + 2^-24)^3 < 1 + 2^-21, so |l| <
// |a/s| < |h| (below the normal range, all three round to a zero code anyway).
// Rounding to e4m3 (nearest-even, saturating) is monotone, so when l and h give
// the same code every value between them does, RN(a/s) included.  Otherwise a/s
// lies within ~2^-21 of a code midpoint: divide exactly.  With bf16 inputs this
// happens to ~0.5% of the values (x 448 / amax is then exactly a midpoint), so
// the division stays per pair: a fallback for a whole lane's values would be
// taken by most warps.
__device__ __forceinline__ uint32_t enc2_guarded(float a, float b, float s, float yl, float yh)
{
    // the products two per packed instruction
    const float2 l = ptx::mul2(a, b, yl, yl);
    const float2 h = ptx::mul2(a, b, yh, yh);
    const uint32_t lo = ptx::e4m3x2_from_f32(l.x, l.y);
    const uint32_t hi = ptx::e4m3x2_from_f32(h.x, h.y);
    if (lo == hi)
        return lo;
    return ptx::e4m3x2_from_f32(__fdiv_rn(a, s), __fdiv_rn(b, s));
}

// Row/group encoder: the guarded products when 1/s is a normal number below
// 2^125, exact division otherwise (s == 0 gives +0 codes).  s = amax / 448 is at
// most FLT_MAX / 448, so y is never subnormal; s = inf gives y = 0 and products
// equal to the exact quotients' codes (+-0, and NaN for an infinite input).
struct Enc {
    float s, yl, yh;
    bool fast;
    __device__ __forceinline__ static float reciprocal(float sc) { return sc > 0.0f ? __frcp_rn(sc) : 0.0f; }
    __device__ __forceinline__ explicit Enc(float sc) : Enc(sc, reciprocal(sc)) {}
    __device__ __forceinline__ Enc(float sc, float y) : s(sc)
    {
        yl = __fmul_rn(y, 1.0f - 0x1p-21f);
        yh = __fmul_rn(y, 1.0f + 0x1p-21f);
        fast = sc >= 0x1p-125f;   // 1/s <= 2^125: finite, and y (1 + 2^-21) cannot overflow
    }
    // from the fields of an encoder built earlier (kept in shared memory)
    __device__ __forceinline__ Enc(float sc, float yl_, float yh_, bool fast_) : s(sc), yl(yl_), yh(yh_), fast(fast_) {}
    __device__ __forceinline__ uint32_t operator()(float a, float b, float c, float d) const
    {
        if (!fast)
            return enc4(a, b, c, d, s);
        return enc2_guarded(a, b, s, yl, yh) | (enc2_guarded(c, d, s, yl, yh) << 16);
    }
    // The same codes for W values that come from fp32 arithmetic, where a quotient this
    // near a midpoint is rare (2^-20 or so a value): one test for all of them, and the
    // divisions for all where it fails.
    template <int W>
    __device__ __forceinline__ void codes(const float (&x)[W], uint32_t (&w)[W / 4]) const
    {
        uint32_t differ = fast ? 0u : 1u;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const float2 l0 = ptx::mul2(x[4 * i], x[4 * i + 1], yl, yl), l1 = ptx::mul2(x[4 * i + 2], x[4 * i + 3], yl, yl);
            const float2 h0 = ptx::mul2(x[4 * i], x[4 * i + 1], yh, yh), h1 = ptx::mul2(x[4 * i + 2], x[4 * i + 3], yh, yh);
            w[i] = ptx::e4m3x2_from_f32(l0.x, l0.y) | (ptx::e4m3x2_from_f32(l1.x, l1.y) << 16);
            differ |= w[i] ^ (ptx::e4m3x2_from_f32(h0.x, h0.y) | (ptx::e4m3x2_from_f32(h1.x, h1.y) << 16));
        }
        if (differ != 0u) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
                w[i] = enc4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], s);
        }
    }
};

}  // namespace gemmar

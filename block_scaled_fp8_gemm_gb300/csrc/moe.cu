// moe.cu -- the experts' layer for a few tokens (moe_apply).
//
//   out[t] = y[t] + sum_s w[t,s] W2[e] (act(G[e] x[t]) * (U[e] x[t])),   e = the expert of slot s
#include "activation.cuh"
#include "e4m3_encode.cuh"
#include "kernels.h"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ int expert_of(const MoeArgs &a, int slot)
{
    int e = a.ids[slot];
    if (a.place != nullptr)
        e = e >= 0 && e < a.places ? a.place[e] : -1;
    return e >= 0 && e < a.E ? e : -1;
}

__device__ __forceinline__ void decode16(const uint8_t *p, float (&v)[16])
{
    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = f32x2_from_e4m3x2((uint16_t)w[i]), hi = f32x2_from_e4m3x2((uint16_t)(w[i] >> 16));
        v[4 * i] = lo.x;
        v[4 * i + 1] = lo.y;
        v[4 * i + 2] = hi.x;
        v[4 * i + 3] = hi.y;
    }
}

__device__ __forceinline__ float warp_sum(float s)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

// hidden[slot, i]: a warp per value
__global__ void __launch_bounds__(kThreads) moe_up_kernel(const MoeArgs a, float *hidden)
{
    const int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), slot = blockIdx.y, lane = threadIdx.x & 31;
    const int e = expert_of(a, slot), t = slot / a.k, HB = a.H / 128;
    if (e < 0)
        return;
    const int64_t row = (int64_t)e * 2 * a.I + i;
    const uint8_t *g = a.w13 + row * a.H, *u = g + (int64_t)a.I * a.H, *x = a.q + (int64_t)t * a.H;
    const float *sg = a.s13 + row / 128 * HB, *su = a.s13 + (row + a.I) / 128 * HB, *sx = a.sx + (int64_t)t * HB;
    float zg = 0.0f, zu = 0.0f;
    for (int c = lane * 16; c < a.H; c += 512) {
        float xv[16], gv[16], uv[16], pg = 0.0f, pu = 0.0f;
        decode16(x + c, xv);
        decode16(g + c, gv);
        decode16(u + c, uv);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            pg = fmaf(xv[j], gv[j], pg);
            pu = fmaf(xv[j], uv[j], pu);
        }
        zg = fmaf(sx[c / 128] * sg[c / 128], pg, zg);
        zu = fmaf(sx[c / 128] * su[c / 128], pu, zu);
    }
    zg = warp_sum(zg);
    zu = warp_sum(zu);
    if (lane == 0)
        with_act(a.act, [&](auto act) {
            hidden[(int64_t)slot * a.I + i] = act_value<decltype(act)::value>(zg) * zu * a.weights[slot];
        });
}

// out[t, n]: a warp per value
__global__ void __launch_bounds__(kThreads) moe_down_kernel(const MoeArgs a, const float *hidden)
{
    const int n = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), t = blockIdx.y, lane = threadIdx.x & 31;
    float sum = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int slot = t * a.k + j, e = expert_of(a, slot);
        if (e < 0)
            continue;
        const int64_t row = (int64_t)e * a.H + n;
        const float *h = hidden + (int64_t)slot * a.I, *s = a.s2 + row / 128 * (a.I / 128);
        for (int c = lane * 16; c < a.I; c += 512) {
            float wv[16], p = 0.0f;
            decode16(a.w2 + row * a.I + c, wv);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                p = fmaf(wv[i], h[c + i], p);
            sum = fmaf(s[c / 128], p, sum);
        }
    }
    sum = warp_sum(sum);
    if (lane == 0) {
        if (a.y != nullptr)
            sum += bf16_lo(a.y[t * a.ys + n]);
        a.out[t * a.os + n] = (uint16_t)bf16x2_from_f32(sum, 0.0f);
    }
}

}  // namespace

int64_t moe_ws_floats(const MoeArgs &a) { return (int64_t)a.T * a.k * a.I; }

cudaError_t launch_moe(const MoeArgs &a, float *ws, cudaStream_t st)
{
    moe_up_kernel<<<dim3(a.I / (kThreads / 32), a.T * a.k), kThreads, 0, st>>>(a, ws);
    moe_down_kernel<<<dim3(a.H / (kThreads / 32), a.T), kThreads, 0, st>>>(a, ws);
    return cudaGetLastError();
}

}  // namespace gemmar

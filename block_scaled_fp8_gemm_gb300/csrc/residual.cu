// residual.cu -- a block's output joins the residual stream: norms before and
// after, gate, residual scale, and the next block's input as bf16 rows or as
// e4m3 codes with 1x128 scales (norm_gate_residual), and its backward pass.
// One CTA takes a row at a time; every pass over the row re-reads it.
#include <cuda_bf16.h>

#include "kernels.h"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const void *p, int bf16, int64_t i)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store1(void *p, int bf16, int64_t i, float v)
{
    if (bf16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kThreads / 32; ++i)
        v += red[i];
    return v;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs a)
{
    __shared__ float red[kThreads / 32];
    const int64_t m = blockIdx.x;
    const int N = a.N, tid = threadIdx.x;
    float r1 = 1.0f, r2 = 1.0f;
    if (a.w1) {
        float s = 0.0f;
        for (int n = tid; n < N; n += kThreads) {
            const float y = load1(a.y, a.y_bf16, m * a.ys + n);
            s += y * y;
        }
        r1 = 1.0f / sqrtf(block_sum(s, red) / N + a.eps);
    }
    auto joined = [&](int n) {
        float z = load1(a.y, a.y_bf16, m * a.ys + n) * r1;
        if (a.w1)
            z *= a.w1[n];
        if (a.gate)
            z *= load1(a.gate, 1, m * a.gs + n);
        return a.alpha * load1(a.h, a.h_bf16, m * a.hs + n) + a.beta * z;
    };
    float s = 0.0f;
    for (int n = tid; n < N; n += kThreads) {
        const float t = joined(n);
        s += t * t;
    }
    if (a.w2)
        r2 = 1.0f / sqrtf(block_sum(s, red) / N + a.eps);
    if (a.rstd && tid == 0) {
        a.rstd[2 * m] = r1;
        a.rstd[2 * m + 1] = r2;
    }
    // a warp takes 128 columns, four a lane: one scale group
    for (int n0 = (tid >> 5) * 128; n0 < N; n0 += kThreads * 4) {
        float x[4];
        float amax = 0.0f;
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + (tid & 31) * 4 + j;
            x[j] = 0.0f;
            if (n < N) {
                const float t = joined(n);
                if (a.w2)
                    x[j] = t * r2 * a.w2[n];
                store1(a.t, a.h_bf16, m * N + n, t);
                if (a.u)
                    store1(a.u, 1, m * N + n, x[j]);
            }
            amax = fmaxf(amax, fabsf(x[j]));
        }
        if (a.q) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            const float sc = __fdiv_rn(amax, 448.0f);
            uint32_t c = 0u;
            if (sc != 0.0f)
                c = e4m3x2_from_f32(__fdiv_rn(x[0], sc), __fdiv_rn(x[1], sc)) |
                    (e4m3x2_from_f32(__fdiv_rn(x[2], sc), __fdiv_rn(x[3], sc)) << 16);
            reinterpret_cast<uint32_t *>(a.q + m * N + n0)[tid & 31] = c;
            if ((tid & 31) == 0)
                a.scales[m * (N / 128) + n0 / 128] = sc;
        }
    }
}

// Rows m = blockIdx.x, + gridDim.x, ...; the CTA's part of the sums over rows is
// kept in ws[blockIdx.x][2][N], each column by one thread.
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormBwdArgs a, float *__restrict__ ws)
{
    __shared__ float red[kThreads / 32];
    const int N = a.N, tid = threadIdx.x;
    float *s1 = ws + (int64_t)blockIdx.x * 2 * N, *s2 = s1 + N;
    for (int n = tid; n < N; n += kThreads)
        s1[n] = s2[n] = 0.0f;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const float r1 = a.rstd[2 * m], r2 = a.rstd[2 * m + 1];
        auto gw = [&](int n) {
            float c = a.beta;
            if (a.w1)
                c *= a.w1[n];
            if (a.gate)
                c *= load1(a.gate, 1, m * a.gs + n);
            return c;
        };
        auto nrm = [&](int n) { return load1(a.y, a.y_bf16, m * a.ys + n) * r1; };
        auto that = [&](int n) { return (a.alpha * load1(a.h, a.h_bf16, m * a.hs + n) + gw(n) * nrm(n)) * r2; };
        auto dv = [&](int n) { return load1(a.du, 1, m * a.dus + n) * a.w2[n]; };
        float mean = 0.0f;
        if (a.w2) {
            for (int n = tid; n < N; n += kThreads)
                mean += dv(n) * that(n);
            mean = block_sum(mean, red) / N;
        }
        auto dsum = [&](int n) {
            float d = a.dt ? load1(a.dt, a.h_bf16, m * a.dts + n) : 0.0f;
            if (a.w2)
                d += r2 * (dv(n) - that(n) * mean);
            return d;
        };
        float mean1 = 0.0f;
        if (a.w1) {
            for (int n = tid; n < N; n += kThreads)
                mean1 += gw(n) * dsum(n) * nrm(n);
            mean1 = block_sum(mean1, red) / N;
        }
        // dy and dh may be y and dt themselves: a column is read whole before it is written
        for (int n = tid; n < N; n += kThreads) {
            const float d = dsum(n), nn = nrm(n);
            const float dy = r1 * (gw(n) * d - nn * mean1);
            s1[n] += nn * d * ((a.gate && a.gs != 0) ? load1(a.gate, 1, m * a.gs + n) : 1.0f);
            if (a.w2)
                s2[n] += load1(a.du, 1, m * a.dus + n) * that(n);
            if (a.dgate && a.gs != 0)
                store1(a.dgate, 1, m * N + n, a.beta * nn * (a.w1 ? a.w1[n] : 1.0f) * d);
            store1(a.dy, a.y_bf16, m * N + n, dy);
            store1(a.dh, a.h_bf16, m * N + n, a.alpha * d);
        }
    }
}

// The CTAs' parts, summed in the order of the CTAs.  s1 = sum n d (times a token's
// gate): dw1 = beta g s1 and dgate = beta w1 s1 for a gate row g.
__global__ void __launch_bounds__(kThreads) norm_bwd_sum_kernel(const NormBwdArgs a, const float *__restrict__ ws,
                                                                int parts)
{
    const int n = blockIdx.x * kThreads + threadIdx.x;
    if (n >= a.N)
        return;
    float s1 = 0.0f, s2 = 0.0f;
    for (int p = 0; p < parts; ++p) {
        s1 += ws[(int64_t)p * 2 * a.N + n];
        s2 += ws[(int64_t)p * 2 * a.N + a.N + n];
    }
    const bool row = a.gate && a.gs == 0;
    if (a.dw1)
        a.dw1[n] = a.beta * (row ? load1(a.gate, 1, n) : 1.0f) * s1;
    if (a.dw2)
        a.dw2[n] = s2;
    if (a.dgate && row)
        static_cast<float *>(a.dgate)[n] = a.beta * (a.w1 ? a.w1[n] : 1.0f) * s1;
}

int bwd_ctas(int64_t M, int num_sms) { return (int)(M < 4 * (int64_t)num_sms ? (M + 3) / 4 : num_sms); }

}  // namespace

int64_t norm_bwd_ws_floats(int64_t M, int N, int num_sms) { return (int64_t)bwd_ctas(M, num_sms) * 2 * N; }

cudaError_t launch_norm(const NormArgs &a, int, cudaStream_t st)
{
    norm_kernel<<<(unsigned)a.M, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, float *ws, int num_sms, cudaStream_t st)
{
    const int ctas = bwd_ctas(a.M, num_sms);
    norm_bwd_kernel<<<ctas, kThreads, 0, st>>>(a, ws);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.dw1 && !a.dw2 && !(a.dgate && a.gs == 0)))
        return e;
    norm_bwd_sum_kernel<<<(a.N + kThreads - 1) / kThreads, kThreads, 0, st>>>(a, ws, ctas);
    return cudaGetLastError();
}

}  // namespace gemmar

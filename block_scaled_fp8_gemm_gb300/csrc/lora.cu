// lora.cu -- low-rank adapters of many requests beside a shared projection.
// Both factors of an adapter are stored rank-major ([R, r, C]), so the forward
// pass and its gradients are three products over the tokens of each adapter:
//   down: v[i,j] = f sum_c x[t,c] W[a,j,c]              (x A^T; dy B^T)
//   up:   out[t,c] = base[t,c] + f sum_j v[i,j] W[a,j,c]  (v B; w A)
//   grad: G[a,j,c] = f sum_i p[i,j] x[t,c]              (w^T x; v^T dy)
// with t = order[i], i in [offsets[a], offsets[a+1]), f = scales[a] or 1.
#include <cuda_bf16.h>

#include "kernels.h"

namespace gemmar {
using namespace ptx;

namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t to_bf(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Adapter of position i: the a with offsets[a] <= i < offsets[a+1]; R past offsets[R].
__device__ __forceinline__ int adapter_of(const int32_t *__restrict__ offsets, int R, int64_t i)
{
    int lo = 0, hi = R;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (offsets[mid + 1] > i)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int rank_of(const LoraArgs &l, int a)
{
    return l.ranks ? min(max(l.ranks[a], 0), l.r) : l.r;
}

// Counting sort by adapter in one CTA of 32 warps: a warp counts its contiguous
// share of the tokens per adapter, the counts are summed over adapters and
// warps, and the warp then places its tokens in order.  Stable, so the sums
// over an adapter's tokens have one order.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t *__restrict__ ids, int T, int R,
                                                         int32_t *__restrict__ order, int32_t *__restrict__ offsets)
{
    extern __shared__ int count[];   // [32][R + 1], then 32
    const int bins = R + 1;
    int *sums = count + 32 * bins;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int *mine = count + warp * bins;
    for (int i = lane; i < bins; i += 32)
        mine[i] = 0;
    __syncwarp();
    const int share = ((T + 31) / 32 + 31) / 32 * 32;
    const int lo = min(warp * share, T), hi = min(lo + share, T);
    for (int pass = 0; pass < 2; ++pass) {
        for (int t0 = lo; t0 < hi; t0 += 32) {
            const int t = t0 + lane;
            int bin = -1;
            if (t < hi) {
                const int a = ids[t];
                bin = a >= 0 && a < R ? a : R;
            }
            const unsigned same = __match_any_sync(0xFFFFFFFFu, bin);
            const int before = __popc(same & ((1u << lane) - 1));
            if (pass == 1 && bin >= 0)
                order[mine[bin] + before] = t;
            __syncwarp();
            if (bin >= 0 && before == 0)
                mine[bin] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        if (pass == 0) {
            // thread i < bins: tokens of adapter i, then the exclusive sum over adapters
            int total = 0;
            const int i = threadIdx.x;
            for (int b0 = 0, base = 0; b0 < bins; b0 += 1024) {
                const int b = b0 + i;
                total = 0;
                if (b < bins)
                    for (int w = 0; w < 32; ++w)
                        total += count[w * bins + b];
                int incl = total;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o)
                        incl += up;
                }
                if (lane == 31)
                    sums[warp] = incl;
                __syncthreads();
                int start = base;
                for (int w = 0; w < 32; ++w) {
                    if (w < warp)
                        start += sums[w];
                    base += sums[w];
                }
                start += incl - total;
                if (b < bins) {
                    offsets[b] = start;   // bin R's start is offsets[R]
                    for (int w = 0; w < 32; ++w) {
                        const int n = count[w * bins + b];
                        count[w * bins + b] = start;
                        start += n;
                    }
                }
                __syncthreads();
            }
        }
    }
}

__global__ void __launch_bounds__(128) down_kernel(const LoraArgs l, const uint16_t *__restrict__ x, int64_t xs,
                                                   const uint16_t *__restrict__ W, int C, bool scaled,
                                                   float *__restrict__ v)
{
    const int64_t i = blockIdx.x;
    const int a = adapter_of(l.offsets, l.R, i), t = l.order[i];
    if (a >= l.R || t < 0 || t >= l.T)
        return;
    const int rank = rank_of(l, a), lane = threadIdx.x & 31;
    for (int j = threadIdx.x >> 5; j < l.r; j += 4) {
        float s = 0.0f;
        if (j < rank)
            for (int c = lane; c < C; c += 32)
                s += bf(x[t * xs + c]) * bf(W[((int64_t)a * l.r + j) * C + c]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0)
            v[i * l.r + j] = scaled ? s * l.scales[a] : s;
    }
}

__global__ void __launch_bounds__(128) up_kernel(const LoraArgs l, const float *__restrict__ v,
                                                 const uint16_t *__restrict__ W, int C, bool scaled,
                                                 const uint16_t *base, int64_t bs, uint16_t *out, int64_t os)
{
    const int64_t i = blockIdx.x;
    const int a = adapter_of(l.offsets, l.R, i), t = l.order[i];
    if (t < 0 || t >= l.T || (a >= l.R && base == out))
        return;
    const int rank = a < l.R ? rank_of(l, a) : 0;
    const float f = scaled && a < l.R ? l.scales[a] : 1.0f;
    for (int c = threadIdx.x; c < C; c += 128) {
        float s = 0.0f;
        for (int j = 0; j < rank; ++j)
            s += v[i * l.r + j] * bf(W[((int64_t)a * l.r + j) * C + c]);
        const float y = base ? bf(base[t * bs + c]) : 0.0f;
        out[t * os + c] = to_bf(rank ? y + f * s : y);
    }
}

__global__ void __launch_bounds__(128) grad_kernel(const LoraArgs l, const float *__restrict__ p,
                                                   const uint16_t *__restrict__ x, int64_t xs, int C, bool scaled,
                                                   uint16_t *__restrict__ G)
{
    const int a = blockIdx.y, c = blockIdx.x * 128 + threadIdx.x;
    if (c >= C)
        return;
    const int rank = rank_of(l, a);
    const int64_t lo = max(l.offsets[a], 0), hi = min((int64_t)l.offsets[a + 1], l.T);
    const float f = scaled ? l.scales[a] : 1.0f;
    for (int j0 = 0; j0 < l.r; j0 += 16) {
        float s[16] = {};
        for (int64_t i = lo; i < hi; ++i) {
            const int t = l.order[i];
            if (t < 0 || t >= l.T)
                continue;
            const float xv = bf(x[t * xs + c]);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j0 + j < rank)
                    s[j] += p[i * l.r + j0 + j] * xv;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (j0 + j < l.r)
                G[((int64_t)a * l.r + j0 + j) * C + c] = to_bf(f * s[j]);
    }
}

}  // namespace

int64_t lora_ws_floats(int64_t, int) { return 0; }

cudaError_t launch_lora_plan(const int32_t *ids, int64_t T, int R, int32_t *order, int32_t *offsets, cudaStream_t st)
{
    const int smem = (32 * (R + 1) + 32) * (int)sizeof(int);
    if (smem > 48 * 1024) {
        const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(lora_plan_kernel),
                                                  (32 * (1024 + 1) + 32) * (int)sizeof(int));
        if (e != cudaSuccess)
            return e;
    }
    lora_plan_kernel<<<1, 1024, smem, st>>>(ids, (int)T, R, order, offsets);
    return cudaGetLastError();
}

cudaError_t launch_lora_down(const LoraArgs &l, const uint16_t *x, int64_t xs, const uint16_t *W, int C, bool scaled,
                             float *v, float *, int, cudaStream_t st)
{
    down_kernel<<<(unsigned)l.T, 128, 0, st>>>(l, x, xs, W, C, scaled, v);
    return cudaGetLastError();
}

cudaError_t launch_lora_up(const LoraArgs &l, const float *v, const uint16_t *W, int C, bool scaled,
                           const uint16_t *base, int64_t bs, uint16_t *out, int64_t os, float *, int, cudaStream_t st)
{
    up_kernel<<<(unsigned)l.T, 128, 0, st>>>(l, v, W, C, scaled, base, bs, out, os);
    return cudaGetLastError();
}

cudaError_t launch_lora_grad(const LoraArgs &l, const float *p, const uint16_t *x, int64_t xs, int C, bool scaled,
                             uint16_t *G, float *, int, cudaStream_t st)
{
    grad_kernel<<<dim3((C + 127) / 128, l.R), 128, 0, st>>>(l, p, x, xs, C, scaled, G);
    return cudaGetLastError();
}

}  // namespace gemmar

// moe_route.cu -- which experts a token goes to, and with which weights (moe_route).
//
//   l[t,e] = sum_h x[t,h] w[e,h];   p = softmax(l) or sigmoid(l);   the k largest of p + bias
//
// For few tokens it reads the router once and is bound by latency and, from some tens of
// tokens on, by fp32 FMAs.  A CTA computes the logits of a few tokens and experts with all
// its threads along h; the CTA that finishes a group of tokens last chooses for them, a warp
// per token, so that no second launch is needed.
//
// The order of two experts whose scores agree to fp32's rounding would depend on how the
// sums are split.  Such tokens are decided in 64 bits: the logits in question are summed
// again in double (a few microseconds, for about one token in a thousand).
#include <algorithm>

#include "e4m3_encode.cuh"
#include "kernels.h"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 8;        // tokens of a group: one warp chooses for each
static_assert(kTokens == kWarps, "a warp per token");

// 8 values of a row of the router
template <bool BF>
__device__ __forceinline__ void load8(const void *row, int h, float (&v)[8])
{
    if (BF) {
        const uint4 r = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + h));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + h);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

__device__ __forceinline__ const void *router_row(const RouteArgs &a, int e)
{
    return static_cast<const char *>(a.w) + (int64_t)e * a.H * (a.w_bf16 ? 2 : 4);
}

// a before b: the larger score, the lower number where they are equal
__device__ __forceinline__ bool before(float sa, int ea, float sb, int eb) { return sa > sb || (sa == sb && ea < eb); }
__device__ __forceinline__ bool before(double sa, int ea, double sb, int eb) { return sa > sb || (sa == sb && ea < eb); }

// The warp's best of (score, expert); lanes without one pass expert -1.
template <typename T>
__device__ __forceinline__ void best_of_warp(T &s, int &e)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const T os = __shfl_xor_sync(0xffffffffu, s, d);
        const int oe = __shfl_xor_sync(0xffffffffu, e, d);
        if (oe >= 0 && (e < 0 || before(os, oe, s, e))) {
            s = os;
            e = oe;
        }
    }
}

// A score an expert can be chosen with: not NaN, not -inf.
template <typename T>
__device__ __forceinline__ bool eligible(T s)
{
    return s > -INFINITY;
}

// x[t] . w[e] in double by the whole warp
__device__ double logit64(const RouteArgs &a, int t, int e)
{
    const int lane = threadIdx.x & 31;
    const uint16_t *x = a.x + (int64_t)t * a.xs;
    const void *w = router_row(a, e);
    double s = 0.0;
    for (int h = lane * 8; h < a.H; h += 256) {
        float xv[8], wv[8];
        load8<true>(x, h, xv);
        if (a.w_bf16)
            load8<true>(w, h, wv);
        else
            load8<false>(w, h, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s = fma((double)xv[i], (double)wv[i], s);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

// One warp chooses token t's experts.  score: [E] in shared memory, the warp's own, holding the
// logits; overwritten.  PER: experts of a lane (E <= 32 PER), lane + 32 i.
template <int PER>
__device__ void choose(const RouteArgs &a, int t, float *score)
{
    const int lane = threadIdx.x & 31;
    const bool soft = a.score == 0;
    float l[PER], sel[PER];
    float top = -INFINITY, big = 0.0f;   // largest logit, largest size of one
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        l[i] = e < a.E ? score[e] : -INFINITY;
        top = fmaxf(top, l[i]);          // skips NaN
        if (fabsf(l[i]) < INFINITY)
            big = fmaxf(big, fabsf(l[i]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
    }
    float sum = 0.0f;
    if (soft) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float x = l[i] - top;   // NaN where both are infinite
            l[i] = l[i] == top ? 1.0f : expf(x);
            if (l[i] >= 0.0f)
                sum += l[i];              // a NaN logit is no expert's
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        const float p = soft ? l[i] / sum : 1.0f / (1.0f + expf(-l[i]));
        sel[i] = -INFINITY;
        if (e < a.E) {
            sel[i] = p + (a.bias ? __ldg(a.bias + e) : 0.0f);
            score[e] = p;                 // the weight, once chosen
        }
        if (!(sel[i] == sel[i]))
            sel[i] = -INFINITY;
    }
    // how far fp32's rounding may move a score: the logits' sums to 2^-20 of the largest
    // logit (twenty times the spread of such sums), the rest to a few units in the last place
    const float peak = soft ? 1.0f / sum : 1.0f;
    const float tol = 0x1p-20f * big * (soft ? peak : 0.25f) + 0x1p-21f * peak;
    // the chosen, and whether neighbours in the order are too close to tell in fp32
    int32_t *ids = a.ids + (int64_t)t * a.k;
    float *weights = a.weights + (int64_t)t * a.k;
    bool close = false;
    int mine = -1;                        // lane j keeps the j-th choice (k <= 16)
    float last = INFINITY;
    auto pick = [&](float &s, int &e) {
        s = -INFINITY;
        e = -1;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (eligible(sel[i]) && (e < 0 || before(sel[i], lane + 32 * i, s, e))) {
                s = sel[i];
                e = lane + 32 * i;
            }
        best_of_warp(s, e);
    };
    auto take = [&](int e) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (e == lane + 32 * i)
                sel[i] = -INFINITY;
    };
    float cut = -INFINITY;                // the last chosen score
    int chosen = 0;
    float kept[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        kept[i] = sel[i];
    for (int j = 0; j <= a.k; ++j) {      // one past the last, to see how near it is
        float s;
        int e;
        pick(s, e);
        if (e < 0)
            break;
        close = close || last - s <= tol + 0x1p-21f * fabsf(s);
        last = s;
        if (j == a.k)
            break;
        take(e);
        cut = s;
        ++chosen;
        if (lane == j)
            mine = e;
    }
    if (close && eligible(cut)) {
        // decide in double: every expert that may be among the chosen
        const float floor_ = cut - 2.0f * (tol + 0x1p-21f * fabsf(cut));
        double dsum = 1.0;
        if (soft && a.bias != nullptr) {
            dsum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < a.E && l[i] >= 0.0f)
                    dsum += (double)l[i];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                dsum += __shfl_xor_sync(0xffffffffu, dsum, d);
        }
        double dsel[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            dsel[i] = -INFINITY;
            unsigned todo = __ballot_sync(0xffffffffu, eligible(kept[i]) && kept[i] >= floor_);
            while (todo) {
                const int who = __ffs(todo) - 1, e = who + 32 * i;
                todo &= todo - 1;
                const double x = big == 0.0f ? 0.0 : logit64(a, t, e);   // a padded row's logits are exact
                if (lane == who) {
                    const double b = a.bias ? (double)__ldg(a.bias + e) : 0.0;
                    // an infinite logit (its score is then exact in fp32) stays as it was
                    if (!(x > -INFINITY && x < INFINITY))
                        dsel[i] = (double)kept[i];
                    else if (!soft)
                        dsel[i] = 1.0 / (1.0 + exp(-x)) + b;
                    else
                        dsel[i] = a.bias ? exp(x - (double)top) / dsum + b : exp(x - (double)top);
                }
            }
        }
        mine = -1;
        for (int j = 0; j < chosen; ++j) {
            double s = -INFINITY;
            int e = -1;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (eligible(dsel[i]) && (e < 0 || before(dsel[i], lane + 32 * i, s, e))) {
                    s = dsel[i];
                    e = lane + 32 * i;
                }
            best_of_warp(s, e);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (e == lane + 32 * i)
                    dsel[i] = -INFINITY;
            if (lane == j)
                mine = e;
        }
    }
    __syncwarp();
    float w = mine >= 0 ? score[mine] : 0.0f, all = w;
    if (a.renorm) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            all += __shfl_xor_sync(0xffffffffu, all, d);
        w = all > 0.0f ? w / all : (mine >= 0 ? w : 0.0f);
    }
    if (lane < a.k) {
        ids[lane] = mine;
        weights[lane] = mine >= 0 ? w * a.factor : 0.0f;
    }
}

// grid: (experts / EB, tokens / kTokens); logits fp32 [T,E]; done: one counter per token group,
// zero before and after.
template <int TB, int EB, bool BF>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a, float *logits, uint32_t *done)
{
    __shared__ float part[kWarps][TB * EB];
    extern __shared__ float scores[];   // [kWarps][E]
    __shared__ bool chooses;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.x * EB;
    const int group0 = blockIdx.y * kTokens, group1 = min(group0 + kTokens, a.T);
    for (int t0 = group0; t0 < group1; t0 += TB) {
        float acc[TB * EB] = {};
        for (int h = threadIdx.x * 8; h < a.H; h += kThreads * 8) {
            float x[TB][8];
#pragma unroll
            for (int i = 0; i < TB; ++i)
                load8<true>(a.x + (int64_t)min(t0 + i, group1 - 1) * a.xs, h, x[i]);
#pragma unroll
            for (int j = 0; j < EB; ++j) {
                float w[8];
                load8<BF>(router_row(a, min(e0 + j, a.E - 1)), h, w);
#pragma unroll
                for (int i = 0; i < TB; ++i)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[i * EB + j] = fmaf(x[i][c], w[c], acc[i * EB + j]);
            }
        }
#pragma unroll
        for (int i = 0; i < TB * EB; ++i) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            if (lane == 0)
                part[warp][i] = acc[i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < TB * EB; i += kThreads) {
            float s = part[0][i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                s += part[w][i];
            const int t = t0 + i / EB, e = e0 + i % EB;
            if (t < group1 && e < a.E)
                __stcg(logits + (int64_t)t * a.E + e, s);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        __threadfence();
        chooses = atomicAdd(done + blockIdx.y, 1u) == gridDim.x - 1;
        if (chooses) {
            __threadfence();
            done[blockIdx.y] = 0;
        }
    }
    __syncthreads();
    if (!chooses)
        return;
    const int t = group0 + warp;
    if (t >= a.T)
        return;
    float *score = scores + warp * a.E;
    for (int e = lane; e < a.E; e += 32)
        score[e] = __ldcg(logits + (int64_t)t * a.E + e);
    __syncwarp();
    if (a.E <= 64)
        choose<2>(a, t, score);
    else if (a.E <= 256)
        choose<8>(a, t, score);
    else
        choose<32>(a, t, score);
}

template <int TB, int EB, bool BF>
cudaError_t launch_typed(const RouteArgs &a, float *ws, uint32_t *counters, cudaStream_t st)
{
    const dim3 grid((a.E + EB - 1) / EB, (a.T + kTokens - 1) / kTokens);
    route_kernel<TB, EB, BF><<<grid, kThreads, sizeof(float) * kWarps * a.E, st>>>(a, ws, counters);
    return cudaGetLastError();
}

}  // namespace

int64_t route_ws_floats(const RouteArgs &a) { return (int64_t)a.T * a.E; }

cudaError_t launch_route(const RouteArgs &a, float *ws, uint32_t *counters, cudaStream_t st)
{
    if (a.T == 1)
        return a.w_bf16 ? launch_typed<1, 1, true>(a, ws, counters, st) : launch_typed<1, 1, false>(a, ws, counters, st);
    return a.w_bf16 ? launch_typed<4, 4, true>(a, ws, counters, st) : launch_typed<4, 4, false>(a, ws, counters, st);
}

}  // namespace gemmar

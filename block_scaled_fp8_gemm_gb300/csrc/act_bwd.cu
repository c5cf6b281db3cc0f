// act_bwd.cu -- the backward pass of what follows a block-scaled product
// (gemm_blockscale_act_bwd): dz = dout act'(z), or both halves of a gated one, as bf16 rows
// and as the e4m3 codes that the product with the transposed weight takes, and the bias's
// gradient, the sums of dz over the rows.
//
// HBM-bound: about 20 flops per element of z against 5 to 8 bytes.  Sixteen lanes take a row's
// group of 128 columns, 8 each, so that a group's maximum is four shuffles; a thread keeps its
// columns and walks down the rows of its CTA's share, so that a column's sum stays in
// registers until the end.  Shares are summed by a second kernel in their order.
// Gated silu of 4096 x 2048 to rows and codes 17.6 us (5.7 TB/s), 16384 rows 67 us (6.0).
#include <algorithm>

#include "activation.cuh"
#include "e4m3_encode.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kGroups = 4;                       // groups of 128 columns side by side in a CTA
constexpr int kLanes = 16;                       // rows of threads
constexpr int kRowThreads = kGroups * kLanes;
constexpr int kRows = 2;                         // rows a CTA takes at a time
constexpr int kThreads = kRowThreads * kRows;

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    return make_uint4(bf16x2_from_f32(x[0], x[1]), bf16x2_from_f32(x[2], x[3]), bf16x2_from_f32(x[4], x[5]),
                      bf16x2_from_f32(x[6], x[7]));
}

// codes and scale of a group's 8 columns; the 16 lanes of the group call together
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float *scale, bool first)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(x[i]));   // skips NaN
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float s = __fdiv_rn(m, 448.0f);
    if (first)
        *scale = s;
    uint32_t w[2];
    Enc(s).codes(x, w);
    return make_uint2(w[0], w[1]);
}

struct Share {
    int strips, shares;
    int64_t rows;   // of a share
};

inline Share share_out(int64_t M, int N, int num_sms)
{
    Share s;
    s.strips = (N / 128 + kGroups - 1) / kGroups;
    // one wave of seven CTAs per SM, which its registers hold, and at least 16 rows to a CTA (gated, N =
    // 2048: 4096 rows, where the 16 count, 17.4 us, four CTAs of twice the rows at a time 20.9, two waves of
    // those 19.8; 16384 rows 67 us, with eight CTAs, the eighth in a wave of its own, 83)
    const int64_t want = std::max<int64_t>(1, (int64_t)num_sms * 7 / s.strips);
    s.rows = (M + want - 1) / want;
    s.rows = s.rows < 16 ? 16 : (s.rows + kRows - 1) / kRows * kRows;
    s.shares = (int)((M + s.rows - 1) / s.rows);
    return s;
}

template <int ACT, bool GATED, bool BF>
__global__ void __launch_bounds__(kThreads, 7) act_bwd_kernel(const ActBwdArgs a, const Share sh, float *ws)
{
    const int lane = threadIdx.x % kLanes, group = (threadIdx.x / kLanes) % kGroups, r0 = threadIdx.x / kRowThreads;
    const int g = blockIdx.x * kGroups + group;
    const bool inside = g < a.N / 128;
    const int col = (inside ? g : 0) * 128 + lane * 8;
    const int P = GATED ? 2 * a.N : a.N;
    const int64_t first = (int64_t)blockIdx.y * sh.rows, end = min(first + sh.rows, a.M);
    float sum0[8] = {}, sum1[8] = {};
    // a row ahead of its use: dout in one or two units of 16 bytes, and z
    uint4 raw_d[BF ? 1 : 2], raw_z[GATED ? 2 : 1];
    auto fetch = [&](int64_t base) {
        const int64_t mm = inside && base + r0 < end ? base + r0 : first;
        const char *dp = static_cast<const char *>(a.dout) + (mm * a.ds + col) * (BF ? 2 : 4);
#pragma unroll
        for (int i = 0; i < (BF ? 1 : 2); ++i)
            raw_d[i] = __ldcs(reinterpret_cast<const uint4 *>(dp) + i);
        const uint16_t *zp = a.z + mm * P + col;
#pragma unroll
        for (int i = 0; i < (GATED ? 2 : 1); ++i)
            raw_z[i] = __ldcs(reinterpret_cast<const uint4 *>(zp + (int64_t)i * a.N));
    };
    fetch(first);
    // every thread of a warp makes every step: a group's lanes meet in shuffles
    for (int64_t base = first; base < end; base += kRows) {
        const int64_t m = base + r0;
        const bool live = inside && m < end;
        const int64_t mm = live ? m : first;
        float d[8], z0[8], z1[8], v0[8], v1[8];
        if constexpr (BF) {
            unpack8(raw_d[0], d);
        } else {
            const uint32_t w[8] = {raw_d[0].x, raw_d[0].y, raw_d[0].z, raw_d[0].w, raw_d[1].x, raw_d[1].y, raw_d[1].z, raw_d[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] = __uint_as_float(w[i]);
        }
        unpack8(raw_z[0], z0);
        if constexpr (GATED)
            unpack8(raw_z[1], z1);
        fetch(base + kRows);
        // two columns an instruction where there is one for two
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float va, vb, sa, sb;
            act_slope<ACT>(z0[i], va, sa);
            act_slope<ACT>(z0[i + 1], vb, sb);
            float2 g = make_float2(d[i], d[i + 1]);
            if constexpr (GATED) {
                const float2 u = mul2(d[i], d[i + 1], va, vb);
                v1[i] = u.x;
                v1[i + 1] = u.y;
                g = mul2(g.x, g.y, z1[i], z1[i + 1]);
            }
            g = mul2(g.x, g.y, sa, sb);
            v0[i] = g.x;
            v0[i + 1] = g.y;
        }
        if (a.dbias != nullptr && live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum0[i] += v0[i];
                if constexpr (GATED)
                    sum1[i] += v1[i];
            }
        }
        if (live && a.dz != nullptr) {
            uint16_t *o = a.dz + m * P + col;
            __stcs(reinterpret_cast<uint4 *>(o), pack8(v0));
            if (GATED)
                __stcs(reinterpret_cast<uint4 *>(o + a.N), pack8(v1));
        }
        if (a.q != nullptr) {
            float *s = a.scales + mm * (P / 128) + col / 128;
            uint8_t *o = a.q + mm * P + col;
            const bool writes = live && lane == 0;
            const uint2 c0 = encode8(v0, s, writes);
            if (live)
                __stcs(reinterpret_cast<uint2 *>(o), c0);
            if (GATED) {
                const uint2 c1 = encode8(v1, s + a.N / 128, writes);
                if (live)
                    __stcs(reinterpret_cast<uint2 *>(o + a.N), c1);
            }
        }
    }
    if (a.dbias == nullptr)
        return;
    grid_launch_next();
    // the CTA's rows of threads in their order, then the share's sums for the second kernel
    __shared__ float part[kRows][kRowThreads][GATED ? 16 : 8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        part[r0][threadIdx.x % kRowThreads][i] = sum0[i];
        if constexpr (GATED)
            part[r0][threadIdx.x % kRowThreads][8 + i] = sum1[i];
    }
    __syncthreads();
    if (r0 == 0 && inside) {
        float *o = (sh.shares > 1 ? ws + (int64_t)blockIdx.y * P : a.dbias) + col;
#pragma unroll
        for (int i = 0; i < (GATED ? 16 : 8); ++i) {
            float s = part[0][threadIdx.x][i];
#pragma unroll
            for (int r = 1; r < kRows; ++r)
                s += part[r][threadIdx.x][i];
            o[i < 8 ? i : a.N + i - 8] = s;
        }
    }
}

// Sums of the shares: a column's in order, eight partial chains of every eighth share.
__global__ void __launch_bounds__(256) act_bwd_sum_kernel(const float *ws, int shares, int P, float *dbias)
{
    const int c = blockIdx.x * 32 + threadIdx.x % 32, r = threadIdx.x / 32;
    float s = 0.0f;
    grid_wait();
#pragma unroll 4
    for (int i = r; i < shares; i += 8)
        s += ld_after_f32(ws + (int64_t)i * P + c);
    __shared__ float part[8][32];
    part[r][threadIdx.x % 32] = s;
    __syncthreads();
    if (r == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            s += part[i][threadIdx.x];
        dbias[c] = s;
    }
}

template <int ACT>
void launch_typed(const ActBwdArgs &a, const Share &sh, float *ws, cudaStream_t st)
{
    const dim3 grid(sh.strips, sh.shares);
    void (*const kernels[2][2])(const ActBwdArgs, const Share, float *) = {
        {act_bwd_kernel<ACT, false, false>, act_bwd_kernel<ACT, false, true>},
        {act_bwd_kernel<ACT, true, false>, act_bwd_kernel<ACT, true, true>}};
    kernels[a.gated][a.d_bf16]<<<grid, kThreads, 0, st>>>(a, sh, ws);
}

}  // namespace

int64_t act_bwd_ws_floats(int64_t M, int N, int gated, int num_sms)
{
    return (int64_t)share_out(M, N, num_sms).shares * N * (gated ? 2 : 1);
}

cudaError_t launch_act_bwd(const ActBwdArgs &a, float *ws, int num_sms, cudaStream_t st)
{
    const Share sh = share_out(a.M, a.N, num_sms);
    switch (a.act) {
    case ACT_RELU: launch_typed<ACT_RELU>(a, sh, ws, st); break;
    case ACT_SILU: launch_typed<ACT_SILU>(a, sh, ws, st); break;
    case ACT_GELU: launch_typed<ACT_GELU>(a, sh, ws, st); break;
    case ACT_GELU_TANH: launch_typed<ACT_GELU_TANH>(a, sh, ws, st); break;
    default: launch_typed<ACT_NONE>(a, sh, ws, st); break;
    }
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.dbias != nullptr && sh.shares > 1) {
        const int P = a.gated ? 2 * a.N : a.N;
        e = launch(act_bwd_sum_kernel, dim3(P / 32), 256, 0, 1, true, st, static_cast<const float *>(ws), (int)sh.shares, P, a.dbias);
    }
    return e;
}

}  // namespace gemmar

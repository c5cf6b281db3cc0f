// residual.cu -- a block's output joins the residual stream: norms before and
// after, gate, residual scale, and the next block's input as bf16 rows or as
// e4m3 codes with 1x128 scales (norm_gate_residual), and its backward pass.
//
// Both are HBM-bound: about 14 and 36 flops per element against 6 to 16 bytes, each
// input read and each output written once.  A persistent CTA takes a row at a
// time, a thread keeping the same 8-column chunks (16 bytes of bf16) of every
// row, so that what a row needs from another thread is only its sums.  Rows
// ahead are copied to shared memory with cp.async into slots that only the
// copying thread reads: no barrier guards them, and a thread waits for nothing
// but its own copies.
#include <cuda_bf16.h>

#include "e4m3_encode.cuh"
#include "kernels.h"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kMaxSmem = 231424;   // of the 232448 a CTA may have; the rest is static

__device__ __forceinline__ void unpack8(const uint4 &w, float (&v)[8])
{
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}

// Eight consecutive fp32 (weights: re-read every row, from L1) or bf16.
__device__ __forceinline__ void ldg8(const float *p, float (&v)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void ldg8(const uint16_t *p, float (&v)[8])
{
    unpack8(__ldg(reinterpret_cast<const uint4 *>(p)), v);
}

template <bool BF>
__device__ __forceinline__ void store8(void *p, int64_t i, const float (&v)[8])
{
    if constexpr (BF) {
        uint4 w;
        w.x = bf16x2_from_f32(v[0], v[1]);
        w.y = bf16x2_from_f32(v[2], v[3]);
        w.z = bf16x2_from_f32(v[4], v[5]);
        w.w = bf16x2_from_f32(v[6], v[7]);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = w;
    } else {
        float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        f[0] = make_float4(v[0], v[1], v[2], v[3]);
        f[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// A thread's slots of one matrix in one stage: J chunks of one (bf16) or two
// (fp32) 16-byte units, unit u of thread t at (u * T + t) * 16, so that a warp's
// accesses are contiguous.
template <bool BF>
__device__ __forceinline__ void fetch8(uint32_t slot, int T, const void *row, int col)
{
    const char *src = static_cast<const char *>(row) + (int64_t)col * (BF ? 2 : 4);
    cp_async_cg16(slot, src);
    if constexpr (!BF)
        cp_async_cg16(slot + T * 16, src + 16);
}

template <bool BF>
__device__ __forceinline__ void slot8(uint32_t slot, int T, float (&v)[8])
{
    const uint4 a = ld_shared_v4(slot);
    if constexpr (BF) {
        unpack8(a, v);
    } else {
        const uint4 b = ld_shared_v4(slot + T * 16);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    }
}

// All but the newest stages - 1 groups of this thread's copies have landed.
__device__ __forceinline__ void wait_stage(int stages)
{
    if (stages == 1)
        cp_async_wait<0>();
    else if (stages == 2)
        cp_async_wait<1>();
    else if (stages == 3)
        cp_async_wait<2>();
    else
        cp_async_wait<3>();
}
constexpr int kMaxStages = 4;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the CTA, the same bits in every thread.  One barrier: two buffers take
// turns, so a warp that is a sum ahead of another writes the one not being read.
__device__ __forceinline__ float cta_sum(float v, float (&bufs)[2][32], int &turn)
{
    v = warp_sum(v);
    const int lane = threadIdx.x & 31;
    float *red = bufs[turn];
    turn ^= 1;
    if (lane == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < (int)(blockDim.x >> 5) ? red[lane] : 0.0f);
}

// ---------------------------------------------------------------- forward

template <int J, bool YB, bool HB>
__global__ void __launch_bounds__(J == 1 ? 1024 : 512, J == 2 ? 2 : 1) norm_kernel(const NormArgs a, int stages)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float red[2][32];
    const int T = blockDim.x, t = threadIdx.x, N = a.N;
    const bool token = a.gate != nullptr && a.gs != 0;
    constexpr int UY = J * (YB ? 1 : 2), UH = J * (HB ? 1 : 2);
    const uint32_t unit = T * 16;
    const uint32_t stage_bytes = (UY + UH + (token ? J : 0)) * unit;
    const uint32_t base = smem_u32(smem_raw) + t * 16;
    const float inv_n = 1.0f / N;

    auto fetch = [&](int64_t m, uint32_t slot) {
        const char *y = static_cast<const char *>(a.y) + m * a.ys * (YB ? 2 : 4);
        const char *h = static_cast<const char *>(a.h) + m * a.hs * (HB ? 2 : 4);
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const int col = (c * T + t) * 8;
            if (col < N) {
                fetch8<YB>(slot + c * (UY / J) * unit, T, y, col);
                fetch8<HB>(slot + (UY + c * (UH / J)) * unit, T, h, col);
                if (token)
                    fetch8<true>(slot + (UY + UH + c) * unit, T, a.gate + m * a.gs, col);
            }
        }
    };

    int64_t ahead = blockIdx.x;   // next row to fetch
    int put = 0, get = 0, turn = 0;
    for (int s = 0; s < stages - 1; ++s, ahead += gridDim.x) {
        if (ahead < a.M)
            fetch(ahead, base + put * stage_bytes);
        cp_async_commit();
        if (++put == stages)
            put = 0;
    }
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, ahead += gridDim.x) {
        // the slot of the row before this one is free: this thread has read it
        if (ahead < a.M)
            fetch(ahead, base + put * stage_bytes);
        cp_async_commit();
        if (++put == stages)
            put = 0;
        wait_stage(stages);
        const uint32_t slot = base + get * stage_bytes;
        if (++get == stages)
            get = 0;

        float v[J][8];   // y, then t
        float r1 = 1.0f, r2 = 1.0f;
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < J; ++c) {
            if ((c * T + t) * 8 < N) {
                slot8<YB>(slot + c * (UY / J) * unit, T, v[c]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[c][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ss = fmaf(v[c][j], v[c][j], ss);
        }
        if (a.w1)
            r1 = rsqrtf(cta_sum(ss, red, turn) * inv_n + a.eps);
        ss = 0.0f;
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const int col = (c * T + t) * 8;
            if (col < N) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[c][j] *= r1;
                if (a.w1) {
                    ldg8(a.w1 + col, f);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[c][j] *= f[j];
                }
                if (a.gate) {
                    if (token)
                        slot8<true>(slot + (UY + UH + c) * unit, T, f);
                    else
                        ldg8(a.gate + col, f);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[c][j] *= f[j];
                }
                slot8<HB>(slot + (UY + c * (UH / J)) * unit, T, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[c][j] = fmaf(a.alpha, f[j], a.beta * v[c][j]);
                    ss = fmaf(v[c][j], v[c][j], ss);
                }
                store8<HB>(a.t, m * N + col, v[c]);
            }
        }
        if (a.w2)
            r2 = rsqrtf(cta_sum(ss, red, turn) * inv_n + a.eps);
        if (a.rstd && t == 0)
            *reinterpret_cast<float2 *>(a.rstd + 2 * m) = make_float2(r1, r2);
        if (a.u == nullptr && a.q == nullptr)
            continue;
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const int col = (c * T + t) * 8;
            float amax = 0.0f;
            if (col < N) {
                float f[8];
                ldg8(a.w2 + col, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[c][j] = v[c][j] * r2 * f[j];
                    amax = fmaxf(amax, fabsf(v[c][j]));
                }
                if (a.u)
                    store8<true>(a.u, m * N + col, v[c]);
            }
            if (a.q) {
                // a group's 128 columns are 16 neighbouring lanes (N % 128 == 0)
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
                if (col < N) {
                    const float sc = __fdiv_rn(amax, 448.0f);
                    const Enc enc(sc);
                    uint2 w;
                    w.x = enc(v[c][0], v[c][1], v[c][2], v[c][3]);
                    w.y = enc(v[c][4], v[c][5], v[c][6], v[c][7]);
                    *reinterpret_cast<uint2 *>(a.q + m * N + col) = w;
                    if ((t & 15) == 0)
                        a.scales[m * (N / 128) + col / 128] = sc;
                }
            }
        }
    }
}

// ---------------------------------------------------------------- backward

// One pass over the row forms four sums, from which both projections follow:
// with dv = du w2, c = beta g w1, n = y r1, t = alpha h + c n and d = dt + r2 dv - k t,
// k = r2^3 mean(dv t),
//   mean(c n d) = mean(c n dt) + r2 mean(c n dv) - k mean(c n t).
// The second pass recomputes n, t, dv from shared memory and writes dy, dh (and a
// token's dgate).  The sums over rows, s1 = sum n d (times a token's gate) and
// s2 = sum du t r2, stay in the thread's registers over all the CTA's rows and
// leave as one part per CTA, summed in the CTAs' order by norm_bwd_sum_kernel.
template <int J, bool YB, bool HB>
__global__ void __launch_bounds__(J == 1 ? 256 : 512, J == 1 ? 3 : 1)
    norm_bwd_kernel(const NormBwdArgs a, float *__restrict__ ws, int stages, int gate_staged)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float4 red[2][32];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, N = a.N;
    const bool token = a.gate != nullptr && a.gs != 0;
    const bool pre = a.w2 != nullptr, post = a.w1 != nullptr;
    constexpr int UY = J * (YB ? 1 : 2), UH = J * (HB ? 1 : 2);
    constexpr int kDu = UY + UH, kDt = kDu + J, kGate = kDt + UH;
    const uint32_t unit = T * 16;
    const uint32_t stage_bytes = (kGate + (gate_staged ? J : 0)) * unit;
    const uint32_t base = smem_u32(smem_raw) + t * 16;
    const float inv_n = 1.0f / N;
    constexpr bool kKeepWeights = J <= 2;   // more chunks would not fit the registers

    auto fetch = [&](int64_t m, uint32_t slot) {
        const char *y = static_cast<const char *>(a.y) + m * a.ys * (YB ? 2 : 4);
        const char *h = static_cast<const char *>(a.h) + m * a.hs * (HB ? 2 : 4);
        const char *dt = static_cast<const char *>(a.dt) + m * a.dts * (HB ? 2 : 4);
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const int col = (c * T + t) * 8;
            if (col < N) {
                fetch8<YB>(slot + c * (UY / J) * unit, T, y, col);
                fetch8<HB>(slot + (UY + c * (UH / J)) * unit, T, h, col);
                if (pre)
                    fetch8<true>(slot + (kDu + c) * unit, T, a.du + m * a.dus, col);
                if (a.dt)
                    fetch8<HB>(slot + (kDt + c * (UH / J)) * unit, T, dt, col);
                if (gate_staged)
                    fetch8<true>(slot + (kGate + c) * unit, T, a.gate + m * a.gs, col);
            }
        }
    };
    // beta w1 (times the gate when it is one row), and w2
    auto weights = [&](int col, float (&cw)[8], float (&w2)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cw[j] = a.beta;
            w2[j] = 0.0f;
        }
        if (col >= N)
            return;
        float f[8];
        if (post) {
            ldg8(a.w1 + col, f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cw[j] *= f[j];
        }
        if (a.gate != nullptr && !token) {
            ldg8(a.gate + col, f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cw[j] *= f[j];
        }
        if (pre)
            ldg8(a.w2 + col, w2);
    };

    float s1[J][8], s2[J][8];
    float kw[kKeepWeights ? J : 1][8], kw2[kKeepWeights ? J : 1][8];
#pragma unroll
    for (int c = 0; c < J; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s1[c][j] = s2[c][j] = 0.0f;
        if constexpr (kKeepWeights)
            weights((c * T + t) * 8, kw[c], kw2[c]);
    }

    int64_t ahead = blockIdx.x;
    int put = 0, get = 0, turn = 0;
    for (int s = 0; s < stages - 1; ++s, ahead += gridDim.x) {
        if (ahead < a.M)
            fetch(ahead, base + put * stage_bytes);
        cp_async_commit();
        if (++put == stages)
            put = 0;
    }
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, ahead += gridDim.x) {
        if (ahead < a.M)
            fetch(ahead, base + put * stage_bytes);
        cp_async_commit();
        if (++put == stages)
            put = 0;
        const float2 rs = __ldg(reinterpret_cast<const float2 *>(a.rstd) + m);
        const float r1 = rs.x, r2 = rs.y;
        wait_stage(stages);
        const uint32_t slot = base + get * stage_bytes;
        if (++get == stages)
            get = 0;

        // n, t, du, c of chunk c
        auto load = [&](int c, float (&n)[8], float (&tt)[8], float (&du)[8], float (&cw)[8], float (&w2)[8],
                        float (&gt)[8]) {
            const int col = (c * T + t) * 8;
            if constexpr (kKeepWeights) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    cw[j] = kw[c][j];
                    w2[j] = kw2[c][j];
                }
            } else {
                weights(col, cw, w2);
            }
            slot8<YB>(slot + c * (UY / J) * unit, T, n);
            slot8<HB>(slot + (UY + c * (UH / J)) * unit, T, tt);
            if (pre)
                slot8<true>(slot + (kDu + c) * unit, T, du);
            if (token) {
                if (gate_staged)
                    slot8<true>(slot + (kGate + c) * unit, T, gt);
                else
                    ldg8(a.gate + m * a.gs + col, gt);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!pre)
                    du[j] = 0.0f;
                if (!token)
                    gt[j] = 1.0f;
                n[j] *= r1;
                tt[j] = fmaf(a.alpha, tt[j], cw[j] * gt[j] * n[j]);
            }
        };
        auto stream_grad = [&](int c, float (&dt)[8]) {
            if (a.dt) {
                slot8<HB>(slot + (kDt + c * (UH / J)) * unit, T, dt);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dt[j] = 0.0f;
            }
        };

        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < J; ++c) {
            if ((c * T + t) * 8 < N) {
                float n[8], tt[8], du[8], cw[8], w2[8], gt[8], dt[8];
                load(c, n, tt, du, cw, w2, gt);
                stream_grad(c, dt);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float dv = du[j] * w2[j], cn = cw[j] * gt[j] * n[j];
                    q.x = fmaf(dv, tt[j], q.x);
                    q.y = fmaf(cn, dt[j], q.y);
                    q.z = fmaf(cn, dv, q.z);
                    q.w = fmaf(cn, tt[j], q.w);
                }
            }
        }
        float k = 0.0f, mean1 = 0.0f;
        if (pre || post) {
            q.x = warp_sum(q.x);
            q.y = warp_sum(q.y);
            q.z = warp_sum(q.z);
            q.w = warp_sum(q.w);
            float4 *buf = red[turn];
            turn ^= 1;
            if (lane == 0)
                buf[t >> 5] = q;
            __syncthreads();
            // lane l: sum l & 3 over the warps l >> 2, + 8, ...
            float s = 0.0f;
            for (int w = lane >> 2; w < (T >> 5); w += 8)
                s += reinterpret_cast<const float *>(buf + w)[lane & 3];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            s *= inv_n;
            k = pre ? r2 * r2 * r2 * __shfl_sync(0xFFFFFFFFu, s, 0) : 0.0f;
            const float m_dt = __shfl_sync(0xFFFFFFFFu, s, 1), m_dv = __shfl_sync(0xFFFFFFFFu, s, 2),
                        m_t = __shfl_sync(0xFFFFFFFFu, s, 3);
            mean1 = post ? (pre ? fmaf(r2, m_dv, m_dt) - k * m_t : m_dt) : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < J; ++c) {
            const int col = (c * T + t) * 8;
            if (col < N) {
                float n[8], tt[8], du[8], cw[8], w2[8], gt[8], d[8], o[8];
                load(c, n, tt, du, cw, w2, gt);
                stream_grad(c, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (pre)
                        d[j] += r2 * (du[j] * w2[j]) - k * tt[j];
                    s1[c][j] = fmaf(n[j] * gt[j], d[j], s1[c][j]);
                    s2[c][j] = fmaf(du[j] * r2, tt[j], s2[c][j]);
                    o[j] = r1 * (cw[j] * gt[j] * d[j] - n[j] * mean1);
                }
                store8<YB>(a.dy, m * N + col, o);
                if (token && a.dgate) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j] = cw[j] * n[j] * d[j];
                    store8<true>(a.dgate, m * N + col, o);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[j] *= a.alpha;
                store8<HB>(a.dh, m * N + col, d);
            }
        }
    }
    float *part = ws + (int64_t)blockIdx.x * 2 * N;
#pragma unroll
    for (int c = 0; c < J; ++c) {
        const int col = (c * T + t) * 8;
        if (col < N) {
            store8<false>(part, col, s1[c]);
            store8<false>(part, N + col, s2[c]);
        }
    }
}

// The CTAs' parts in the order of the CTAs: eight threads a column, each a
// contiguous eighth of the parts.  s1 = sum n d (times a token's gate):
// dw1 = beta g s1 and dgate = beta w1 s1 for a gate row g.
__global__ void __launch_bounds__(256) norm_bwd_sum_kernel(const NormBwdArgs a, const float *__restrict__ ws, int parts)
{
    __shared__ float sums[2][8][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int n = blockIdx.x * 32 + lane;
    const int share = (parts + 7) / 8, lo = part * share, hi = min(lo + share, parts);
    float s1 = 0.0f, s2 = 0.0f;
    if (n < a.N) {
#pragma unroll 8
        for (int p = lo; p < hi; ++p) {
            s1 += ws[(int64_t)p * 2 * a.N + n];
            s2 += ws[(int64_t)p * 2 * a.N + a.N + n];
        }
    }
    sums[0][part][lane] = s1;
    sums[1][part][lane] = s2;
    __syncthreads();
    if (part != 0 || n >= a.N)
        return;
    for (int p = 1; p < 8; ++p) {
        s1 += sums[0][p][lane];
        s2 += sums[1][p][lane];
    }
    const bool row = a.gate && a.gs == 0;
    if (a.dw1)
        a.dw1[n] = a.beta * (row ? bf16_lo(a.gate[n]) : 1.0f) * s1;
    if (a.dw2)
        a.dw2[n] = s2;
    if (a.dgate && row)
        static_cast<float *>(a.dgate)[n] = a.beta * (a.w1 ? a.w1[n] : 1.0f) * s1;
}

// ---------------------------------------------------------------- launches

struct Shape {
    int threads, ctas_per_sm;
};

int round32(int v) { return (v + 31) / 32 * 32; }

// Chunks a thread: 1, 2 or 4, the fewest that keep a row in `most` threads.
int chunks(int N, int most1, int most2) { return N <= 8 * most1 ? 1 : N <= 16 * most2 ? 2 : 4; }

// Stages of the ring that fit a CTA's share of the SM's shared memory.
int ring_stages(int stage_bytes, int ctas_per_sm, int64_t rows)
{
    int s = (kMaxSmem / ctas_per_sm - 1024) / stage_bytes;
    if (ctas_per_sm == 1)
        s = kMaxSmem / stage_bytes;
    s = s < 1 ? 1 : s > kMaxStages ? kMaxStages : s;
    return rows < s ? (int)rows : s;
}

Shape bwd_shape(int N)
{
    const int J = chunks(N, 256, 512);
    const int threads = round32((N + 8 * J - 1) / (8 * J));
    return {threads, J == 1 ? (threads <= 64 ? 12 : 768 / threads) : 1};
}

int bwd_ctas(int64_t M, int N, int num_sms)
{
    // at least two rows a CTA, so that the parts never need more room than the rows themselves
    const int64_t most = (int64_t)num_sms * bwd_shape(N).ctas_per_sm, some = (M + 1) / 2;
    return (int)(some < most ? some : most);
}

template <int J, bool YB, bool HB>
cudaError_t run_norm(const NormArgs &a, int threads, int num_sms, cudaStream_t st)
{
    const int stage_bytes = (J * (YB ? 1 : 2) + J * (HB ? 1 : 2) + (a.gate && a.gs ? J : 0)) * threads * 16;
    int per_sm = J == 1 ? 1024 / threads : J == 2 ? 1024 / threads : 1;
    per_sm = per_sm > 16 ? 16 : per_sm;
    while (per_sm > 1 && stage_bytes * 2 > kMaxSmem / per_sm - 1024)
        --per_sm;
    const int64_t most = (int64_t)num_sms * per_sm;
    const int grid = (int)(a.M < most ? a.M : most);
    const int stages = ring_stages(stage_bytes, per_sm, (a.M + grid - 1) / grid);
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(norm_kernel<J, YB, HB>), kMaxSmem);
    if (e != cudaSuccess)
        return e;
    norm_kernel<J, YB, HB><<<grid, threads, stages * stage_bytes, st>>>(a, stages);
    return cudaGetLastError();
}

template <int J>
cudaError_t pick_norm(const NormArgs &a, int num_sms, cudaStream_t st)
{
    const int threads = round32((a.N + 8 * J - 1) / (8 * J));
    if (a.y_bf16)
        return a.h_bf16 ? run_norm<J, true, true>(a, threads, num_sms, st) : run_norm<J, true, false>(a, threads, num_sms, st);
    return a.h_bf16 ? run_norm<J, false, true>(a, threads, num_sms, st) : run_norm<J, false, false>(a, threads, num_sms, st);
}

template <int J, bool YB, bool HB>
cudaError_t run_norm_bwd(const NormBwdArgs &a, float *ws, int grid, Shape s, cudaStream_t st)
{
    const int units = J * ((YB ? 1 : 2) + 2 * (HB ? 1 : 2) + 1);
    // a token's gate is staged with the row unless a single stage would not fit
    const bool token = a.gate && a.gs;
    const int staged = token && (units + J) * s.threads * 16 <= kMaxSmem / s.ctas_per_sm ? 1 : 0;
    const int stage_bytes = (units + (staged ? J : 0)) * s.threads * 16;
    const int stages = ring_stages(stage_bytes, s.ctas_per_sm, (a.M + grid - 1) / grid);
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(norm_bwd_kernel<J, YB, HB>), kMaxSmem);
    if (e != cudaSuccess)
        return e;
    norm_bwd_kernel<J, YB, HB><<<grid, s.threads, stages * stage_bytes, st>>>(a, ws, stages, staged);
    return cudaGetLastError();
}

template <int J>
cudaError_t pick_norm_bwd(const NormBwdArgs &a, float *ws, int grid, Shape s, cudaStream_t st)
{
    if (a.y_bf16)
        return a.h_bf16 ? run_norm_bwd<J, true, true>(a, ws, grid, s, st) : run_norm_bwd<J, true, false>(a, ws, grid, s, st);
    return a.h_bf16 ? run_norm_bwd<J, false, true>(a, ws, grid, s, st) : run_norm_bwd<J, false, false>(a, ws, grid, s, st);
}

}  // namespace

int64_t norm_bwd_ws_floats(int64_t M, int N, int num_sms) { return (int64_t)bwd_ctas(M, N, num_sms) * 2 * N; }

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t st)
{
    // one chunk a thread for narrow rows, and for the few rows of a decode step
    const int J = a.M <= num_sms ? chunks(a.N, 1024, 0) : chunks(a.N, 512, 512);
    return J == 1 ? pick_norm<1>(a, num_sms, st) : J == 2 ? pick_norm<2>(a, num_sms, st) : pick_norm<4>(a, num_sms, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, float *ws, int num_sms, cudaStream_t st)
{
    const int J = chunks(a.N, 256, 512), grid = bwd_ctas(a.M, a.N, num_sms);
    const Shape s = bwd_shape(a.N);
    const cudaError_t e = J == 1   ? pick_norm_bwd<1>(a, ws, grid, s, st)
                          : J == 2 ? pick_norm_bwd<2>(a, ws, grid, s, st)
                                   : pick_norm_bwd<4>(a, ws, grid, s, st);
    if (e != cudaSuccess || (!a.dw1 && !a.dw2 && !(a.dgate && a.gs == 0)))
        return e;
    norm_bwd_sum_kernel<<<(a.N + 31) / 32, 256, 0, st>>>(a, ws, grid);
    return cudaGetLastError();
}

}  // namespace gemmar

// residual.cu -- a block's output joins the residual stream: norms before and
// after, gate, residual scale, and the next block's input as bf16 rows or as
// e4m3 codes with 1x128 scales (norm_gate_residual), and its backward pass.
//
// Both are HBM-bound: about 14 and 36 flops per element against 6 to 16 bytes, each
// input read and each output written once.  A persistent CTA takes a row at a
// time, a thread keeping the same units of 8 or 4 columns of every row, so that
// what a row needs from another thread is only its sums.  Rows
// ahead are copied to shared memory with cp.async into slots that only the
// copying thread reads: no barrier guards them, and a thread waits for nothing
// but its own copies.
#include <cuda_bf16.h>

#include <algorithm>

#include "e4m3_encode.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kMaxSmem = 231424;   // of the 232448 a CTA may have; the rest is static

// Two fp32 lanes in one register pair: the packed instructions round each lane as
// the scalar ones do and halve the issue slots, which bound these kernels before
// HBM does (see the measured figures at the kernels).
typedef uint64_t f2;

__device__ __forceinline__ f2 pack2(uint32_t lo, uint32_t hi)
{
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ f2 pack2(float lo, float hi) { return pack2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }
__device__ __forceinline__ float lo2(f2 v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(f2 v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// W consecutive values of a row as pairs.  W is 8 where the row's matrices are all
// bf16 and 4 where one of them is fp32: a thread's unit is then 16 bytes of the
// wider type, so that a warp's accesses cover whole 32-byte sectors (units of 8
// columns read and wrote fp32 rows in half sectors: 102 us instead of 66 at
// 4096 x 7168 with an fp32 stream).
template <int W>
struct Vec {
    f2 v[W / 2];
};

template <int W>
__device__ __forceinline__ Vec<W> all_of(float x)
{
    Vec<W> r;
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        r.v[i] = both(x);
    return r;
}

template <int W>
__device__ __forceinline__ Vec<W> operator*(const Vec<W> &a, const Vec<W> &b)
{
    Vec<W> r;
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        r.v[i] = mul2(a.v[i], b.v[i]);
    return r;
}

template <int W>
__device__ __forceinline__ Vec<W> operator*(const Vec<W> &a, f2 b)
{
    Vec<W> r;
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        r.v[i] = mul2(a.v[i], b);
    return r;
}

// a * b + c
template <int W>
__device__ __forceinline__ Vec<W> fma_of(const Vec<W> &a, f2 b, const Vec<W> &c)
{
    Vec<W> r;
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        r.v[i] = fma2(a.v[i], b, c.v[i]);
    return r;
}

template <int W>
__device__ __forceinline__ f2 dot_of(const Vec<W> &a, const Vec<W> &b, f2 s)
{
#pragma unroll
    for (int i = 0; i < W / 2; ++i)
        s = fma2(a.v[i], b.v[i], s);
    return s;
}

// A unit as it lies in memory: W * 2 or W * 4 bytes.
template <int W, bool BF>
struct Raw {
    static constexpr int kWords = W * (BF ? 2 : 4) / 4;   // 2, 4 or 8
    static constexpr int kBytes = kWords * 4;
    uint32_t w[kWords];

    __device__ __forceinline__ f2 pair(int i) const   // columns 2i, 2i + 1
    {
        if constexpr (BF)
            return pack2(w[i] << 16, w[i] & 0xFFFF0000u);
        else
            return pack2(w[2 * i], w[2 * i + 1]);
    }
    __device__ __forceinline__ Vec<W> vec() const
    {
        Vec<W> r;
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
            r.v[i] = pair(i);
        return r;
    }
    __device__ __forceinline__ void set(const Vec<W> &r)
    {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            if constexpr (BF) {
                w[i] = bf16x2_from_f32(lo2(r.v[i]), hi2(r.v[i]));
            } else {
                w[2 * i] = (uint32_t)r.v[i];
                w[2 * i + 1] = (uint32_t)(r.v[i] >> 32);
            }
        }
    }
    // from a shared-memory slot, or through the read-only cache
    __device__ __forceinline__ void read(uint32_t slot)
    {
        if constexpr (kWords == 2) {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(slot) : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < kWords; k += 4)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[k]), "=r"(w[k + 1]), "=r"(w[k + 2]), "=r"(w[k + 3])
                             : "r"(slot + k * 4)
                             : "memory");
        }
    }
    __device__ __forceinline__ void ldg(const void *p)
    {
        if constexpr (kWords == 2) {
            const uint2 x = __ldg(static_cast<const uint2 *>(p));
            w[0] = x.x;
            w[1] = x.y;
        } else {
#pragma unroll
            for (int k = 0; k < kWords; k += 4) {
                const uint4 x = __ldg(static_cast<const uint4 *>(p) + k / 4);
                w[k] = x.x;
                w[k + 1] = x.y;
                w[k + 2] = x.z;
                w[k + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void store(void *p) const
    {
        if constexpr (kWords == 2) {
            *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int k = 0; k < kWords; k += 4)
                static_cast<uint4 *>(p)[k / 4] = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        }
    }
};

template <int W>
__device__ __forceinline__ Vec<W> ldg_f32(const float *p)
{
    Raw<W, false> r;
    r.ldg(p);
    return r.vec();
}
template <int W>
__device__ __forceinline__ Vec<W> ldg_bf16(const uint16_t *p)
{
    Raw<W, true> r;
    r.ldg(p);
    return r.vec();
}
template <int W, bool BF>
__device__ __forceinline__ Vec<W> from_slot(uint32_t slot)
{
    Raw<W, BF> r;
    r.read(slot);
    return r.vec();
}
template <int W, bool BF>
__device__ __forceinline__ void store_vec(void *base, int64_t i, const Vec<W> &v)
{
    Raw<W, BF> r;
    r.set(v);
    r.store(static_cast<char *>(base) + i * (BF ? 2 : 4));
}

template <int BYTES>
__device__ __forceinline__ void zero_slot(uint32_t slot)
{
    if constexpr (BYTES == 8) {
        asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(slot), "r"(0u) : "memory");
    } else {
#pragma unroll
        for (int k = 0; k < BYTES; k += 16)
            st_shared_v4(slot + k, make_uint4(0, 0, 0, 0));
    }
}

// Copy the unit at column `col` of a row to the thread's slot.
template <int W, bool BF>
__device__ __forceinline__ void fetch(uint32_t slot, const void *row, int col)
{
    const char *src = static_cast<const char *>(row) + (int64_t)col * (BF ? 2 : 4);
    if constexpr (W * (BF ? 2 : 4) == 8)
        cp_async_ca8(slot, src);
    else
        cp_async_cg16(slot, src);
}

// This thread's oldest row of one or two under way has landed.
__device__ __forceinline__ void wait_stage(int stages)
{
    if (stages == 1)
        cp_async_wait<0>();
    else
        cp_async_wait<1>();
}

// Sum over the CTA, the same bits in every thread.  One barrier: two buffers take
// turns, so a warp that is a sum ahead of another writes the one not being read.
// Entries past the CTA's warps stay zero.
__device__ __forceinline__ float cta_sum(f2 pair, float (&bufs)[2][32], int &turn)
{
    float v = lo2(pair) + hi2(pair);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    float *red = bufs[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    const ulonglong2 *w = reinterpret_cast<const ulonglong2 *>(red);   // the sums of four warps
    f2 s0 = add2(add2(w[0].x, w[1].x), add2(w[2].x, w[3].x)), s1 = add2(add2(w[0].y, w[1].y), add2(w[2].y, w[3].y));
    if (blockDim.x > 512) {
        s0 = add2(s0, add2(add2(w[4].x, w[5].x), add2(w[6].x, w[7].x)));
        s1 = add2(s1, add2(add2(w[4].y, w[5].y), add2(w[6].y, w[7].y)));
    }
    s0 = add2(s0, s1);
    return lo2(s0) + hi2(s0);
}

// ---------------------------------------------------------------- forward

// First column of the thread's units; unit k is 32 W k further on.
template <int U, int W>
__device__ __forceinline__ int first_col()
{
    return ((int)(threadIdx.x & ~31u) * U + (int)(threadIdx.x & 31u)) * W;
}

// Unit k of an fp32 row kept in shared memory, in planes of 16 bytes a unit: a lane's 32
// bytes side by side would put two lanes on every bank.
template <int U, int W>
__device__ __forceinline__ uint32_t plane_of(uint32_t at, int k, int p)
{
    return at + p * (U * 16 * blockDim.x) + (first_col<U, W>() / W + k * 32) * 16;
}
template <int U, int W>
__device__ __forceinline__ void put_plane(uint32_t at, int k, const Vec<W> &v)
{
    Raw<W, false> r;
    r.set(v);
#pragma unroll
    for (int p = 0; p < W / 4; ++p)
        st_shared_v4(plane_of<U, W>(at, k, p), make_uint4(r.w[4 * p], r.w[4 * p + 1], r.w[4 * p + 2], r.w[4 * p + 3]));
}
template <int U, int W>
__device__ __forceinline__ Vec<W> get_plane(uint32_t at, int k)
{
    Raw<W, false> r;
#pragma unroll
    for (int p = 0; p < W / 4; ++p) {
        const uint4 x = ld_shared_v4(plane_of<U, W>(at, k, p));
        r.w[4 * p] = x.x;
        r.w[4 * p + 1] = x.y;
        r.w[4 * p + 2] = x.z;
        r.w[4 * p + 3] = x.w;
    }
    return r.vec();
}

// e4m3 codes of a row's units with one scale per 128 columns: a group is 128 / W
// neighbouring lanes of one unit (N % 128 == 0, so whole groups are inside the row).
// The U maxima are reduced together: while more than one is left, a step halves the
// lanes' distance and each lane keeps half of them, so lane l ends with the maximum
// of unit unit_of(l) and computes that unit's scale and reciprocal for the others.
template <int U, int W>
__device__ __forceinline__ void encode_units(const Vec<W> (&v)[U], uint8_t *q, float *scales, int N)
{
    constexpr int L = 128 / W;   // lanes of a group
    const int lane = threadIdx.x & 31, c0 = first_col<U, W>();
    float amax[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        amax[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
            amax[k] = fmaxf(amax[k], fmaxf(fabsf(lo2(v[k].v[i])), fabsf(hi2(v[k].v[i]))));
    }
    int o = L / 2, mine = 0;
#pragma unroll
    for (int n = U; n > 1; n /= 2, o /= 2) {
        const bool up = lane & o;
        mine = mine * 2 + (up ? 1 : 0);
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float keep = up ? amax[n / 2 + k] : amax[k], send = up ? amax[k] : amax[n / 2 + k];
            amax[k] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, send, o));
        }
    }
#pragma unroll
    for (; o > 0; o /= 2)
        amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xFFFFFFFFu, amax[0], o));
    const float sc = __fdiv_rn(amax[0], 448.0f);
    const float y = Enc::reciprocal(sc);
    // the first lane of a group with this unit writes its scale
    const int first = c0 - (lane & (L - 1)) * W + mine * 32 * W;
    if ((lane & (L / U - 1)) == 0 && first < N)
        scales[first / 128] = sc;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int col = c0 + k * 32 * W, src = (lane & ~(L - 1)) + k * (L / U);
        const Enc enc(__shfl_sync(0xFFFFFFFFu, sc, src), __shfl_sync(0xFFFFFFFFu, y, src));
        if (col < N) {
            float x[W];
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                x[2 * i] = lo2(v[k].v[i]);
                x[2 * i + 1] = hi2(v[k].v[i]);
            }
            uint32_t w[W / 4];
            enc.codes<W>(x, w);
            if constexpr (W == 8)
                *reinterpret_cast<uint2 *>(q + col) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(q + col) = w[0];
        }
    }
}

// STAGED (CTAs of several rows): the weights are kept in shared memory, w_post times a gate row
// as one, since 72 KB of them do not stay in L1 beside the rows: 16384 x 7168 bf16 with codes
// 147 us, 183 through L1.  With fp32 rows w_pre stays in L1, which then has room for it:
// 4096 x 7168 57 us, 61 with both, 61 with none.
__host__ __device__ constexpr bool stage_pre(int W) { return W == 8; }

// A thread holds U units of W columns of its row.  A warp takes 32 U W neighbouring
// columns and its units lie 32 W apart, so one address per matrix and fixed
// offsets reach them all (with units T W apart address arithmetic was a third of
// the instructions: 71 us instead of 66 at 4096 x 7168, fp32 stream, codes).
// Two rows an SM in flight (two CTAs) hide each other's two sums.
// 16384 x 7168 with a gate per token, bf16: 175 us, 6.7 TB/s, the rate of a copy.  4096 x
// 7168 with an fp32 stream and codes: 56 us, 5.8 TB/s (16384 rows 202 us, 6.4): the first
// rows' copies and 14 turns for 13.5 rows a CTA are the rest.
template <int U, bool YB, bool HB, bool STAGED>
__global__ void __launch_bounds__(1024, 1) norm_kernel(const NormArgs a, int stages)
{
    constexpr int W = YB && HB ? 8 : 4;
    constexpr int kY = Raw<W, YB>::kBytes, kH = Raw<W, HB>::kBytes, kG = Raw<W, true>::kBytes;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ __align__(16) float red[2][32];
    const int T = blockDim.x, t = threadIdx.x, N = a.N;
    const bool token = a.gate != nullptr && a.gs != 0;
    const uint32_t off_h = U * kY * T, off_g = off_h + U * kH * T;
    const uint32_t stage_bytes = off_g + (token ? U * kG * T : 0);
    const uint32_t base = smem_u32(smem_raw);
    const uint32_t at_cw = base + stages * stage_bytes;   // STAGED
    const float inv_n = 1.0f / N;
    const int c0 = first_col<U, W>();
    auto col_of = [&](int k) { return c0 + k * 32 * W; };
    // a stage holds each matrix's row in the order of its columns
    auto y_slot = [&](uint32_t st, int k) { return st + c0 * (kY / W) + k * 32 * kY; };
    auto h_slot = [&](uint32_t st, int k) { return st + off_h + c0 * (kH / W) + k * 32 * kH; };
    auto g_slot = [&](uint32_t st, int k) { return st + off_g + c0 * (kG / W) + k * 32 * kG; };

    auto fetch_row = [&](int64_t m, uint32_t st) {
        const char *y = static_cast<const char *>(a.y) + m * a.ys * (YB ? 2 : 4);
        const char *h = static_cast<const char *>(a.h) + m * a.hs * (HB ? 2 : 4);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (col_of(k) < N) {
                fetch<W, YB>(y_slot(st, k), y, col_of(k));
                fetch<W, HB>(h_slot(st, k), h, col_of(k));
                if (token)
                    fetch<W, true>(g_slot(st, k), a.gate + m * a.gs, col_of(k));
            }
        }
    };

    // Units past the row's end read as zero and add nothing: their scale is zero too, since 0
    // times an infinite weight would. Only their copies and stores are left out, so the row's
    // passes have no branches.
    bool ok[U];
    int wcol[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        ok[k] = col_of(k) < N;
        wcol[k] = ok[k] ? col_of(k) : 0;
        if (!ok[k]) {
            for (int s = 0; s < stages; ++s) {
                const uint32_t st = base + s * stage_bytes;
                zero_slot<kY>(y_slot(st, k));
                zero_slot<kH>(h_slot(st, k));
                if (token)
                    zero_slot<kG>(g_slot(st, k));
            }
        }
    }
    int64_t ahead = blockIdx.x;   // next row to fetch
    for (int s = 0; s < stages; ++s, ahead += gridDim.x) {
        if (ahead < a.M)
            fetch_row(ahead, base + s * stage_bytes);
        cp_async_commit();
    }
    // w_post times a gate that is one row, and w_pre
    const bool scaled = a.w1 != nullptr || (a.gate != nullptr && !token);
    const bool normed = a.u != nullptr || a.q != nullptr;
    auto scale = [&](int k) {
        Vec<W> cw = all_of<W>(1.0f);
        if (a.w1)
            cw = ldg_f32<W>(a.w1 + wcol[k]);
        if (a.gate && !token)
            cw = cw * ldg_bf16<W>(a.gate + wcol[k]);
        if constexpr (!STAGED)
            return ok[k] ? cw : all_of<W>(0.0f);
        return cw;
    };
    constexpr bool kStageW2 = STAGED && stage_pre(W);
    const uint32_t at_w2 = at_cw + (scaled ? U * W * 4 * T : 0);
    if constexpr (STAGED) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (scaled)
                put_plane<U, W>(at_cw, k, scale(k));
            if (kStageW2 && normed)
                put_plane<U, W>(at_w2, k, ldg_f32<W>(a.w2 + wcol[k]));
        }
    }
    // The zeros by themselves: 4096 x 7168, fp32 stream 57.8 us a pass, 59.4 as a choice at the store above.
    if constexpr (STAGED) {
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (scaled && !ok[k])
                put_plane<U, W>(at_cw, k, all_of<W>(0.0f));
    }
    for (int i = t; i < 64; i += T)
        red[i >> 5][i & 31] = 0.0f;
    __syncthreads();
    int get = 0, turn = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, ahead += gridDim.x) {
        wait_stage(stages);
        const uint32_t st = base + get * stage_bytes;
        if (++get == stages)
            get = 0;

        Vec<W> v[U];   // y, then t, then x
        float r1 = 1.0f, r2 = 1.0f;
#pragma unroll
        for (int k = 0; k < U; ++k)
            v[k] = from_slot<W, YB>(y_slot(st, k));
        if (a.w1) {
            f2 ss = both(0.0f);
#pragma unroll
            for (int k = 0; k < U; ++k)
                ss = dot_of(v[k], v[k], ss);
            r1 = rsqrtf(cta_sum(ss, red, turn) * inv_n + a.eps);
        }
        const f2 br1 = both(a.beta * r1), alpha = both(a.alpha);
#pragma unroll
        for (int k = 0; k < U; ++k)
            v[k] = v[k] * br1;
        if (scaled) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if constexpr (STAGED)
                    v[k] = v[k] * get_plane<U, W>(at_cw, k);
                else
                    v[k] = v[k] * scale(k);
            }
        }
        if (token) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                v[k] = v[k] * from_slot<W, true>(g_slot(st, k));
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            v[k] = fma_of(from_slot<W, HB>(h_slot(st, k)), alpha, v[k]);
        // this thread has read all of its slots: the row `stages` ahead takes them
        if (ahead < a.M)
            fetch_row(ahead, st);
        cp_async_commit();
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (ok[k])
                store_vec<W, HB>(a.t, m * N + col_of(k), v[k]);
        if (a.w2) {
            f2 ss = both(0.0f);
#pragma unroll
            for (int k = 0; k < U; ++k)
                ss = dot_of(v[k], v[k], ss);
            r2 = rsqrtf(cta_sum(ss, red, turn) * inv_n + a.eps);
        }
        if (a.rstd && t == 0)
            *reinterpret_cast<float2 *>(a.rstd + 2 * m) = make_float2(r1, r2);
        if (!normed)
            continue;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if constexpr (kStageW2)
                v[k] = v[k] * both(r2) * get_plane<U, W>(at_w2, k);
            else
                v[k] = v[k] * both(r2) * ldg_f32<W>(a.w2 + wcol[k]);
        }
        if (a.u) {
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (ok[k])
                    store_vec<W, true>(a.u, m * N + col_of(k), v[k]);
        }
        if (a.q)
            encode_units<U, W>(v, a.q + m * N, a.scales + m * (N / 128), N);
    }
}

// ---------------------------------------------------------------- backward

// One pass over the row forms four sums, from which both projections follow:
// with dv = du w2, c = beta g w1, n = y r1, t = alpha h + c n and d = dt + r2 (dv - k t),
// k = r2 (r2 mean(dv t)) (`proj`),
//   mean(c n d) = mean(c n dt) + r2 (mean(c n dv) - k mean(c n t)).
// k t is of dv's size whatever the row's; r2^3, where it appears by itself, leaves the fp32 range
// for rows of rms above 1e12 or below 1e-12.
// The second pass recomputes n, t and dv and writes dy, dh (and a token's dgate).
// The sums over rows, s1 = sum n d (times a token's gate) and s2 = sum du t r2,
// stay in the thread's registers over all the CTA's rows and leave as one part per
// CTA, summed in the CTAs' order by norm_bwd_sum_kernel.
// HOLD (rows up to 8192, 16 columns a thread): the row's packed values stay in
// registers between the passes, so its slots are free for the next row before the
// sums are exchanged; the weights sit in shared memory.  Wider rows take 32 columns
// a thread, read the slots twice and the weights through L1.
// BOTH: both norms are there (known when compiling, a pass of the row is one loop).
// 4096 x 7168 bf16: 74 us, 4.8 TB/s; 16384 rows 255, 5.5.  Not bound by HBM (56% busy) nor
// by one pipe (issue slots 44%): 14 warps of 122 registers, whose two sums over the rows
// leave no room for a second CTA, do not hide the latencies of shared memory and of the
// arithmetic.  Running a row's first pass before the second of the row before it, so
// that the exchange of sums is off the path, was no faster (78 and 268 us against 78 and 265),
// nor twice the threads with 8 columns each (95 against 81).  Rows wider than 8192 have one CTA's ring for a
// single row: 4096 x 16384 210 us, 3.8 TB/s.
template <int U, bool YB, bool HB, bool TOKEN, bool HOLD, bool BOTH>
__global__ void __launch_bounds__(512, 1)
    norm_bwd_kernel(const NormBwdArgs a, float *__restrict__ ws, int stages, int gate_staged)
{
    constexpr int W = YB && HB ? 8 : 4;
    constexpr int kY = Raw<W, YB>::kBytes, kH = Raw<W, HB>::kBytes, kB = Raw<W, true>::kBytes, kF = Raw<W, false>::kBytes;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ float red[2][16][4];
    const int T = blockDim.x, t = threadIdx.x, lane = t & 31, N = a.N;
    const bool pre = BOTH || a.w2 != nullptr, post = BOTH || a.w1 != nullptr;
    const uint32_t off_h = U * kY * T, off_dt = off_h + U * kH * T, off_du = off_dt + U * kH * T, off_g = off_du + U * kB * T;
    const uint32_t stage_bytes = off_g + (gate_staged ? U * kB * T : 0);
    const uint32_t base = smem_u32(smem_raw);
    const uint32_t off_cw = stages * stage_bytes, off_w2 = off_cw + U * kF * T;   // HOLD
    const float inv_n = 1.0f / N;
    const int c0 = first_col<U, W>();
    auto col_of = [&](int k) { return c0 + k * 32 * W; };
    // of a row kept at `off` in the order of its columns, unit k's `bytes`
    auto at = [&](uint32_t off, int bytes, int k) { return off + c0 * (bytes / W) + k * 32 * bytes; };

    auto fetch_row = [&](int64_t m, uint32_t st) {
        const char *y = static_cast<const char *>(a.y) + m * a.ys * (YB ? 2 : 4);
        const char *h = static_cast<const char *>(a.h) + m * a.hs * (HB ? 2 : 4);
        const char *dt = static_cast<const char *>(a.dt) + m * a.dts * (HB ? 2 : 4);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int col = col_of(k);
            if (col < N) {
                fetch<W, YB>(at(st, kY, k), y, col);
                fetch<W, HB>(at(st + off_h, kH, k), h, col);
                if (a.dt)
                    fetch<W, HB>(at(st + off_dt, kH, k), dt, col);
                if (pre)
                    fetch<W, true>(at(st + off_du, kB, k), a.du + m * a.dus, col);
                if (gate_staged)
                    fetch<W, true>(at(st + off_g, kB, k), a.gate + m * a.gs, col);
            }
        }
    };
    // a gradient that is absent reads as zero
    for (int s = 0; s < stages; ++s) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!a.dt) {
                Raw<W, HB> z;
                z.set(all_of<W>(0.0f));
                z.store(smem_raw + at(s * stage_bytes + off_dt, kH, k));
            }
            if (!pre) {
                Raw<W, true> z;
                z.set(all_of<W>(0.0f));
                z.store(smem_raw + at(s * stage_bytes + off_du, kB, k));
            }
        }
    }
    int64_t ahead = blockIdx.x;
    for (int s = 0; s < stages; ++s, ahead += gridDim.x) {
        if (ahead < a.M)
            fetch_row(ahead, base + s * stage_bytes);
        cp_async_commit();
    }

    // beta w1 (times the gate when it is one row), and w2
    auto weights = [&](int col, Vec<W> &cw, Vec<W> &w2) {
        cw = all_of<W>(a.beta);
        w2 = all_of<W>(0.0f);
        if (post)
            cw = cw * ldg_f32<W>(a.w1 + col);
        if (a.gate != nullptr && !TOKEN)
            cw = cw * ldg_bf16<W>(a.gate + col);
        if (pre)
            w2 = ldg_f32<W>(a.w2 + col);
    };
    if constexpr (HOLD) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (col_of(k) < N) {
                Vec<W> cw, w2;
                weights(col_of(k), cw, w2);
                put_plane<U, W>(base + off_cw, k, cw);
                put_plane<U, W>(base + off_w2, k, w2);
            }
        }
    }

    Vec<W> s1[U], s2[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
        s1[k] = s2[k] = all_of<W>(0.0f);

    int get = 0, turn = 0;
    // the reciprocal norms are loaded a row ahead
    const float2 *rstd = reinterpret_cast<const float2 *>(a.rstd);
    float2 next = __ldg(rstd + blockIdx.x);
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, ahead += gridDim.x) {
        const float r1s = next.x, r2s = next.y;
        if (m + gridDim.x < a.M)
            next = __ldg(rstd + m + gridDim.x);
        const f2 r1 = both(r1s), r2 = both(r2s), alpha = both(a.alpha);
        wait_stage(stages);
        const uint32_t st = base + get * stage_bytes;
        if (++get == stages)
            get = 0;

        Raw<W, YB> ry[HOLD ? U : 1];
        Raw<W, HB> rh[HOLD ? U : 1], rdt[HOLD ? U : 1];
        Raw<W, true> rdu[HOLD ? U : 1], rg[HOLD ? U : 1];
        auto read = [&](int k) {
            const int i = HOLD ? k : 0;
            ry[i].read(at(st, kY, k));
            rh[i].read(at(st + off_h, kH, k));
            rdt[i].read(at(st + off_dt, kH, k));
            rdu[i].read(at(st + off_du, kB, k));
            if constexpr (TOKEN) {
                if (gate_staged)
                    rg[i].read(at(st + off_g, kB, k));
                else
                    rg[i].ldg(a.gate + m * a.gs + col_of(k));
            }
        };
        // pair i of unit k: n, gcw = cw (times a token's gate), cn = gcw n, t = alpha h + cn, dv = du w2
        struct Pair {
            f2 n, cw, gcw, cn, t, du, dv;
        };
        auto form = [&](int k, int i, const Vec<W> &cws, const Vec<W> &w2s) {
            const int r = HOLD ? k : 0;
            Pair p;
            p.n = mul2(ry[r].pair(i), r1);
            p.gcw = p.cw = cws.v[i];
            if constexpr (TOKEN)
                p.gcw = mul2(p.cw, rg[r].pair(i));
            p.cn = mul2(p.gcw, p.n);
            p.t = fma2(rh[r].pair(i), alpha, p.cn);
            p.du = rdu[r].pair(i);
            p.dv = mul2(p.du, w2s.v[i]);
            return p;
        };
        auto row_weights = [&](int k, Vec<W> &cw, Vec<W> &w2) {
            if constexpr (HOLD) {
                cw = get_plane<U, W>(base + off_cw, k);
                w2 = get_plane<U, W>(base + off_w2, k);
            } else {
                weights(col_of(k), cw, w2);
            }
        };

        f2 q0 = both(0.0f), q1 = q0, q2 = q0, q3 = q0;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (col_of(k) < N) {
                read(k);
                Vec<W> cw, w2;
                row_weights(k, cw, w2);
#pragma unroll
                for (int i = 0; i < W / 2; ++i) {
                    const Pair p = form(k, i, cw, w2);
                    q0 = fma2(p.dv, p.t, q0);
                    q1 = fma2(p.cn, rdt[HOLD ? k : 0].pair(i), q1);
                    q2 = fma2(p.cn, p.dv, q2);
                    q3 = fma2(p.cn, p.t, q3);
                }
            }
        }
        if constexpr (HOLD) {
            if (ahead < a.M)
                fetch_row(ahead, st);
            cp_async_commit();
        }
        float proj = 0.0f, mean1 = 0.0f;
        if (pre || post) {
            // as in encode_units: lane l ends with sum l >> 3 of its warp
            const bool up = lane & 16, up2 = lane & 8;
            float s0 = lo2(q0) + hi2(q0), s1w = lo2(q1) + hi2(q1), s2w = lo2(q2) + hi2(q2), s3 = lo2(q3) + hi2(q3);
            const float k0 = (up ? s2w : s0) + __shfl_xor_sync(0xFFFFFFFFu, up ? s0 : s2w, 16);
            const float k1 = (up ? s3 : s1w) + __shfl_xor_sync(0xFFFFFFFFu, up ? s1w : s3, 16);
            float s = (up2 ? k1 : k0) + __shfl_xor_sync(0xFFFFFFFFu, up2 ? k0 : k1, 8);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            float(*buf)[4] = red[turn];
            turn ^= 1;
            if ((lane & 7) == 0)
                buf[t >> 5][lane >> 3] = s;
            __syncthreads();
            // lane l: sum l & 3 of the warps l >> 2 and l >> 2 + 8
            const int w0 = lane >> 2, warps = T >> 5;
            s = (w0 < warps ? buf[w0][lane & 3] : 0.0f) + (w0 + 8 < warps ? buf[w0 + 8][lane & 3] : 0.0f);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
                s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            s *= inv_n;
            proj = r2s * (r2s * __shfl_sync(0xFFFFFFFFu, s, 0));   // used with a pre norm alone
            const float m_dt = __shfl_sync(0xFFFFFFFFu, s, 1), m_dv = __shfl_sync(0xFFFFFFFFu, s, 2),
                        m_t = __shfl_sync(0xFFFFFFFFu, s, 3);
            // h is in m_t alone: without a pre norm it must not come in as 0 * inf
            mean1 = !post ? 0.0f : pre ? fmaf(r2s, fmaf(-proj, m_t, m_dv), m_dt) : m_dt;
        }
        const f2 mk = both(-proj), mm = both(-r1s * mean1);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int col = col_of(k), r = HOLD ? k : 0;
            if (col < N) {
                if constexpr (!HOLD)
                    read(k);
                Vec<W> cw, w2, d = rdt[r].vec(), dy, dg;
                row_weights(k, cw, w2);
                if constexpr (BOTH) {
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        const Pair p = form(k, i, cw, w2);
                        d.v[i] = fma2(fma2(p.t, mk, p.dv), r2, d.v[i]);
                        s2[k].v[i] = fma2(mul2(p.du, r2), p.t, s2[k].v[i]);
                        if constexpr (TOKEN) {
                            const f2 nd = mul2(p.n, d.v[i]);
                            dg.v[i] = mul2(p.cw, nd);
                            s1[k].v[i] = fma2(nd, rg[r].pair(i), s1[k].v[i]);
                        } else {
                            s1[k].v[i] = fma2(p.n, d.v[i], s1[k].v[i]);
                        }
                        dy.v[i] = fma2(p.n, mm, mul2(mul2(p.gcw, d.v[i]), r1));
                    }
                } else {
                    // a norm that is absent must not bring its row's infinities in as 0 * inf
                    if (pre) {
#pragma unroll
                        for (int i = 0; i < W / 2; ++i) {
                            const Pair p = form(k, i, cw, w2);
                            d.v[i] = fma2(fma2(p.t, mk, p.dv), r2, d.v[i]);
                            s2[k].v[i] = fma2(mul2(p.du, r2), p.t, s2[k].v[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        const Pair p = form(k, i, cw, w2);
                        if constexpr (TOKEN) {
                            const f2 nd = mul2(p.n, d.v[i]);
                            dg.v[i] = mul2(p.cw, nd);
                            s1[k].v[i] = fma2(nd, rg[r].pair(i), s1[k].v[i]);
                        } else {
                            s1[k].v[i] = fma2(p.n, d.v[i], s1[k].v[i]);
                        }
                        dy.v[i] = mul2(mul2(p.gcw, d.v[i]), r1);
                    }
                    if (post) {
#pragma unroll
                        for (int i = 0; i < W / 2; ++i)
                            dy.v[i] = fma2(mul2(ry[r].pair(i), r1), mm, dy.v[i]);
                    }
                }
                store_vec<W, YB>(a.dy, m * N + col, dy);
                store_vec<W, HB>(a.dh, m * N + col, d * alpha);
                if constexpr (TOKEN) {
                    if (a.dgate)
                        store_vec<W, true>(a.dgate, m * N + col, dg);
                }
            }
        }
        if constexpr (!HOLD) {
            if (ahead < a.M)
                fetch_row(ahead, st);
            cp_async_commit();
        }
    }
    grid_launch_next();
    float *part = ws + (int64_t)blockIdx.x * 2 * N;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int col = col_of(k);
        if (col < N) {
            store_vec<W, false>(part, col, s1[k]);
            store_vec<W, false>(part, N + col, s2[k]);
        }
    }
}

// The sums of the CTAs' parts, in an order that their number fixes.  A CTA takes eight
// columns (a 32-byte sector of a part), its groups of eight lanes take the parts in
// turn, and a warp a column then adds the groups' sums.  Wide rows have few parts and
// many columns, narrow ones the opposite: 32 groups or 128 (the whole backward pass of
// 4096 x 7168 80 us with 32 groups, 84 with 128; of 16384 x 1024 54 and 42).
// s1 = sum n d (times a token's gate): dw1 = beta g s1 and dgate = beta w1 s1 for a gate
// row g.
constexpr int kSumGroups = 128;   // at most

__global__ void __launch_bounds__(kSumGroups * 8) norm_bwd_sum_kernel(const NormBwdArgs a, const float *ws,
                                                                      int parts)
{
    __shared__ float sums[2][8][kSumGroups + 1];
    grid_wait();
    const int col = threadIdx.x & 7, group = threadIdx.x >> 3, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = blockDim.x / 8;
    float s1 = 0.0f, s2 = 0.0f;
    const float *src = ws + blockIdx.x * 8 + col;   // N is a multiple of eight
#pragma unroll 4
    for (int p = group; p < parts; p += groups) {
        s1 += ld_after_f32(src + (int64_t)p * 2 * a.N);
        s2 += ld_after_f32(src + (int64_t)p * 2 * a.N + a.N);
    }
    sums[0][col][group] = s1;
    sums[1][col][group] = s2;
    __syncthreads();
    if (warp >= 8)
        return;
    s1 = s2 = 0.0f;
    for (int k = 0; k < groups; k += 32) {
        s1 += sums[0][warp][k + lane];
        s2 += sums[1][warp][k + lane];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
        s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
    }
    const int n = blockIdx.x * 8 + warp;
    if (lane != 0)
        return;
    const bool row = a.gate && a.gs == 0;
    if (a.dw1)
        a.dw1[n] = a.beta * (row ? bf16_lo(a.gate[n]) : 1.0f) * s1;
    if (a.dw2)
        a.dw2[n] = s2;
    if (a.dgate && row)
        static_cast<float *>(a.dgate)[n] = a.beta * (a.w1 ? a.w1[n] : 1.0f) * s1;
}

// ---------------------------------------------------------------- launches

int round32(int v) { return (v + 31) / 32 * 32; }

constexpr int kWide = 8192;            // widest row of 16 columns a thread in 512 threads
constexpr int kSmSmem = 228 * 1024, kCtaSmem = 2048;   // an SM's, and a CTA's besides the dynamic part
constexpr int kStageRows = 3;   // of a CTA, from which staged weights pay (3 of 7168 bf16 columns: 13.9 us, 15.9 without)

struct Plan {
    int threads, per_sm;   // CTAs an SM
};

// As many CTAs an SM as fill `most` threads.
Plan plan_rows(int N, int cols, int most)
{
    const int threads = round32((N + cols - 1) / cols);
    const int per_sm = most / threads;
    return {threads, per_sm < 1 ? 1 : per_sm > 16 ? 16 : per_sm};
}

// Rows of a CTA under way: two if they fit, one if it has no second.
int ring_stages(int64_t room, int stage_bytes, int64_t rows) { return rows >= 2 && room >= 2 * stage_bytes ? 2 : 1; }

Plan plan_bwd(int N) { return plan_rows(N, N <= kWide ? 16 : 32, 512); }

int bwd_ctas(int64_t M, int N, int num_sms)
{
    // at least two rows a CTA, so that the parts never need more room than the rows themselves
    const int64_t most = (int64_t)num_sms * plan_bwd(N).per_sm, some = (M + 1) / 2;
    return (int)(some < most ? some : most);
}

// COLS columns a thread.
template <int COLS, bool YB, bool HB>
cudaError_t run_norm(const NormArgs &a, int num_sms, cudaStream_t st)
{
    constexpr int W = YB && HB ? 8 : 4;
    const Plan p = plan_rows(a.N, COLS, 1024);
    const int stage_bytes = p.threads * COLS * ((YB ? 2 : 4) + (HB ? 2 : 4) + (a.gate && a.gs ? 2 : 0));
    const int64_t most = (int64_t)num_sms * p.per_sm;
    const int grid = (int)(a.M < most ? a.M : most);
    const int64_t rows = (a.M + grid - 1) / grid;
    const int kept = (a.w1 || (a.gate && a.gs == 0) ? 1 : 0) + (stage_pre(W) && (a.u || a.q) ? 1 : 0);
    const int weight_bytes = kept * p.threads * COLS * 4;
    const int64_t room = kSmSmem / p.per_sm - kCtaSmem - weight_bytes;
    const bool staged = rows >= kStageRows && room >= stage_bytes;
    // One row: a second takes its shared memory from L1 (16384 x 7168 bf16 147 us, 168 with
    // two), but narrow rows with a gate each have too few bytes under way (3584 columns
    // 108 us, 94 with two).
    const int stages = COLS == 8 && a.gate && a.gs ? ring_stages(room, stage_bytes, rows) : 1;
    const auto kernel = staged ? norm_kernel<COLS / W, YB, HB, true> : norm_kernel<COLS / W, YB, HB, false>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), kMaxSmem);
    if (e != cudaSuccess)
        return e;
    kernel<<<grid, p.threads, stages * stage_bytes + (staged ? weight_bytes : 0), st>>>(a, stages);
    return cudaGetLastError();
}

template <int COLS>
cudaError_t pick_norm(const NormArgs &a, int num_sms, cudaStream_t st)
{
    if (a.y_bf16)
        return a.h_bf16 ? run_norm<COLS, true, true>(a, num_sms, st) : run_norm<COLS, true, false>(a, num_sms, st);
    return a.h_bf16 ? run_norm<COLS, false, true>(a, num_sms, st) : run_norm<COLS, false, false>(a, num_sms, st);
}

template <int COLS, bool YB, bool HB, bool TOKEN>
cudaError_t run_norm_bwd(const NormBwdArgs &a, float *ws, int grid, cudaStream_t st)
{
    constexpr int W = YB && HB ? 8 : 4;
    constexpr bool kHold = COLS == 16;
    const Plan p = plan_bwd(a.N);
    const int cols = p.threads * COLS;
    const int weight_bytes = kHold ? 2 * cols * 4 : 0;
    const int bytes = cols * ((YB ? 2 : 4) + 2 * (HB ? 2 : 4) + 2);
    // a token's gate is staged with the row unless one stage would not fit
    const int staged = TOKEN && bytes + cols * 2 + weight_bytes <= kMaxSmem ? 1 : 0;
    const int stage_bytes = bytes + (staged ? cols * 2 : 0);
    const int64_t room = (p.per_sm == 1 ? kMaxSmem : kMaxSmem / p.per_sm - 2048) - weight_bytes;
    // a third row would slow the first one down: 608 x 7168 23 us, 21 with two, 4096 rows 77.4 and 75.6
    const int stages = ring_stages(room, stage_bytes, (a.M + grid - 1) / grid);
    const auto kernel = a.w1 && a.w2 ? norm_bwd_kernel<COLS / W, YB, HB, TOKEN, kHold, true>
                                     : norm_bwd_kernel<COLS / W, YB, HB, TOKEN, kHold, false>;
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kernel), kMaxSmem);
    if (e != cudaSuccess)
        return e;
    kernel<<<grid, p.threads, stages * stage_bytes + weight_bytes, st>>>(a, ws, stages, staged);
    return cudaGetLastError();
}

template <int COLS, bool TOKEN>
cudaError_t pick_norm_bwd(const NormBwdArgs &a, float *ws, int grid, cudaStream_t st)
{
    if (a.y_bf16)
        return a.h_bf16 ? run_norm_bwd<COLS, true, true, TOKEN>(a, ws, grid, st)
                        : run_norm_bwd<COLS, true, false, TOKEN>(a, ws, grid, st);
    return a.h_bf16 ? run_norm_bwd<COLS, false, true, TOKEN>(a, ws, grid, st)
                    : run_norm_bwd<COLS, false, false, TOKEN>(a, ws, grid, st);
}

}  // namespace

int64_t norm_bwd_ws_floats(int64_t M, int N, int num_sms) { return (int64_t)bwd_ctas(M, N, num_sms) * 2 * N; }

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t st)
{
    // 16 columns a thread, two CTAs an SM; 8 for narrow rows and for the few rows of a decode step
    return a.N <= kWide / 2 || (a.N <= kWide && a.M <= num_sms) ? pick_norm<8>(a, num_sms, st)
                                                               : pick_norm<16>(a, num_sms, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, float *ws, int num_sms, cudaStream_t st)
{
    const int grid = bwd_ctas(a.M, a.N, num_sms);
    const bool token = a.gate && a.gs;
    const cudaError_t e = a.N <= kWide ? (token ? pick_norm_bwd<16, true>(a, ws, grid, st) : pick_norm_bwd<16, false>(a, ws, grid, st))
                                       : (token ? pick_norm_bwd<32, true>(a, ws, grid, st) : pick_norm_bwd<32, false>(a, ws, grid, st));
    if (e != cudaSuccess || (!a.dw1 && !a.dw2 && !(a.dgate && a.gs == 0)))
        return e;
    return launch(norm_bwd_sum_kernel, dim3(a.N / 8), (grid <= 256 ? 32 : kSumGroups) * 8, 0, 1, true, st, a, static_cast<const float *>(ws), grid);
}

}  // namespace gemmar

// lora.cu -- low-rank adapters of many requests beside a shared projection.
// Both factors of an adapter are stored rank-major ([R, r, C]), so the forward
// pass and its gradients are three products over the tokens of each adapter:
//   down: v[i,j] = f sum_c x[t,c] W[a,j,c]              (x A^T; dy B^T)
//   up:   out[t,c] = base[t,c] + f sum_j v[i,j] W[a,j,c]  (v B; w A)
//   grad: G[a,j,c] = f sum_i p[i,j] x[t,c]              (w^T x; v^T dy)
// with t = order[i], i in [offsets[a], offsets[a+1]), f = scales[a] or 1.
#include <cuda_bf16.h>

#include <algorithm>

#include "gemmar.h"
#include "lora.cuh"

namespace gemmar {
using namespace ptx;

namespace {

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

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- few tokens
//
// A decode batch: every adapter in it brings its weights for a token or a few, so
// the weights are what is read, and latency is what counts.  Both kernels load
// their fragments straight from memory into registers, 16 bytes a lane, no
// staging: the contraction index of an MMA may be permuted as long as both
// operands agree, so lane (g, q) takes eight consecutive elements of its row for
// two MMAs.  Weights are the M operand, tokens the N operand (8 a tile).

constexpr int kFewBatch = 256;   // largest batch for these kernels
constexpr int kFewTokens = 32;   // tokens a tile: four N tiles
constexpr int kFewWarps = 8;
constexpr int kFewRanks = 32;    // ranks a CTA of the down kernel: two M tiles

// v[i][j] of a tile: the CTAs of a cluster share the columns (blockIdx.y) and so do a
// CTA's eight warps; their sums are added in warp and in rank order.
__global__ void __launch_bounds__(kFewWarps * 32) few_down_kernel(const LoraArgs l, const uint16_t *__restrict__ x,
                                                                  int64_t xs, const uint16_t *__restrict__ W, int C,
                                                                  bool scaled, float *__restrict__ v)
{
    __shared__ float sums[kFewWarps][kFewRanks][kFewTokens + 1];
    const Tile tile = find_tile(l, blockIdx.x, kFewTokens, false);
    const int rank = tile.of ? rank_of(l, tile.a) : 0, j0 = blockIdx.z * kFewRanks;
    if (tile.of == 0)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    float acc[2][4][4] = {};
    if (j0 < rank) {
        const uint16_t *wr[4];   // rows j0 + g, + 8, + 16, + 24
        bool wok[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + g + 8 * i;
            wok[i] = j < rank;
            wr[i] = W + ((int64_t)tile.a * l.r + (wok[i] ? j : 0)) * C + q * 8;
        }
        const int nt = (tile.count + 7) / 8;
        const uint16_t *xr[4];
        bool xok[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i = n * 8 + g;
            const int t = i < tile.count ? __ldg(l.order + tile.i0 + i) : -1;
            xok[n] = t >= 0 && t < l.T;
            xr[n] = x + (xok[n] ? t : 0) * xs + q * 8;
        }
        // blocks of 32 columns, dealt evenly to splits and warps
        const int blocks = (C + 31) / 32, shares = gridDim.y * kFewWarps, share = blockIdx.y * kFewWarps + warp;
        const int b0 = (int)((int64_t)blocks * share / shares), b1 = (int)((int64_t)blocks * (share + 1) / shares);
        const bool wide = j0 + 16 < rank;
#pragma unroll 4
        for (int b = b0; b < b1; ++b) {
            const bool in = b * 32 + q * 8 < C;
            uint4 w[4], xv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = make_uint4(0, 0, 0, 0);
                if (in && wok[i])
                    w[i] = __ldg(reinterpret_cast<const uint4 *>(wr[i] + b * 32));
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                xv[n] = make_uint4(0, 0, 0, 0);
                if (in && xok[n])
                    xv[n] = __ldg(reinterpret_cast<const uint4 *>(xr[n] + b * 32));
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (m == 1 && !wide)
                    break;
                const uint32_t lo[4] = {w[2 * m].x, w[2 * m + 1].x, w[2 * m].y, w[2 * m + 1].y};
                const uint32_t hi[4] = {w[2 * m].z, w[2 * m + 1].z, w[2 * m].w, w[2 * m + 1].w};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    if (n < nt) {
                        mma_bf16(acc[m][n], lo, xv[n].x, xv[n].y);
                        mma_bf16(acc[m][n], hi, xv[n].z, xv[n].w);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sums[warp][m * 16 + g + (e >> 1) * 8][n * 8 + q * 2 + (e & 1)] = acc[m][n][e];
    __syncthreads();
    for (int e = threadIdx.x; e < kFewRanks * kFewTokens; e += kFewWarps * 32) {
        float *at = &sums[0][e / kFewTokens][e % kFewTokens];
        float s = *at;
#pragma unroll
        for (int w = 1; w < kFewWarps; ++w)
            s += sums[w][e / kFewTokens][e % kFewTokens];
        *at = s;
    }
    const float f = scaled ? l.scales[tile.a] : 1.0f;
    float *out = v + (int64_t)tile.i0 * l.r + j0;
    cluster_sum(smem_u32(sums), min(kFewRanks, l.r - j0), tile.count, kFewTokens + 1, gridDim.y,
                [&](int j, int i, float s) { out[(int64_t)i * l.r + j] = f * s; });
}

// out rows of a tile, 64 columns a warp; v enters as two bf16 parts.  D[n, token] = sum_j W[j, n] v[token, j]:
// an MMA's two row halves are the even and odd columns of a lane's eight, so the
// lane ends with eight consecutive columns of two tokens.
constexpr int kFewCols = 64 * kFewWarps;

__global__ void __launch_bounds__(kFewWarps * 32) few_up_kernel(const LoraArgs l, const float *__restrict__ v,
                                                                const uint16_t *__restrict__ W, int C, bool scaled,
                                                                const uint16_t *base, int64_t bs, uint16_t *out,
                                                                int64_t os)
{
    constexpr int kRow = GEMMAR_LORA_MAX_RANK / 2 + 4;   // pairs of a token, padded off the banks
    __shared__ uint32_t hi[kFewTokens][kRow], lo[kFewTokens][kRow];
    const Tile tile = find_tile(l, blockIdx.y, kFewTokens, base != out);
    if (tile.of == 0)
        return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int rank = tile.a < l.R ? rank_of(l, tile.a) : 0, steps = (rank + 15) / 16;
    const int n0 = blockIdx.x * kFewCols + warp * 64 + g * 8;
    const bool in = n0 < C;
    const uint16_t *w0 = W + (int64_t)min(tile.a, l.R - 1) * l.r * C + n0;
    auto load = [&](int s, uint4 (&w)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = s * 16 + q * 2 + (i & 1) + (i >> 1) * 8;
            w[i] = make_uint4(0, 0, 0, 0);
            if (in && j < rank)
                w[i] = __ldg(reinterpret_cast<const uint4 *>(w0 + (int64_t)j * C));
        }
    };
    uint4 w[4];
    load(0, w);   // in flight while v is read
    const int pairs = steps * 8;
    for (int e = threadIdx.x; e < kFewTokens * pairs; e += kFewWarps * 32) {
        const int i = e / pairs, p = e - i * pairs;
        const float *src = v + (int64_t)(tile.i0 + i) * l.r + 2 * p;
        const float v0 = i < tile.count && 2 * p < rank ? __ldg(src) : 0.0f;
        const float v1 = i < tile.count && 2 * p + 1 < rank ? __ldg(src + 1) : 0.0f;
        const uint32_t h = bf16x2_from_f32(v0, v1);
        hi[i][p] = h;
        lo[i][p] = bf16x2_from_f32(v0 - __uint_as_float(h << 16), v1 - __uint_as_float(h & 0xFFFF0000u));
    }
    __syncthreads();
    float acc[4][4][4] = {};   // column pair, token tile, fragment
    const int nt = (tile.count + 7) / 8;
    for (int s = 0; s < steps; ++s) {
        uint4 next[4];
        load(s + 1, next);
        const uint32_t rows[4][4] = {{w[0].x, w[0].y, w[0].z, w[0].w}, {w[1].x, w[1].y, w[1].z, w[1].w},
                                     {w[2].x, w[2].y, w[2].z, w[2].w}, {w[3].x, w[3].y, w[3].z, w[3].w}};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n < nt) {
                const int i = n * 8 + g;
                const uint32_t h0 = hi[i][s * 8 + q], h1 = hi[i][s * 8 + 4 + q];
                const uint32_t l0 = lo[i][s * 8 + q], l1 = lo[i][s * 8 + 4 + q];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t a[4] = {__byte_perm(rows[0][c], rows[1][c], 0x5410), __byte_perm(rows[0][c], rows[1][c], 0x7632),
                                           __byte_perm(rows[2][c], rows[3][c], 0x5410), __byte_perm(rows[2][c], rows[3][c], 0x7632)};
                    mma_bf16(acc[c][n], a, h0, h1);
                    mma_bf16(acc[c][n], a, l0, l1);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = next[i];
    }
    if (!in)
        return;
    const float f = scaled && tile.a < l.R ? l.scales[tile.a] : 1.0f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = n * 8 + q * 2 + k;
            const int t = i < tile.count ? __ldg(l.order + tile.i0 + i) : -1;
            if (t < 0 || t >= l.T)
                continue;
            uint4 y = make_uint4(0, 0, 0, 0);
            if (base)
                y = *reinterpret_cast<const uint4 *>(base + t * bs + n0);
            if (rank > 0) {
                uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    yw[c] = bf16x2_from_f32(fmaf(f, acc[c][n][k], __uint_as_float(yw[c] << 16)),
                                            fmaf(f, acc[c][n][2 + k], __uint_as_float(yw[c] & 0xFFFF0000u)));
            }
            *reinterpret_cast<uint4 *>(out + t * os + n0) = y;
        }
    }
}

}  // namespace

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

cudaError_t launch_lora_down(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const uint16_t *W,
                             int C, bool scaled, float *v, cudaStream_t st)
{
    if (l.T > kFewBatch)
        return launch_tile_down(l, p, x, xs, W, C, scaled, v, st);
    // two CTAs an SM, a block of 32 columns a warp at least
    const int64_t tiles = most_tiles(l.T, l.R, kFewTokens, false);
    const int rank_blocks = (l.r + kFewRanks - 1) / kFewRanks;
    const int64_t want = std::min<int64_t>({2 * (int64_t)p.num_sms / (tiles * rank_blocks), (C + 31) / 32 / kFewWarps, kMaxSplits});
    const int splits = (int)std::max<int64_t>(1, want);
    return launch_split(few_down_kernel, dim3((unsigned)tiles, splits, rank_blocks), kFewWarps * 32, 0, splits, st, l, x, xs,
                        W, C, scaled, v);
}

cudaError_t launch_lora_up(const LoraArgs &l, const LoraCall &p, const float *v, const uint16_t *W, int C,
                           bool scaled, const uint16_t *base, int64_t bs, uint16_t *out, int64_t os, cudaStream_t st)
{
    if (l.T > kFewBatch)
        return launch_tile_up(l, p, v, W, C, scaled, base, bs, out, os, st);
    const dim3 grid((C + kFewCols - 1) / kFewCols, (unsigned)most_tiles(l.T, l.R, kFewTokens, base != out));
    few_up_kernel<<<grid, kFewWarps * 32, 0, st>>>(l, v, W, C, scaled, base, bs, out, os);
    return cudaGetLastError();
}

}  // namespace gemmar

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
// the weights are what is read, and latency is what counts.  One launch does both
// products: a cluster takes 8 tokens of one adapter (the N of one MMA), its CTAs share
// the columns of the first product, exchange v through distributed shared memory, and
// share the columns of the second, whose weights they have meanwhile asked into L2.
// r = 16, N = 7168: one token, K = 2048, 6.8 us; 96 tokens of 48 adapters, K = 16384, 12.6 us
// for 42 MB, 3.3 TB/s.  What bounds it is the chain of trips to memory: the plan, the
// first weights, the exchange, the second weights, the stores.
//
// Fragments are loaded straight from memory into registers, 16 bytes a lane, no
// staging: the contraction index of an MMA may be permuted as long as both
// operands agree, so lane (g, q) takes eight consecutive elements of its row for
// two MMAs.  Weights are the M operand, tokens the N operand.

constexpr int kFewTokens = 8;    // tokens a tile: one N tile
constexpr int kFewWarps = 8;
constexpr int kFewRanks = 32;    // ranks at a time in the first product: two M tiles
constexpr int kPairRow = GEMMAR_LORA_MAX_RANK / 2 + 4;   // rank pairs of a token, padded off the banks

struct FewSmem {
    float part[GEMMAR_LORA_MAX_RANK][kFewTokens + 1];   // this CTA's sums
    union {
        float sums[kFewWarps][kFewRanks][kFewTokens + 1];
        struct {
            uint32_t hi[kFewTokens][kPairRow], lo[kFewTokens][kPairRow];
        } v;
    };
};

// One product's weights [R, r, C], and what its result is scaled by.
struct Factor {
    const uint16_t *W;
    int C;
    bool scaled;
};

// Sums of 16 MT ranks from j0 over the warp's share of the columns into sums[rank][token];
// t: the token of lane >> 2, or -1.
template <int MT>
__device__ __forceinline__ void few_down(const LoraArgs &l, const Tile &tile, int rank, int j0, const Factor &f,
                                         const uint16_t *__restrict__ x, int64_t xs, int t,
                                         float (&sums)[kFewRanks][kFewTokens + 1])
{
    constexpr int kUnroll = MT == 1 ? 8 : 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint16_t *wr[2 * MT];   // rows j0 + g, + 8, ...
    bool wok[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        const int j = j0 + g + 8 * i;
        wok[i] = j < rank;
        wr[i] = f.W + ((int64_t)tile.a * l.r + (wok[i] ? j : 0)) * f.C + q * 8;
    }
    const bool xok = t >= 0;
    const uint16_t *xr = x + (xok ? t : 0) * xs + q * 8;
    // blocks of 32 columns, dealt evenly to the cluster's warps
    const int blocks = (f.C + 31) / 32, shares = gridDim.y * kFewWarps, share = blockIdx.y * kFewWarps + warp;
    const int b0 = (int)((int64_t)blocks * share / shares), b1 = (int)((int64_t)blocks * (share + 1) / shares);
    float acc[MT][4] = {};
    auto block = [&](int b, bool in) {
        uint4 w[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
            w[i] = in && wok[i] ? __ldg(reinterpret_cast<const uint4 *>(wr[i] + b * 32)) : make_uint4(0, 0, 0, 0);
        const uint4 xv = in && xok ? __ldg(reinterpret_cast<const uint4 *>(xr + b * 32)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t lo[4] = {w[2 * m].x, w[2 * m + 1].x, w[2 * m].y, w[2 * m + 1].y};
            const uint32_t hi[4] = {w[2 * m].z, w[2 * m + 1].z, w[2 * m].w, w[2 * m + 1].w};
            mma_bf16(acc[m], lo, xv.x, xv.y);
            mma_bf16(acc[m], hi, xv.z, xv.w);
        }
    };
    int b = b0;
    for (; b + kUnroll <= b1 && (b + kUnroll) * 32 <= f.C; b += kUnroll) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            block(b + k, true);
    }
    for (; b < b1; ++b)
        block(b, b * 32 + q * 8 < f.C);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sums[m * 16 + g + (e >> 1) * 8][q * 2 + (e & 1)] = acc[m][e];
}

// out rows of a tile, 64 columns a warp at a time; v enters as two bf16 parts.
// D[n, token] = sum_j W[j, n] v[token, j]: an MMA's two row halves are the even and odd
// columns of a lane's eight, so the lane ends with eight consecutive columns of two
// tokens.
__device__ __forceinline__ void few_up(const LoraArgs &l, const Tile &tile, int rank, const Factor &f, const FewSmem &sm,
                                       const uint16_t *base, int64_t bs, uint16_t *out, int64_t os)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int steps = (rank + 15) / 16;
    const float scale = f.scaled && tile.a < l.R ? l.scales[tile.a] : 1.0f;
    int tok[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = q * 2 + k, t = i < tile.count ? __ldg(l.order + tile.i0 + i) : -1;
        tok[k] = t >= 0 && t < l.T ? t : -1;
    }
    for (int b = blockIdx.y * kFewWarps + warp; b * 64 < f.C; b += gridDim.y * kFewWarps) {
        const int n0 = b * 64 + g * 8;
        const bool in = n0 < f.C;
        const uint16_t *w0 = f.W + (int64_t)min(tile.a, l.R - 1) * l.r * f.C + n0;
        auto load = [&](int s, uint4 (&w)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = s * 16 + q * 2 + (i & 1) + (i >> 1) * 8;
                w[i] = in && j < rank ? __ldg(reinterpret_cast<const uint4 *>(w0 + (int64_t)j * f.C)) : make_uint4(0, 0, 0, 0);
            }
        };
        uint4 w[4], y[2];
        load(0, w);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            y[k] = base && in && tok[k] >= 0 ? *reinterpret_cast<const uint4 *>(base + tok[k] * bs + n0) : make_uint4(0, 0, 0, 0);
        float acc[4][4] = {};   // column pair, fragment
        for (int s = 0; s < steps; ++s) {
            uint4 next[4];
            load(s + 1, next);
            const uint32_t rows[4][4] = {{w[0].x, w[0].y, w[0].z, w[0].w}, {w[1].x, w[1].y, w[1].z, w[1].w},
                                         {w[2].x, w[2].y, w[2].z, w[2].w}, {w[3].x, w[3].y, w[3].z, w[3].w}};
            const uint32_t h0 = sm.v.hi[g][s * 8 + q], h1 = sm.v.hi[g][s * 8 + 4 + q];
            const uint32_t l0 = sm.v.lo[g][s * 8 + q], l1 = sm.v.lo[g][s * 8 + 4 + q];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t a[4] = {
                    __byte_perm(rows[0][c], rows[1][c], 0x5410), __byte_perm(rows[0][c], rows[1][c], 0x7632),
                    __byte_perm(rows[2][c], rows[3][c], 0x5410), __byte_perm(rows[2][c], rows[3][c], 0x7632)};
                mma_bf16(acc[c], a, h0, h1);
                mma_bf16(acc[c], a, l0, l1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = next[i];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!in || tok[k] < 0)
                continue;
            uint32_t yw[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
            if (rank > 0) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    yw[c] = bf16x2_from_f32(fmaf(scale, acc[c][k], __uint_as_float(yw[c] << 16)),
                                            fmaf(scale, acc[c][2 + k], __uint_as_float(yw[c] & 0xFFFF0000u)));
            }
            *reinterpret_cast<uint4 *>(out + tok[k] * os + n0) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
        }
    }
}

__global__ void __launch_bounds__(kFewWarps * 32, 3) few_kernel(const LoraArgs l, const uint16_t *__restrict__ x, int64_t xs,
                                                              const Factor down, const Factor up, const uint16_t *base,
                                                              int64_t bs, uint16_t *out, int64_t os, float *v_out, const Halves halves)
{
    __shared__ FewSmem sm;
    const Tile tile = find_tile(l, blockIdx.x, kFewTokens, base != out);
    if (tile.of == 0)
        return;
    grid_launch_next();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = tile.a < l.R ? rank_of(l, tile.a) : 0, ctas = gridDim.y;
    const int pairs = (rank + 15) / 16 * 8;
    int t = (lane >> 2) < tile.count ? __ldg(l.order + tile.i0 + (lane >> 2)) : -1;
    t = t < l.T ? t : -1;
    // the 128-byte pieces of the second product's operands that this warp will read
    for (int b = blockIdx.y * kFewWarps + warp; b * 64 < up.C; b += ctas * kFewWarps) {
        for (int j = lane; j < rank; j += 32)
            prefetch_l2(up.W + ((int64_t)tile.a * l.r + j) * up.C + b * 64);
        if (base && (lane & 3) == 0 && t >= 0)
            prefetch_l2(base + t * bs + b * 64);
    }
    for (int j0 = 0; j0 < rank; j0 += kFewRanks) {
        if (rank - j0 > 16)
            few_down<2>(l, tile, rank, j0, down, x, xs, t, sm.sums[warp]);
        else
            few_down<1>(l, tile, rank, j0, down, x, xs, t, sm.sums[warp]);
        __syncthreads();
        const int nj = min(kFewRanks, rank - j0);
        for (int e = tid; e < nj * tile.count; e += kFewWarps * 32) {
            const int j = e / tile.count, i = e - j * tile.count;
            float s = sm.sums[0][j][i];
#pragma unroll
            for (int w = 1; w < kFewWarps; ++w)
                s += sm.sums[w][j][i];
            sm.part[j0 + j][i] = s;
        }
        __syncthreads();
    }
    if (rank > 0) {
        if (ctas > 1)
            cluster_sync();
        // v, in rank order, by every CTA for itself
        const float f = down.scaled ? l.scales[tile.a] : 1.0f;
        for (int e = tid; e < kFewTokens * pairs; e += kFewWarps * 32) {
            const int i = e / pairs, p = e - i * pairs;
            float v[2] = {0.0f, 0.0f}, part[2][kMaxSplits];
#pragma unroll
            for (int k = 0; k < 2; ++k) {   // all on their way before the first is added
                const uint32_t at = smem_u32(&sm.part[2 * p + k][i]);
#pragma unroll
                for (int c = 0; c < kMaxSplits; ++c)
                    part[k][c] = c < ctas && i < tile.count && 2 * p + k < rank ? ld_shared_cluster_f32(mapa_shared(at, c)) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = 2 * p + k;
#pragma unroll
                for (int c = 0; c < kMaxSplits; ++c)
                    v[k] += part[k][c];
                v[k] = j < rank ? v[k] * f : 0.0f;
                if (blockIdx.y == 0 && i < tile.count) {
                    if (v_out && j < l.r)
                        v_out[(int64_t)(tile.i0 + i) * l.r + j] = v[k];
                    put_pair(halves, tile.i0 + i, j, l.r, v[k]);
                }
            }
            const uint32_t h = high_halves(v[0], v[1]);
            sm.v.hi[i][p] = h;
            sm.v.lo[i][p] = bf16x2_from_f32(v[0] - __uint_as_float(h << 16), v[1] - __uint_as_float(h & 0xFFFF0000u));
        }
        if (ctas > 1)
            cluster_arrive();   // its sums have been read
    }
    if (blockIdx.y == 0 && tile.a < l.R) {   // columns past the rank's last step
        const int rest = pad_rank(l.r) - 2 * pairs;
        for (int e = tid; e < tile.count * rest; e += kFewWarps * 32) {
            const int i = tile.i0 + e / rest, j = 2 * pairs + e % rest;
            if (v_out && j < l.r)
                v_out[(int64_t)i * l.r + j] = 0.0f;
            put_pair(halves, i, j, l.r, 0.0f);
        }
    }
    __syncthreads();
    few_up(l, tile, rank, up, sm, base, bs, out, os);
    if (rank > 0 && ctas > 1)
        cluster_wait();   // no CTA leaves while another reads its sums
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

namespace {

// Few tokens an adapter: its weights are read again for every eight of them, from L2 after
// the first, which costs T r and beats the tensor-core tiles up to here (K = 2048 or 16384,
// N = 7168; this kernel against the tiles): T = 64 of 16 adapters, r = 16, 8 us against 16;
// 512 of 64, 25 against 68; 1024 of 32, 22 against 28; 2048 of 256, 45 against 106; and past
// the rule, 256 of 8 with r = 64, 26 against 16.  All for tokens spread evenly over the R
// adapters: how many of them have tokens is known on the device alone, and a few of many
// take this kernel past where it pays (2048 tokens of 4 adapters, r = 64, K = 2048: 29 us
// with R = 4, 98 with R = 1024).
bool few(const LoraArgs &l) { return l.T <= 4096 && l.T * l.r <= 1024 * (int64_t)l.R; }

cudaError_t launch_few(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const Factor &down,
                       const Factor &up, const uint16_t *base, int64_t bs, uint16_t *out, int64_t os, float *v,
                       const Halves &halves, cudaStream_t st)
{
    // clusters as large as fill the SMs, of which three CTAs each, were all tiles there are
    // to be half of the most there can be
    const int64_t tiles = most_tiles(l.T, l.R, kFewTokens, base != out);
    int ctas = kMaxSplits;
    while (ctas > 1 && tiles * ctas > 4 * p.num_sms)
        ctas /= 2;
    return launch(few_kernel, dim3((unsigned)tiles, ctas), kFewWarps * 32, 0, ctas, false, st, l, x, xs, down, up, base, bs,
                  out, os, v, halves);
}

}  // namespace

#define TRY(x)                           \
    do {                                 \
        const cudaError_t e_ = (x);      \
        if (e_ != cudaSuccess)           \
            return e_;                   \
    } while (0)

int64_t lora_apply_floats(const LoraArgs &l) { return few(l) ? 0 : l.T * pad_rank(l.r); }

cudaError_t launch_lora_apply(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const uint16_t *A, int K,
                              const uint16_t *B, int N, const uint16_t *y, int64_t ys, uint16_t *out, int64_t os, float *v,
                              float *ws, cudaStream_t st)
{
    if (few(l))
        return launch_few(l, p, x, xs, Factor{A, K, false}, Factor{B, N, true}, y, ys, out, os, v, Halves{}, st);
    const Halves h = lora_halves(nullptr, l.T, l.r, ws);
    TRY(launch_tile_down(l, p, x, xs, A, K, false, v, h, st));
    return launch_tile_up(l, p, h.w2, B, N, true, y, ys, out, os, st);
}

cudaError_t launch_lora_apply_bwd(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const uint16_t *dy,
                                  int64_t dys, const uint16_t *A, int K, const uint16_t *B, int N, const float *v,
                                  const uint16_t *dx0, int64_t dx0s, uint16_t *dx, int64_t dxs, uint16_t *dA, uint16_t *dB,
                                  float *ws, int64_t ws_floats, cudaStream_t st)
{
    const Halves h = lora_halves(v, l.T, l.r, ws);
    const GradCall g = lora_grad_call(l, p, h, x, xs, K, dA, dy, dys, N, dB, ws, ws_floats);
    if (few(l)) {
        TRY(launch_few(l, p, dy, dys, Factor{B, N, true}, Factor{A, K, false}, dx0, dx0s, dx, dxs, nullptr, h, st));
        TRY(launch_tile_grad(l, p, g, st));
    } else {
        // the weight gradients and dx need only w, but each launch waits for the one before it
        TRY(launch_tile_down(l, p, dy, dys, B, N, true, nullptr, h, st));
        TRY(launch_tile_grad(l, p, g, st));
        TRY(launch_tile_up(l, p, h.w2, A, K, false, dx0, dx0s, dx, dxs, st));
    }
    return launch_grad_join(l, p, g, st);
}

}  // namespace gemmar

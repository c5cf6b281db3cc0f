// lora.cuh -- what the adapter kernels share: ranks, and the tiles of tokens.
#pragma once

#include "kernels.h"
#include "launch.cuh"

namespace gemmar {

__device__ __forceinline__ int rank_of(const LoraArgs &l, int a)
{
    return l.ranks ? min(max(l.ranks[a], 0), l.r) : l.r;
}

// A CTA's share of the tokens: positions [i0, i0 + count) of adapter a (a == R:
// tokens without one), its tile `index` of `of`.
struct Tile {
    int a, i0, count, index, of;
};

// Where group g's positions begin (g == R: the tokens without an adapter; R + 1: T).
__device__ __forceinline__ int group_begin(const LoraArgs &l, int g)
{
    const int T = (int)l.T;
    return g > l.R ? T : min(max(__ldg(l.offsets + g), 0), T);
}

// Tile number `want` when every adapter's tokens (and, with `bare`, those without
// one) are cut into tiles of `size`, an adapter without tokens into `least` (0 or 1)
// empty ones; of == 0 past the last.  Warp-collective: lane l counts the tiles of a
// contiguous share of the adapters, a scan finds the lane.
__device__ __forceinline__ Tile find_tile(const LoraArgs &l, int want, int size, bool bare, int least = 0)
{
    const int lane = threadIdx.x & 31, groups = l.R + (bare ? 1 : 0);
    const int per = (groups + 31) / 32, g0 = min(lane * per, groups), g1 = min(g0 + per, groups);
    auto cut = [&](int n) { return max(least, (max(n, 0) + size - 1) / size); };
    int tiles = 0, at = group_begin(l, g0);
    for (int g = g0; g < g1; ++g) {
        const int next = group_begin(l, g + 1);
        tiles += cut(next - at);
        at = next;
    }
    int before = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o)
            before += up;
    }
    before -= tiles;
    const unsigned here = __ballot_sync(0xFFFFFFFFu, want >= before && want < before + tiles);
    Tile t{0, 0, 0, 0, 0};
    if (here == 0u)
        return t;
    const int owner = __ffs(here) - 1;
    if (lane == owner) {
        int rest = want - before;
        at = group_begin(l, g0);
        for (int g = g0; g < g1; ++g) {
            const int next = group_begin(l, g + 1), n = cut(next - at);
            if (rest < n) {
                t = Tile{g, at + rest * size, min(size, max(next - at, 0) - rest * size), rest, n};
                break;
            }
            rest -= n;
            at = next;
        }
    }
    t.a = __shfl_sync(0xFFFFFFFFu, t.a, owner);
    t.i0 = __shfl_sync(0xFFFFFFFFu, t.i0, owner);
    t.count = __shfl_sync(0xFFFFFFFFu, t.count, owner);
    t.index = __shfl_sync(0xFFFFFFFFu, t.index, owner);
    t.of = __shfl_sync(0xFFFFFFFFu, t.of, owner);
    return t;
}

// Tiles of `size` that the adapters before `a` with more than one tile have (warp-collective).
__device__ __forceinline__ int split_tiles_before(const LoraArgs &l, int a, int size)
{
    int n = 0;
    for (int g = threadIdx.x & 31; g < a; g += 32) {
        const int c = (max(group_begin(l, g + 1) - group_begin(l, g), 0) + size - 1) / size;
        n += c > 1 ? c : 0;
    }
    return __reduce_add_sync(0xFFFFFFFFu, n);
}

constexpr int kMaxSplits = 8;   // CTAs of a cluster

// Sum over the CTAs of the cluster, in the order of their ranks, of the fp32 array
// [rows][cols] that each has at the same shared-memory address, rows `pitch` floats
// apart; put(row, col, sum) is called for every four columns by one thread of one of
// them.  The whole cluster calls it, after its threads have written the array.
template <typename Put>
__device__ __forceinline__ void cluster_sum(uint32_t array, int rows, int cols, int pitch, int ctas, Put put)
{
    if (ctas == 1)
        __syncthreads();
    else
        ptx::cluster_sync();
    const int me = ctas == 1 ? 0 : (int)ptx::cluster_ctarank(), share = (rows + ctas - 1) / ctas, quads = cols / 4;
    const int lo = me * share, n = max(0, min(share, rows - lo)) * quads;
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
        const int row = lo + e / quads, col = e % quads * 4;
        const uint32_t at = array + (row * pitch + col) * 4;
        // all on their way before the first is added
        float4 a[kMaxSplits];
#pragma unroll
        for (int p = 0; p < kMaxSplits; ++p)
            a[p] = p < ctas ? ptx::ld_shared_cluster_f32x4(ptx::mapa_shared(at, p)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float4 s = a[0];
#pragma unroll
        for (int p = 1; p < kMaxSplits; ++p) {
            s.x += a[p].x; s.y += a[p].y; s.z += a[p].z; s.w += a[p].w;
        }
        put(row, col, s);
    }
    if (ctas > 1)
        ptx::cluster_sync();   // no CTA leaves while another reads its array
}


// A product's inner factor in two bf16 parts, x = hi + lo to 2^-16 of x: [T][RP hi, RP lo]
// with RP the padded rank, 0 past the rank.  hi stays finite: rounded to infinity it would
// leave lo = x - hi the opposite one, or NaN; so lo alone is infinite where x is.  `v` and `v2`: the backward pass has the
// forward pass's v [T, r] split on the way; nullptr: not asked for.
struct Halves {
    uint16_t *w2;
    const float *v;
    uint16_t *v2;
    int RP;
};

__device__ __forceinline__ float finite_bf16(float x)
{
    constexpr float kMost = 0x1.FEp127f;
    return fminf(fmaxf(x, -kMost), kMost);
}

// hi of two values
__device__ __forceinline__ uint32_t high_halves(float a, float b) { return ptx::bf16x2_from_f32(finite_bf16(a), finite_bf16(b)); }

__device__ __forceinline__ void put_halves(uint16_t *row, int RP, int j, float x)
{
    const uint32_t p = high_halves(x, x) & 0xFFFFu;
    row[j] = (uint16_t)p;
    row[RP + j] = (uint16_t)(ptx::bf16x2_from_f32(x - __uint_as_float(p << 16), 0.0f) & 0xFFFFu);
}

// Element (i, j) of both, i a position, w its value; j runs over the padded rank.
__device__ __forceinline__ void put_pair(const Halves &h, int64_t i, int j, int r, float w)
{
    if (h.w2)
        put_halves(h.w2 + i * 2 * h.RP, h.RP, j, w);
    if (h.v2)
        put_halves(h.v2 + i * 2 * h.RP, h.RP, j, j < r ? __ldg(h.v + i * r + j) : 0.0f);
}

__device__ __forceinline__ void put_halves4(uint16_t *row, int RP, int j, const float4 &x)
{
    const uint32_t a = high_halves(x.x, x.y), b = high_halves(x.z, x.w);
    *reinterpret_cast<uint2 *>(row + j) = make_uint2(a, b);
    *reinterpret_cast<uint2 *>(row + RP + j) =
        make_uint2(ptx::bf16x2_from_f32(x.x - __uint_as_float(a << 16), x.y - __uint_as_float(a & 0xFFFF0000u)),
                   ptx::bf16x2_from_f32(x.z - __uint_as_float(b << 16), x.w - __uint_as_float(b & 0xFFFF0000u)));
}

// The same for j .. j + 3, j a multiple of four.
__device__ __forceinline__ void put_pair4(const Halves &h, int64_t i, int j, int r, const float4 &w)
{
    if (h.w2)
        put_halves4(h.w2 + i * 2 * h.RP, h.RP, j, w);
    if (h.v2) {
        const float *v = h.v + i * r + j;
        put_halves4(h.v2 + i * 2 * h.RP, h.RP, j,
                    make_float4(j < r ? __ldg(v) : 0.0f, j + 1 < r ? __ldg(v + 1) : 0.0f, j + 2 < r ? __ldg(v + 2) : 0.0f,
                                j + 3 < r ? __ldg(v + 3) : 0.0f));
    }
}

__host__ __device__ constexpr int pad_rank(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

// Most tiles of `size` that T tokens of R adapters (and the bare ones) can make.
inline int64_t most_tiles(int64_t T, int R, int size, bool bare)
{
    const int64_t groups = R + (bare ? 1 : 0);
    return T / size + (groups < T ? groups : T);
}

// One weight gradient: G[a,j,c] = f sum_i p[i,j] x[order[i],c], p from its halves.
struct GradSide {
    const uint16_t *x;    // tokens' rows
    int64_t xs;
    int C, scaled;
    const uint16_t *p2;   // [T][2 RP]
    uint16_t *G;
    float *part;          // [split tile][r][C]
};

// Both of a call, the tokens a tile, and the split tiles that the scratch has room for:
// enough for any plan, which offsets that are none could still exceed.
struct GradCall {
    GradSide A, B;
    int RP, size, slots;
};

// The launches of lora_tile.cu.
cudaError_t launch_tile_down(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const uint16_t *W,
                             int C, bool scaled, float *v, const Halves &halves, cudaStream_t st);
cudaError_t launch_tile_up(const LoraArgs &l, const LoraCall &p, const uint16_t *v2, const uint16_t *W, int C, bool scaled,
                           const uint16_t *base, int64_t bs, uint16_t *out, int64_t os, cudaStream_t st);
Halves lora_halves(const float *v, int64_t T, int r, float *ws);
GradCall lora_grad_call(const LoraArgs &l, const LoraCall &p, const Halves &h, const uint16_t *x, int64_t xs, int K,
                        uint16_t *dA, const uint16_t *dy, int64_t ys, int N, uint16_t *dB, float *ws, int64_t ws_floats);
cudaError_t launch_tile_grad(const LoraArgs &l, const LoraCall &p, const GradCall &g, cudaStream_t st);
cudaError_t launch_grad_join(const LoraArgs &l, const LoraCall &p, const GradCall &g, cudaStream_t st);

}  // namespace gemmar

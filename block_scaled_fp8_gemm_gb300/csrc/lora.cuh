// lora.cuh -- what the adapter kernels share: ranks, and the tiles of tokens.
#pragma once

#include "kernels.h"

namespace gemmar {

__device__ __forceinline__ int rank_of(const LoraArgs &l, int a)
{
    return l.ranks ? min(max(l.ranks[a], 0), l.r) : l.r;
}

// A CTA's share of the tokens: positions [i0, i0 + count) of adapter a (a == R:
// tokens without one).
struct Tile {
    int a, i0, count;
};

// Tile number `want` when every adapter's tokens (and, with `bare`, those without
// one) are cut into tiles of `size`; count 0 past the last.  Warp-collective: lane l
// counts the tiles of a contiguous share of the adapters, a scan finds the lane.
__device__ __forceinline__ Tile find_tile(const LoraArgs &l, int want, int size, bool bare)
{
    const int lane = threadIdx.x & 31, groups = l.R + (bare ? 1 : 0), T = (int)l.T;
    const int per = (groups + 31) / 32, g0 = min(lane * per, groups), g1 = min(g0 + per, groups);
    auto edge = [&](int g) { return g > l.R ? T : min(max(__ldg(l.offsets + g), 0), T); };
    int tiles = 0, at = edge(g0);
    for (int g = g0; g < g1; ++g) {
        const int next = edge(g + 1);
        tiles += (max(next - at, 0) + size - 1) / size;
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
    Tile t{0, 0, 0};
    if (here == 0u)
        return t;
    const int owner = __ffs(here) - 1;
    if (lane == owner) {
        int rest = want - before;
        at = edge(g0);
        for (int g = g0; g < g1; ++g) {
            const int next = edge(g + 1), n = (max(next - at, 0) + size - 1) / size;
            if (rest < n) {
                t.a = g;
                t.i0 = at + rest * size;
                t.count = min(size, next - t.i0);
                break;
            }
            rest -= n;
            at = next;
        }
    }
    t.a = __shfl_sync(0xFFFFFFFFu, t.a, owner);
    t.i0 = __shfl_sync(0xFFFFFFFFu, t.i0, owner);
    t.count = __shfl_sync(0xFFFFFFFFu, t.count, owner);
    return t;
}

// Most tiles of `size` that T tokens of R adapters (and the bare ones) can make.
inline int64_t most_tiles(int64_t T, int R, int size, bool bare)
{
    const int64_t groups = R + (bare ? 1 : 0);
    return T / size + (groups < T ? groups : T);
}

}  // namespace gemmar

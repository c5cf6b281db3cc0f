// lora_tile.cu -- the adapter products for many tokens, on the tensor cores: tiles
// of 128 tokens of one adapter, tcgen05 MMAs (kind::f16, bf16 operands, fp32 sums in
// TMEM).  The tokens' rows are gathered by cp.async into 128-byte-swizzled tiles;
// every thread copies, one thread issues the MMAs.
//
// A rank r contraction does 2r flops for every element it reads, below the 283
// flops a byte of the tensor peak over the copy rate even at r = 128: the tokens'
// rows are what bounds these kernels, and the low-rank side costs little enough to
// enter as two bf16 parts (its rounding error then is 2^-16; the result's own, one
// bf16 rounding, is 2^-8, and its distance from the 64-bit value is that of the same
// formula in fp32).
#include <cuda_bf16.h>

#include <algorithm>

#include "gemmar.h"
#include "lora.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kRows = 128;      // tokens a tile, rows of the accumulator
constexpr int kSw = 1024;       // a swizzle atom: 8 rows of 128 bytes

// 16-byte chunk c of row `row` in a tile of 128-byte rows under the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

__device__ __forceinline__ uint8_t *align_1024(uint8_t *p)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

struct Waits {
    DevStatus *status;
    uint64_t timeout_ns;
};

// Bounded: after a wait that ran out (or another thread's) the kernel goes on to its
// end without waiting, its result is void and the status word says so.
__device__ __forceinline__ void wait_mma(uint64_t *bar, uint32_t parity, volatile int *abort, const Waits &w)
{
    mbar_wait(bar, parity, abort, w.status, w.timeout_ns, SITE_LORA_MMA);
    tc_fence_after();
}

__host__ __device__ constexpr int tmem_cols(int n) { return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512; }

// ---------------------------------------------------------------- down

// v[i][j] = f sum_c x[t,c] W[a,j,c]: D[128 tokens, ranks], both operands K-major, 64
// columns a stage.  The CTAs of a cluster share the columns of a tile (blockIdx.y) and
// add their sums in rank order through distributed shared memory.
// Bound by the reads of x: 87 us for the 483 MB of 14746 tokens, K = 16384, r = 64, 5.6 TB/s;
// of that 19 us do not depend on K (launch, first stages, the cluster's sum), the rest
// runs at 6.8 TB/s.  A TMA gather of four rows a copy takes 155 us (128 bytes of a row at
// a time leave it at 20 bytes a ns and SM), TMA boxes of neighbouring rows 86.
constexpr int kDownThreads = 256;

template <int RP>   // ranks rounded up to 16, 32, 64 or 128
struct DownCfg {
    static constexpr int kX = kRows * 128, kW = RP * 128, kStage = kX + kW;
    static constexpr int kCtas = RP <= 64 ? 3 : 2;   // an SM
    static constexpr int kStages = RP == 16 ? 4 : 3;
    static constexpr int kSmem = kStages * kStage + 1024;
};

template <int RP>
__global__ void __launch_bounds__(kDownThreads, DownCfg<RP>::kCtas) tile_down_kernel(const LoraArgs l, const uint16_t *__restrict__ x,
                                                                 int64_t xs, const uint16_t *__restrict__ W, int C,
                                                                 bool scaled, float *__restrict__ v, const Halves halves, int cols, const Waits waits)
{
    using Cfg = DownCfg<RP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t done[Cfg::kStages];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const Tile tile = find_tile(l, blockIdx.x, kRows, false);
    if (tile.of == 0)
        return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *smem = align_1024(smem_raw);
    const uint32_t base = smem_u32(smem);
    const int rank = rank_of(l, tile.a);
    if (tid == 0) {
        for (int s = 0; s < Cfg::kStages; ++s)
            mbar_init(done + s, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_slot, tmem_cols(RP));
        tmem_relinquish();
    }
    // this thread's chunk of every stage: column chunk tid & 7 of rows tid / 8 + 32 i
    const int ch = tid & 7, row0 = tid >> 3;
    const uint16_t *xr[4];
    bool xok[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = row0 + 32 * i;
        const int t = p < tile.count ? __ldg(l.order + tile.i0 + p) : -1;
        xok[i] = t >= 0 && t < l.T;
        xr[i] = x + (xok[i] ? t : 0) * xs;
    }
    const int c_lo = blockIdx.y * cols, c_hi = min(c_lo + cols, C);
    const int steps = (c_hi - c_lo + 63) / 64;
    // rows 32 apart are 4096 bytes apart in a stage and share their swizzle
    const uint32_t at_x = sw128(row0, ch);
    const uint16_t *wr = W + ((int64_t)tile.a * l.r + row0) * C;
    int c = c_lo + ch * 8;   // of the next step
    auto fetch = [&](int s) {
        if (s < steps) {
            const uint32_t st = base + (s % Cfg::kStages) * Cfg::kStage + at_x;
            const bool in = c < c_hi;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cp_async_cg16_or_zero(st + i * 4096, in && xok[i] ? xr[i] + c : x, in && xok[i]);
#pragma unroll
            for (int j = 0; j < RP; j += 32) {
                if (RP >= 32 || row0 < RP) {
                    const bool ok = in && row0 + j < rank;
                    cp_async_cg16_or_zero(st + Cfg::kX + j * 128, ok ? wr + (int64_t)j * C + c : W, ok);
                }
            }
            c += 64;
        }
        cp_async_commit();
    };
    for (int s = 0; s < Cfg::kStages - 1; ++s)
        fetch(s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t d = tmem_slot;
    grid_launch_next();   // not before this CTA has its TMEM: the next kernel's would wait holding theirs
    for (int s = 0; s < steps; ++s) {
        cp_async_wait<Cfg::kStages - 2>();
        fence_async_shared();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            const uint32_t st = base + (s % Cfg::kStages) * Cfg::kStage;
            const uint64_t ad = desc_kmajor_sw128(st), bd = desc_kmajor_sw128(st + Cfg::kX);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma_bf16_ss(d, ad + 2 * k, bd + 2 * k, idesc_bf16(kRows, RP, 0, 0), s > 0 || k > 0);
            tc_commit(done + s % Cfg::kStages);
        }
        // the stage of step s - 1 takes step s + stages - 1
        if (s > 0 && s + Cfg::kStages - 1 < steps)
            wait_mma(done + (s - 1) % Cfg::kStages, ((s - 1) / Cfg::kStages) & 1, &abort_flag, waits);
        fetch(s + Cfg::kStages - 1);
    }
    wait_mma(done + (steps - 1) % Cfg::kStages, ((steps - 1) / Cfg::kStages) & 1, &abort_flag, waits);
    // the stages are free: D goes there for the cluster's sum
    constexpr int kPitch = RP + 4;   // whole 16-byte pieces, a row's off the banks of the next
    static_assert(kRows * kPitch * 4 <= Cfg::kStages * Cfg::kStage, "D fits the stages");
    if (warp < 4) {
        const uint32_t mine = base + (warp * 32 + lane) * kPitch * 4;
#pragma unroll
        for (int j0 = 0; j0 < RP; j0 += 16) {
            uint32_t r[16];
            tmem_ld_x16(d + ((uint32_t)(warp * 32) << 16) + j0, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                st_shared_v4(mine + (j0 + j) * 4, make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]));
        }
    }
    const float f = scaled ? l.scales[tile.a] : 1.0f;
    float *out = v ? v + (int64_t)tile.i0 * l.r : nullptr;
    cluster_sum(base, tile.count, RP, kPitch, gridDim.y, [&](int i, int j, float4 s) {
        // past the rank the product was with zeros, which a NaN or an infinity makes NaN
        s = make_float4(j < rank ? f * s.x : 0.0f, j + 1 < rank ? f * s.y : 0.0f, j + 2 < rank ? f * s.z : 0.0f,
                        j + 3 < rank ? f * s.w : 0.0f);
        if (v) {
            float *o = out + (int64_t)i * l.r + j;
            const float e[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j + k < l.r)
                    o[k] = e[k];
        }
        put_pair4(halves, tile.i0 + i, j, l.r, s);
    });
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_dealloc(d, tmem_cols(RP));
}

// ---------------------------------------------------------------- up

// out[t, c] = base[t, c] + f sum_j v[i, j] W[a, j, c]: D[128 tokens, 64 columns] for 64
// columns a step, A the two bf16 parts of v in TMEM, B the weights' rows (N
// contiguous).  A warp owns 32 tokens: it copies their rows of base ahead into a
// ring of its own, adds its lanes' rows of D there and writes whole 128-byte row
// pieces out of it.  A step is a chain (barrier, MMA, TMEM read, transposition,
// stores) that its own CTA does not overlap; three or four CTAs an SM do, so the
// accumulator is single and the ring short.
// 89 us for the 470 MB of 16384 tokens, N = 7168, r = 64, 5.3 TB/s.  A version of 97 us took 82
// without MMAs and sums, 85 without stores and 60 without either: reads, the chain of a
// step and writes share the time.  mma.sync fragments instead of tcgen05 took 149 where this
// took 95, eight warps a CTA 102 against 96.
// In the backward pass the kernel before this one is tile_grad_kernel, whose results it does
// not read; v2 comes from the one before that.  It waits all the same: its writes are
// promised to be seen only through that wait, which follows the gradient kernel's own.
// Reading v2 at once, beside the gradients, took 42 us instead of 44 for 4096 tokens of rank
// 16, 61 instead of 66 at rank 64, 221 instead of 225 for 8191 (the whole backward pass).
constexpr int kUpThreads = 128;

template <int RP, int RING>   // RING: steps copied ahead
struct UpCfg {
    static constexpr int kCtas = RP == 16 || RING == 2 ? 4 : RP <= 64 ? 3 : 2;   // an SM
    static constexpr int kRing = RING;
    static constexpr int kY = kRows * 128, kW = RP * 128, kStage = kY + kW;
    static constexpr int kSmem = kRing * kStage + 1024;
    static constexpr int kA = 64;                     // TMEM: the accumulator, then hi, lo
    static constexpr int kTmem = 64 + RP <= 128 ? 128 : 256;
    static_assert(kCtas * kTmem <= 512, "the CTAs of an SM share its TMEM");
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "and its shared memory");
};

template <int RP, int RING>
__global__ void __launch_bounds__(kUpThreads, UpCfg<RP, RING>::kCtas) tile_up_kernel(const LoraArgs l, const uint16_t *v2,
                                                             const uint16_t *__restrict__ W, int C, bool scaled,
                                                             const uint16_t *base, int64_t bs, uint16_t *out,
                                                             int64_t os, int cols, const Waits waits)
{
    using Cfg = UpCfg<RP, RING>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const Tile tile = find_tile(l, blockIdx.x, kRows, base != out);
    if (tile.of == 0) {
        grid_wait();
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = smem_u32(align_1024(smem_raw));
    const int rank = tile.a < l.R ? rank_of(l, tile.a) : 0;
    if (tid == 0) {
        mbar_init(&done, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_slot, Cfg::kTmem);
        tmem_relinquish();
    }
    // chunk lane & 7 of the warp's rows lane / 8 + 4 i
    const int ch = lane & 7, row0 = warp * 32 + (lane >> 3);
    const uint32_t piece[2] = {sw128(row0, ch), sw128(row0 + 4, ch)};   // + 1024 every second i
    const uint16_t *yr[8];
    uint16_t *orow[8];
    uint32_t tok = 0;   // bit i: row i is a token
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int p = row0 + 4 * i;
        const int t = p < tile.count ? __ldg(l.order + tile.i0 + p) : -1;
        const bool ok = t >= 0 && t < l.T;
        tok |= (ok ? 1u : 0u) << i;
        yr[i] = base + (ok ? t : 0) * bs;
        orow[i] = out + (ok ? t : 0) * os;
    }
    const uint16_t *wr = W + ((int64_t)min(tile.a, l.R - 1) * l.r + (tid >> 3)) * C;
    const uint32_t at_w = sw128(tid >> 3, ch);
    const int c_lo = blockIdx.y * cols, c_hi = min(c_lo + cols, C);
    const int steps = (c_hi - c_lo + 63) / 64;
    auto fetch = [&](int s) {
        if (s < steps) {
            const uint32_t st = smem + (s % Cfg::kRing) * Cfg::kStage;
            const int c = c_lo + s * 64 + ch * 8;
            const bool in = c < c_hi;
            if (base) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (in && (tok >> i & 1))
                        cp_async_cg16(st + piece[i & 1] + (i >> 1) * kSw, yr[i] + c);
            }
#pragma unroll
            for (int j = 0; j < RP; j += kUpThreads / 8) {   // rows 16 apart share their swizzle
                const bool ok = in && (tid >> 3) + j < rank;
                cp_async_cg16_or_zero(st + Cfg::kY + at_w + j * 128, ok ? wr + (int64_t)j * C + c : W, ok);
            }
        }
        cp_async_commit();
    };
    if (!base) {   // a base that is absent reads as zero
        for (int s = 0; s < Cfg::kRing; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                st_shared_v4(smem + s * Cfg::kStage + piece[i & 1] + (i >> 1) * kSw, make_uint4(0, 0, 0, 0));
    }
    for (int s = 0; s < Cfg::kRing; ++s)
        fetch(s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int ksteps = (rank + 15) / 16;
    grid_wait();   // v2
    grid_launch_next();
    {
        // a thread's token: its row of v2 is the A operand's row, word for word
        const bool some = tid < tile.count;
        const uint4 *src = reinterpret_cast<const uint4 *>(v2 + (int64_t)(tile.i0 + (some ? tid : 0)) * (2 * RP));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k0 = 0; k0 < RP / 16; k0 += 2) {
                constexpr int kBatch = RP == 16 ? 1 : 2;   // 16 ranks each, loads before stores
                uint4 w[kBatch][2];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    w[k][0] = w[k][1] = make_uint4(0, 0, 0, 0);
                    if (some && k0 + k < ksteps) {
                        w[k][0] = ld_after_v4(src + h * (RP / 8) + (k0 + k) * 2);
                        w[k][1] = ld_after_v4(src + h * (RP / 8) + (k0 + k) * 2 + 1);
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    if (k0 + k < ksteps) {
                        const uint4 a = w[k][0], b = w[k][1];
                        const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                        tmem_st_x8(tm + lanes + Cfg::kA + h * (RP / 2) + (k0 + k) * 8, x);
                    }
                }
            }
        }
    }
    tmem_wait_st();
    tc_fence_before();
    const float f = scaled && tile.a < l.R ? l.scales[tile.a] : 1.0f;
    for (int s = 0; s < steps; ++s) {
        cp_async_wait<Cfg::kRing - 1>();
        const uint32_t st = smem + (s % Cfg::kRing) * Cfg::kStage;
        if (ksteps > 0) {
            fence_async_shared();
            __syncthreads();   // the weights have landed; D has been read
            if (tid == 0) {
                tc_fence_after();
                for (int k = 0; k < ksteps; ++k) {
                    const uint64_t bd = smem_desc(st + Cfg::kY + k * 2 * kSw, kSw, kSw, 2);
                    const uint32_t a = tm + Cfg::kA + k * 8;
                    mma_bf16_ts(tm, a, bd, idesc_bf16(kRows, 64, 0, 1), k > 0);
                    mma_bf16_ts(tm, a + RP / 2, bd, idesc_bf16(kRows, 64, 0, 1), 1);
                }
                tc_commit(&done);
            }
            __syncwarp();
            wait_mma(&done, s & 1, &abort_flag, waits);
            const uint32_t row = st + tid * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t r[32];
                tmem_ld_x32(tm + lanes + h * 32, r);
                tmem_wait_ld(r);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t at = row + (((h * 4 + c) ^ (lane & 7)) << 4);
                    const uint4 y = ld_shared_v4(at);
                    uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        float y0 = __uint_as_float(w[p] << 16), y1 = __uint_as_float(w[p] & 0xFFFF0000u);
                        fma2(y0, y1, f, r[c * 8 + 2 * p], r[c * 8 + 2 * p + 1]);
                        w[p] = bf16x2_from_f32(y0, y1);
                    }
                    st_shared_v4(at, make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
            tc_fence_before();
            __syncwarp();
        }
        const int c = c_lo + s * 64 + ch * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = st + piece[i & 1] + (i >> 1) * kSw;
            const uint4 y = ld_shared_v4(at);
            if ((tok >> i & 1) && c < c_hi)
                *reinterpret_cast<uint4 *>(orow[i] + c) = y;
            if (!base)
                st_shared_v4(at, make_uint4(0, 0, 0, 0));
        }
        __syncwarp();
        fetch(s + Cfg::kRing);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_dealloc(tm, Cfg::kTmem);
}

// ---------------------------------------------------------------- grad

// G[a,j,c] = f sum_i p[i,j] x[t,c] over an adapter's tokens: D[128 columns, ranks] with
// the tokens as the contracted index, both operands in rows that run along M and N, 32
// tokens a stage.  p comes as two bf16 parts side by side (p2), so an MMA of twice
// the ranks gives both products, and the halves are added at the end (GradCfg::kJoint).
// Both gradients of a call are one launch: blockIdx.y counts first dA's and then dB's
// column tiles.
// 89 us for the 385 MB of 8191 tokens of 9 adapters, K = 16384, N = 7168, r = 64, 4.3 TB/s:
// a version of 90 us took 52 with neither loads nor MMAs, the chain of its steps (rows'
// numbers, barrier, issue, commit).  Three accumulators (384 columns a tile, a third less
// of p2) gain 3 us there and lose more elsewhere (4 adapters of 1024 tokens, K = 2048, the
// whole backward pass: 66 against 62).  A ring with mbarriers and copying warps of their own took 136 where
// this took 116, a TMA gather of four rows a copy 165 against 90.
constexpr int kGradThreads = 256;
constexpr int kGradTokens = 32;   // a stage
constexpr int kGradCols = 256;    // two accumulators

template <int RP>
struct GradCfg {
    static constexpr int kAtoms = RP <= 32 ? 1 : 2 * RP / 64;   // 64-wide tiles of p2
    static constexpr int kTile = kGradTokens * 128, kX = kGradCols / 64 * kTile, kStage = kX + kAtoms * kTile;
    static constexpr int kStages = RP == 64 ? 4 : 3;
    static constexpr int kCtas = RP <= 32 ? 3 : 2;   // an SM
    static constexpr int kSmem = kStages * kStage + 1024;
    // one MMA for both parts of p, or two into one accumulator: at 128 ranks the TMEM of a
    // second CTA (8191 tokens, K = 16384: the backward pass 316 us, 350 with one; 288 since)
    static constexpr bool kJoint = RP <= 64;
    static constexpr int kAcc = kJoint ? 2 * RP : RP;   // TMEM columns of an accumulator
    static constexpr int kTmem = 2 * kAcc;   // 64 to 256
    static_assert(kCtas * kTmem <= 512 && kCtas * (kSmem + 2048) <= 228 * 1024, "the CTAs of an SM share it");
};

template <int RP>
__global__ void __launch_bounds__(kGradThreads, GradCfg<RP>::kCtas) tile_grad_kernel(const LoraArgs l, const GradSide A, const GradSide B,
                                                                 int size, int slots, const Waits waits)
{
    using Cfg = GradCfg<RP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t done[Cfg::kStages];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const Tile tile = find_tile(l, blockIdx.x, size, false, 1);
    if (tile.of == 0) {
        grid_wait();
        return;
    }
    const int a_tiles = (A.C + kGradCols - 1) / kGradCols;
    const bool second = (int)blockIdx.y >= a_tiles;
    const GradSide S = second ? B : A;
    const int c0 = ((int)blockIdx.y - (second ? a_tiles : 0)) * kGradCols;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(align_1024(smem_raw));
    const int rank = rank_of(l, tile.a);
    if (tid == 0) {
        for (int s = 0; s < Cfg::kStages; ++s)
            mbar_init(done + s, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_slot, Cfg::kTmem);
        tmem_relinquish();
    }
    const int steps = (tile.count + kGradTokens - 1) / kGradTokens;
    // x: chunk tid & 7 of every 64 columns of token tid / 8; p2: RP / 4 chunks a token, tokens
    // kPer apart.  Tokens 8 apart are 1024 bytes apart in a tile and share their swizzle.
    const int col = c0 + (tid & 7) * 8;
    const uint32_t at_x = sw128(tid >> 3, tid & 7);
    static_assert(kGradThreads == 8 * kGradTokens, "a thread copies of one token");
    constexpr int kPer = kGradThreads / (RP / 4);
    const int prow = tid / (RP / 4), pc = tid % (RP / 4);
    const uint32_t at_p = Cfg::kX + (pc >> 3) * Cfg::kTile + sw128(prow, pc & 7);
    const uint16_t *pr = S.p2 + (int64_t)(tile.i0 + prow) * (2 * RP) + pc * 8;
    // the token of this thread's copies, looked up two steps ahead
    auto token = [&](int s) {
        const int i = s * kGradTokens + (tid >> 3), t = i < tile.count ? __ldg(l.order + tile.i0 + i) : -1;
        return t < l.T ? t : -1;
    };
    int t0 = token(0), t1 = token(1), put = 0;   // put: stage of the next copies
    int left = tile.count - prow;
    auto fetch = [&](int s) {
        if (s < steps) {
            const uint32_t st = base + put * Cfg::kStage;
            const uint16_t *row = S.x + (t0 >= 0 ? t0 : 0) * S.xs + col;
#pragma unroll
            for (int i = 0; i < kGradCols / 64; ++i) {
                const bool ok = t0 >= 0 && col + i * 64 < S.C;
                cp_async_cg16_or_zero(st + at_x + i * Cfg::kTile, ok ? row + i * 64 : S.x, ok);
            }
#pragma unroll
            for (int i = 0; i < kGradTokens; i += kPer) {
                if (kPer <= kGradTokens || prow < kGradTokens) {
                    const bool ok = i < left;
                    cp_async_cg16_or_zero(st + at_p + i * 128, ok ? pr + i * 2 * RP : S.p2, ok);
                }
            }
            pr += kGradTokens * 2 * RP;
            left -= kGradTokens;
            t0 = t1;
            t1 = token(s + 2);
            put = put + 1 == Cfg::kStages ? 0 : put + 1;
        }
        cp_async_commit();
    };
    __syncthreads();
    grid_wait();   // the two parts of w and v
    grid_launch_next();
    for (int s = 0; s < Cfg::kStages - 1; ++s)
        fetch(s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t d = tmem_slot;
    for (int s = 0; s < steps; ++s) {
        cp_async_wait<Cfg::kStages - 2>();
        fence_async_shared();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            const uint32_t st = base + (s % Cfg::kStages) * Cfg::kStage;
#pragma unroll
            for (int k = 0; k < kGradTokens / 16; ++k) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {   // 128 columns each
                    const uint64_t xd = smem_desc(st + h * 2 * Cfg::kTile + k * 2 * kSw, Cfg::kTile, kSw, 2);
                    const uint32_t p = st + Cfg::kX + k * 2 * kSw, id = idesc_bf16(128, Cfg::kAcc, 1, 1);
                    mma_bf16_ss(d + h * Cfg::kAcc, xd, smem_desc(p, Cfg::kTile, kSw, 2), id, s > 0 || k > 0);
                    if constexpr (!Cfg::kJoint)
                        mma_bf16_ss(d + h * Cfg::kAcc, xd, smem_desc(p + Cfg::kAtoms / 2 * Cfg::kTile, Cfg::kTile, kSw, 2), id, 1);
                }
            }
            tc_commit(done + s % Cfg::kStages);
        }
        if (s > 0 && s + Cfg::kStages - 1 < steps)
            wait_mma(done + (s - 1) % Cfg::kStages, ((s - 1) / Cfg::kStages) & 1, &abort_flag, waits);
        fetch(s + Cfg::kStages - 1);
    }
    if (steps > 0)
        wait_mma(done + (steps - 1) % Cfg::kStages, ((steps - 1) / Cfg::kStages) & 1, &abort_flag, waits);
    // lane: a column, warps 4 to 7 the second accumulator's
    const int c = c0 + warp * 32 + lane;
    const uint32_t dw = d + (warp >> 2) * Cfg::kAcc + ((uint32_t)((warp & 3) * 32) << 16);
    const float f = S.scaled ? l.scales[tile.a] : 1.0f;
    const int slot = tile.of > 1 ? split_tiles_before(l, tile.a, size) + tile.index : -1;
#pragma unroll
    for (int j0 = 0; j0 < RP; j0 += 8) {
        uint32_t hi[8], lo[8] = {};
        if (steps > 0) {
            tmem_ld_x8(dw + j0, hi);
            if constexpr (Cfg::kJoint)
                tmem_ld_x8(dw + RP + j0, lo);
            tmem_wait_ld(hi, lo);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int j = j0 + k;
            const float g = steps > 0 && j < rank ? f * (__uint_as_float(hi[k]) + __uint_as_float(lo[k])) : 0.0f;
            if (j < l.r && c < S.C && slot < slots) {
                if (tile.of > 1)
                    S.part[((int64_t)slot * l.r + j) * S.C + c] = g;
                else
                    S.G[((int64_t)tile.a * l.r + j) * S.C + c] = __bfloat16_as_ushort(__float2bfloat16_rn(g));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_dealloc(d, Cfg::kTmem);
}

// The gradients of adapters whose tokens were cut: their tiles' parts in order.
__global__ void __launch_bounds__(256) grad_join_kernel(const LoraArgs l, const GradSide A, const GradSide B, int size,
                                                        int slots)
{
    const int a = blockIdx.x;
    grid_wait();
    const int n = (max(group_begin(l, a + 1) - group_begin(l, a), 0) + size - 1) / size;
    if (n <= 1)
        return;
    const GradSide &S = blockIdx.z ? B : A;
    const int64_t elems = (int64_t)l.r * S.C;
    const int first = split_tiles_before(l, a, size);
    if (first + n > slots)
        return;
    const float *part = S.part + first * elems;
    for (int64_t e = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4; e < elems; e += (int64_t)gridDim.y * 1024) {
        float4 s = ld_after_f32x4(part + e);
#pragma unroll 4
        for (int k = 1; k < n; ++k) {
            const float4 p = ld_after_f32x4(part + k * elems + e);
            s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
        }
        uint2 o;
        o.x = bf16x2_from_f32(s.x, s.y);
        o.y = bf16x2_from_f32(s.z, s.w);
        *reinterpret_cast<uint2 *>(S.G + a * elems + e) = o;
    }
}

// The tiles of 128 tokens, which the host does not know: every adapter's last one counts for half.
int64_t host_tiles(const LoraArgs &l) { return l.T / kRows + 1 + std::min<int64_t>(l.R, l.T) / 2; }

// How many ways to share `steps` of 64 columns so that the tiles fill `slots` CTAs once (one
// CTA too many would be a second wave), four steps a share at least.
int shares(const LoraArgs &l, int steps, int slots, int most)
{
    const int64_t want = std::min<int64_t>(slots / host_tiles(l), most);
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, steps / 4));
}

template <int RP>
cudaError_t run_down(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const uint16_t *W, int C,
                     bool scaled, float *v, const Halves &halves, cudaStream_t st)
{
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(tile_down_kernel<RP>), DownCfg<RP>::kSmem);
    if (e != cudaSuccess)
        return e;
    const int steps = (C + 63) / 64, want = shares(l, steps, DownCfg<RP>::kCtas * p.num_sms, kMaxSplits), per = (steps + want - 1) / want;
    const int splits = (steps + per - 1) / per;   // none empty
    const dim3 grid((unsigned)most_tiles(l.T, l.R, kRows, false), splits);
    return launch(tile_down_kernel<RP>, grid, kDownThreads, DownCfg<RP>::kSmem, splits, false, st, l, x, xs, W, C, scaled, v,
                  halves, per * 64, Waits{p.status, p.timeout_ns});
}

template <int RP, int RING>
cudaError_t run_up(const LoraArgs &l, const LoraCall &p, const uint16_t *v2, const uint16_t *W, int C, bool scaled,
                   const uint16_t *base, int64_t bs, uint16_t *out, int64_t os, cudaStream_t st)
{
    using Cfg = UpCfg<RP, RING>;
    const int steps = (C + 63) / 64, slots = Cfg::kCtas * p.num_sms, ranges = shares(l, steps, slots, steps);
    // A shorter ring lets a fourth CTA in: 4096 tokens of rank 32 34.3 us, 35.3 without, 16384 104.6
    // and 105.7; where there are not that many, a longer one is better: 1024 tokens 21.5 and 20.1.
    if constexpr (RING == 3 && (RP == 32 || RP == 64))
        if (host_tiles(l) * (steps / 4) >= UpCfg<RP, 2>::kCtas * p.num_sms)
            return run_up<RP, 2>(l, p, v2, W, C, scaled, base, bs, out, os, st);
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(tile_up_kernel<RP, RING>), Cfg::kSmem);
    if (e != cudaSuccess)
        return e;
    const int per = (steps + ranges - 1) / ranges;
    const dim3 grid((unsigned)most_tiles(l.T, l.R, kRows, base != out), (steps + per - 1) / per);
    return launch(tile_up_kernel<RP, RING>, grid, kUpThreads, Cfg::kSmem, 1, true, st, l, v2, W, C, scaled, base, bs, out, os,
                  per * 64, Waits{p.status, p.timeout_ns});
}

template <int RP>
cudaError_t run_grad(const LoraArgs &l, const LoraCall &p, const GradCall &g, cudaStream_t st)
{
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(tile_grad_kernel<RP>), GradCfg<RP>::kSmem);
    if (e != cudaSuccess)
        return e;
    const int tiles = (g.A.C + kGradCols - 1) / kGradCols + (g.B.C + kGradCols - 1) / kGradCols;
    const dim3 grid((unsigned)(l.T / g.size + l.R), tiles);
    return launch(tile_grad_kernel<RP>, grid, kGradThreads, GradCfg<RP>::kSmem, 1, true, st, l, g.A, g.B, g.size, g.slots,
                  Waits{p.status, p.timeout_ns});
}

// Floats of scratch when the tokens are cut into tiles of `size`: the two halves of w
// and v, and a part of both gradients for every tile of an adapter that has several.
int64_t grad_floats(int64_t T, int r, int K, int N, int64_t size)
{
    const int64_t parts = size < T ? 2 * (T / size) : 0;
    return 2 * T * pad_rank(r) + parts * r * ((int64_t)K + N);
}

}  // namespace

cudaError_t launch_tile_down(const LoraArgs &l, const LoraCall &p, const uint16_t *x, int64_t xs, const uint16_t *W,
                             int C, bool scaled, float *v, const Halves &halves, cudaStream_t st)
{
    switch (pad_rank(l.r)) {
    case 16: return run_down<16>(l, p, x, xs, W, C, scaled, v, halves, st);
    case 32: return run_down<32>(l, p, x, xs, W, C, scaled, v, halves, st);
    case 64: return run_down<64>(l, p, x, xs, W, C, scaled, v, halves, st);
    default: return run_down<128>(l, p, x, xs, W, C, scaled, v, halves, st);
    }
}

cudaError_t launch_tile_up(const LoraArgs &l, const LoraCall &p, const uint16_t *v2, const uint16_t *W, int C, bool scaled,
                           const uint16_t *base, int64_t bs, uint16_t *out, int64_t os, cudaStream_t st)
{
    switch (pad_rank(l.r)) {
    case 16: return run_up<16, 3>(l, p, v2, W, C, scaled, base, bs, out, os, st);
    case 32: return run_up<32, 3>(l, p, v2, W, C, scaled, base, bs, out, os, st);
    case 64: return run_up<64, 3>(l, p, v2, W, C, scaled, base, bs, out, os, st);
    default: return run_up<128, 3>(l, p, v2, W, C, scaled, base, bs, out, os, st);
    }
}

int64_t lora_grad_floats(int64_t T, int r, int K, int N) { return grad_floats(T, r, K, N, T); }

Halves lora_halves(const float *v, int64_t T, int r, float *ws)
{
    uint16_t *w2 = reinterpret_cast<uint16_t *>(ws);
    return {w2, v, v ? w2 + T * 2 * pad_rank(r) : nullptr, pad_rank(r)};
}

GradCall lora_grad_call(const LoraArgs &l, const LoraCall &p, const Halves &h, const uint16_t *x, int64_t xs, int K,
                        uint16_t *dA, const uint16_t *dy, int64_t ys, int N, uint16_t *dB, float *ws, int64_t ws_floats)
{
    // Cut an adapter's tokens so that one adapter alone would fill the SMs once, a quarter
    // larger than that since several adapters end inside a tile each, 384 at least, and no
    // finer than the scratch allows.  Without the quarter 4 adapters of rank 16 over 8192
    // tokens take 77 us, with it 71, at half as large again 72; 4 of rank 64 over 16384: 167,
    // 159, 155; rank 16 over 4096: 44.1, 44.2, 44.8.  At least 256 tokens instead of 384 change
    // none of these.
    const int tiles = (K + kGradCols - 1) / kGradCols + (N + kGradCols - 1) / kGradCols;
    const int ctas = h.RP <= 32 ? 3 : h.RP == 64 ? 2 : 1;   // an SM; 128 ranks have the largest parts to join
    const int64_t ways = (ctas * p.num_sms + tiles - 1) / tiles;
    int64_t size = std::max<int64_t>(384, (5 * l.T / (4 * ways) + 63) / 64 * 64);
    while (size < l.T && grad_floats(l.T, l.r, K, N, size) > ws_floats)
        size *= 2;
    size = std::min<int64_t>(size, (l.T + 63) / 64 * 64);
    float *part = ws + 2 * l.T * h.RP;
    const int64_t slots = size < l.T ? 2 * (l.T / size) : 0;
    return {{x, xs, K, 0, h.w2, dA, part}, {dy, ys, N, 1, h.v2, dB, part + slots * l.r * K}, h.RP, (int)size, (int)slots};
}

cudaError_t launch_tile_grad(const LoraArgs &l, const LoraCall &p, const GradCall &g, cudaStream_t st)
{
    switch (g.RP) {
    case 16: return run_grad<16>(l, p, g, st);
    case 32: return run_grad<32>(l, p, g, st);
    case 64: return run_grad<64>(l, p, g, st);
    default: return run_grad<128>(l, p, g, st);
    }
}

cudaError_t launch_grad_join(const LoraArgs &l, const LoraCall &p, const GradCall &g, cudaStream_t st)
{
    if (g.size >= l.T)
        return cudaSuccess;   // no adapter was cut
    const int64_t most = (int64_t)l.r * std::max(g.A.C, g.B.C);
    const int join = (int)std::min<int64_t>((most + 1023) / 1024, std::max(1, 8 * p.num_sms / l.R));
    return launch(grad_join_kernel, dim3(l.R, join, 2), 256, 0, 1, true, st, l, g.A, g.B, g.size, g.slots);
}

}  // namespace gemmar

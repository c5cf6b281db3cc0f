// gemm_act_few.cu -- gemm_blockscale_act for few rows, where the weights are most of the bytes.
//
// With one row to some tens the product is bound by HBM and, at these sizes (4 us of it), by
// latency: a tile kernel with the rows as its M would leave most SMs without a tile and most of
// an MMA without rows.  Here the weights are the M operand, a pair of 128-row tiles (the gate's
// and the up-projection's rows of the same columns, or 256 columns), and the rows the N: 16, 32
// or 64 of them, larger M in chunks of 64.  K is cut over a cluster of up to 8 CTAs, so
// that the launch has about one CTA per SM; each streams its part of the weights through a
// ring of TMA stages as deep as shared memory, promotes the 128-K sums by their block scales in
// registers, and lays them in its shared memory.  The cluster's CTAs then share out the rows:
// each adds the parts of its rows in the order of K and does what follows the product.
//
// Gated 7168 -> 2 x 2048 to codes, 29 MB of weights: 8.2 us for one row (3.6 TB/s; launch, first bytes
// and join are half of it; 8.6 where two weights take turns), 13.6 for 128; 2048 -> 7168 with a residual, 48 rows: 7.6 us.
#include <algorithm>

#include "activation.cuh"
#include "e4m3_encode.cuh"
#include "epilogue.cuh"
#include "few_rows.cuh"
#include "per_device.h"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kMaxSplits = 8;    // the portable cluster size

// CTAS: of an SM.  Two with rings of half the depth have the same bytes under way, and clusters of
// eight find room: of those with a whole SM per CTA only 15 fit on the GPU at a time, and the
// sixteenth was a second wave.
template <int NT_, int STAGES_, int BUFS_, int CTAS_>
struct Cfg {
    static constexpr int NT = NT_, kStages = STAGES_, kBufs = BUFS_, kCtas = CTAS_;
    static constexpr int kLow = CTAS_ == 1 ? kRegsLow : 40, kHigh = CTAS_ == 1 ? kRegsHigh : 96;   // of 168 or 80 a thread
    static constexpr int kStageBytes = 2 * kTileBytes + NT * 128;
    static constexpr int kBufCols = 2 * NT;
    static constexpr int kTmemCols = kBufCols * kBufs;
    static constexpr int kOffScale = kStages * kStageBytes;   // [8 warps][2][NT]
    static constexpr int kOffBar = kOffScale + 8 * 2 * NT * 4;
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmemBytes = kOffMisc + 16 + 1024;
    static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory budget");
    static_assert(kCtas * kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM budget");
    static_assert(2 * NT * 128 * 4 <= kStages * kStageBytes, "the sums lie in the ring");
};

using Rows16 = Cfg<16, 3, 4, 2>;
using Rows32 = Cfg<32, 3, 4, 2>;
using Rows64 = Cfg<64, 5, 4, 1>;

// 4 consecutive values of a row
__device__ __forceinline__ float4 load4(const void *p, int64_t at, bool bf16)
{
    if (bf16) {
        const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + at);
        return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
    }
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
}

__device__ __forceinline__ void store4(void *p, int64_t at, bool bf16, const float4 &v)
{
    if (bf16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at) = make_uint2(bf16x2_from_f32(v.x, v.y), bf16x2_from_f32(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) = v;
}

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b)
{
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// grid: (splits of K, tile pairs, chunks of rows); the splits are a cluster
template <class C, bool GATED>
__global__ void __launch_bounds__(kThreads, C::kCtas) gemm_act_few_kernel(const __grid_constant__ ActParams prm)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *empty = full + C::kStages;
    uint64_t *tfull = empty + C::kStages;
    uint64_t *tempty = tfull + C::kBufs;
    uint64_t *final_bar = tempty + C::kBufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

    const ActEpilogue &e = prm.e;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x, splits = gridDim.x, j = blockIdx.y, m0 = blockIdx.z * C::NT;
    const int KB = e.K / 128, kb0 = KB * rank / splits, kb1 = KB * (rank + 1) / splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(tfull + b, 1);
            mbar_init(tempty + b, 8);
        }
        mbar_init(final_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&prm.tmA);
        prefetch_tmap(&prm.tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (warp < 4) {
        setmaxnreg_dec<C::kLow>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            const int r0 = GATED ? j * 128 : j * 256, r1 = GATED ? e.N + r0 : r0 + 128;   // zeros past the last row
            int issued = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                const int stage = issued % C::kStages;
                if (!mbar_wait(empty + stage, (issued / C::kStages & 1) ^ 1, abort_flag, prm.status, prm.timeout_ns,
                               SITE_PRODUCER_EMPTY))
                    break;
                uint8_t *w = smem + stage * C::kStageBytes;
                mbar_arrive_expect_tx(full + stage, C::kStageBytes);
                tma_load_2d(w, &prm.tmB, full + stage, kb * 128, r0);
                tma_load_2d(w + kTileBytes, &prm.tmB, full + stage, kb * 128, r1);
                tma_load_2d(w + 2 * kTileBytes, &prm.tmA, full + stage, kb * 128, m0);
            }
            drain_loads(full, C::kStages, issued, prm.timeout_ns);
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc = idesc_f8_e4m3(128, C::NT);
            for (int i = 0; i < kb1 - kb0; ++i) {
                const int stage = i % C::kStages, buf = i % C::kBufs;
                if (!mbar_wait(tempty + buf, (i / C::kBufs & 1) ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_TMEM_EMPTY) ||
                    !mbar_wait(full + stage, i / C::kStages & 1, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_FULL))
                    break;
                tc_fence_after();
                const uint32_t w = smem_u32(smem + stage * C::kStageBytes);
                const uint64_t xd = desc_kmajor_sw128(w + 2 * kTileBytes);
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint64_t wd = desc_kmajor_sw128(w + tile * kTileBytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8(tmem_base + buf * C::kBufCols + tile * C::NT, wd + 2 * k, xd + 2 * k, idesc, k > 0 ? 1u : 0u);
                }
                tc_commit(empty + stage);
                tc_commit(tfull + buf);
            }
            tc_commit(final_bar);
            wait_teardown(final_bar, prm.status, prm.timeout_ns);
        }
    } else {
        setmaxnreg_inc<C::kHigh>();
        // ---------------------------------------------------- promotion
        const int q = warp & 3, h = (warp - 4) >> 2;   // lane quarter, tile of the pair
        float *ts = reinterpret_cast<float *>(smem + C::kOffScale) + (warp - 4) * 2 * C::NT;
        const uint32_t taddr0 = tmem_base + ((uint32_t)(q * 32) << 16) + h * C::NT;
        const int block = GATED ? h * (e.N / 128) + j : min(j * 2 + h, e.N / 128 - 1);
        const float *sw = prm.sb + (int64_t)block * KB;
        constexpr int PER = (C::NT + 31) / 32;
        int at[PER];   // where a row's scales begin; -1: no row at this column
        float next_ts[PER], next_sw = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            at[i] = lane + 32 * i < min(C::NT, e.M - m0) ? lane + 32 * i : -1;
        auto fetch = [&](int kb) {
            next_sw = __ldg(sw + kb);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                next_ts[i] = at[i] >= 0 ? __ldg(prm.sa + (int64_t)(m0 + at[i]) * KB + kb) : 0.0f;
        };
        float acc[C::NT];
#pragma unroll
        for (int t = 0; t < C::NT; ++t)
            acc[t] = 0.0f;
        if (kb0 < kb1)
            fetch(kb0);
        bool ok = true;
        for (int i = 0; i < kb1 - kb0; ++i) {
            float *now = ts + (i & 1) * C::NT;   // the warp's own, read last two steps back
#pragma unroll
            for (int k = 0; k < PER; ++k)
                if (lane + 32 * k < C::NT)
                    now[lane + 32 * k] = next_sw * next_ts[k];
            if (kb0 + i + 1 < kb1)
                fetch(kb0 + i + 1);
            const int buf = i % C::kBufs;
            ok = mbar_wait(tfull + buf, i / C::kBufs & 1, abort_flag, prm.status, prm.timeout_ns, SITE_EPI_TMEM_FULL);
            if (!ok)
                break;
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < C::NT; c += 16)
                if (c < e.M - m0) {
                    uint32_t r[16];
                    tmem_ld_x16(taddr0 + buf * C::kBufCols + c, r);
                    tmem_wait_ld(r);
                    promote8(acc + c, *reinterpret_cast<uint32_t(*)[8]>(&r[0]), now + c);
                    promote8(acc + c + 8, *reinterpret_cast<uint32_t(*)[8]>(&r[8]), now + c + 8);
                }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tempty + buf);
        }
        // the part's sums, [tile][row of activations][128]: the ring is read, as the last step's
        // MMAs have completed
        if (ok) {
            float *part = reinterpret_cast<float *>(smem) + h * C::NT * 128 + q * 32 + lane;
#pragma unroll
            for (int t = 0; t < C::NT; ++t)
                if (t < e.M - m0)
                    part[t * 128] = acc[t];
        }
    }
    __syncwarp();
    cluster_sync();
    if (warp >= 4) {
        // ---------------------------------------------------- what follows the product: a warp takes a
        // row's 128 columns, the cluster's warps in turn
        const int rows = min(C::NT, e.M - m0), P = GATED ? 2 * e.N : e.N;
        constexpr int TILES = GATED ? 1 : 2;
        const uint32_t own = smem_u32(smem) + lane * 16;
        auto column = [&](int i) { return (GATED ? j * 128 : j * 256 + i % TILES * 128) + lane * 4; };
        auto residual = [&](int i) {
            const int n = column(i);
            if (e.res == nullptr || i >= rows * TILES || n >= e.N)
                return make_float4(0, 0, 0, 0);
            return load4(e.res, (int64_t)(m0 + i / TILES) * e.rs + n, e.r_bf16);
        };
        int i = rank + splits * (warp - 4);
        float4 next_res = residual(i);
        for (; i < rows * TILES; i += splits * 8) {
            const int t = i / TILES, tile = i % TILES, n = column(i);
            const int64_t m = m0 + t;
            const float4 res = next_res;
            next_res = residual(i + splits * 8);
            if (n >= e.N)
                continue;   // the whole warp: an odd number of blocks of columns
            float4 z = make_float4(0, 0, 0, 0), zu = z;
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
                if (s < splits) {
                    const uint32_t there = mapa_shared(own, s);
                    z = add4(z, ld_shared_cluster_f32x4(there + (tile * C::NT + t) * 512));
                    if (GATED)
                        zu = add4(zu, ld_shared_cluster_f32x4(there + (C::NT + t) * 512));
                }
            if (e.bias != nullptr) {
                z = add4(z, __ldg(reinterpret_cast<const float4 *>(e.bias + n)));
                if (GATED)
                    zu = add4(zu, __ldg(reinterpret_cast<const float4 *>(e.bias + e.N + n)));
            }
            if (e.z != nullptr) {
                store4(e.z, m * P + n, true, z);
                if (GATED)
                    store4(e.z, m * P + e.N + n, true, zu);
            }
            float4 out;
            with_act(e.act, [&](auto act) {
                constexpr int ACT = decltype(act)::value;
                out = make_float4(act_value<ACT>(z.x), act_value<ACT>(z.y), act_value<ACT>(z.z), act_value<ACT>(z.w));
            });
            if (GATED)
                out = make_float4(out.x * zu.x, out.y * zu.y, out.z * zu.z, out.w * zu.w);
            if (e.res != nullptr)
                out = add4(out, res);
            if (e.C != nullptr)
                store4(e.C, m * e.cs + n, e.c_bf16, out);
            if (e.q != nullptr) {
                const float size = fmaxf(fmaxf(fmaxf(0.0f, fabsf(out.x)), fabsf(out.y)), fmaxf(fabsf(out.z), fabsf(out.w)));   // skips NaN
                const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(size)));
                const float scale = __fdiv_rn(top, 448.0f);
                *reinterpret_cast<uint32_t *>(e.q + m * e.N + n) = enc4(out.x, out.y, out.z, out.w, scale);
                if (lane == 0)
                    e.scales[m * (e.N / 128) + n / 128] = scale;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();   // the others have read this CTA's sums
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, C::kTmemCols);
}

// Clusters of each size that the GPU runs at a time: fewer CTAs than SMs where a GPC's are no
// multiple of the size.
struct Room {
    int clusters[kMaxSplits + 1];
};

template <class C, bool GATED>
cudaLaunchConfig_t config(int splits, cudaLaunchAttribute *attrs)
{
    cudaLaunchConfig_t cfg = {};
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = (unsigned)splits;
    attrs[0].val.clusterDim.y = 1;
    attrs[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    return cfg;
}

template <class C, bool GATED>
bool measure_room(Room &r)
{
    r = Room{};
    bool ok = ensure_dynamic_smem(reinterpret_cast<const void *>(gemm_act_few_kernel<C, GATED>), C::kSmemBytes) == cudaSuccess;
    for (int s = 1; s <= kMaxSplits && ok; ++s) {
        cudaLaunchAttribute attrs[1];
        const cudaLaunchConfig_t cfg = config<C, GATED>(s, attrs);
        ok = cudaOccupancyMaxActiveClusters(&r.clusters[s], gemm_act_few_kernel<C, GATED>, &cfg) == cudaSuccess;
    }
    if (!ok)
        cudaGetLastError();   // the call goes on without this kernel
    return ok;
}

// The current device's; none where it cannot be told.
template <class C, bool GATED>
Room room_here()
{
    static PerDevice<Room> rooms;
    Room r;
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && rooms.get(dev, r, measure_room<C, GATED>) ? r : Room{};
}

template <bool GATED>
int tile_pairs(int N) { return GATED ? N / 128 : (N + 255) / 256; }

// The parts of K that end soonest, and when: a wave of clusters takes 0.54 us per 128 of K, 0.35 us
// per turn of its warps through the rows, and 2 us besides, a launch 3 (measured: 20 us for 256
// gated rows at N = 2048, K = 7168, 11.9 for 128 at N = 7168, K = 2048, 10.5 for 512 at 1920 x 1152).
struct Plan {
    int splits;
    int64_t ns;
};

template <class C, bool GATED>
Plan plan(int M, int N, int K)
{
    const Room room = room_here<C, GATED>();
    const int KB = K / 128, rows = std::min(M, C::NT) * (GATED ? 1 : 2);
    const int64_t clusters = (int64_t)tile_pairs<GATED>(N) * ((M + C::NT - 1) / C::NT);
    Plan best{1, INT64_MAX};
    for (int s = 1; s <= std::min(kMaxSplits, KB); ++s) {
        if (room.clusters[s] < 1)
            continue;
        const int64_t waves = (clusters + room.clusters[s] - 1) / room.clusters[s];
        const int64_t ns = waves * (540 * ((KB + s - 1) / s) + 350 * ((rows + 8 * s - 1) / (8 * s)) + 2000) + 3000;
        if (ns < best.ns)
            best = {s, ns};
    }
    return best;
}

template <class C, bool GATED>
cudaError_t launch_typed(const ActParams &p, cudaStream_t st)
{
    const void *kernel = reinterpret_cast<const void *>(gemm_act_few_kernel<C, GATED>);
    const cudaError_t e = ensure_dynamic_smem(kernel, C::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    static std::atomic<bool> split_ok{false};
    if (!few_rows_split_ok(split_ok, kernel, C::kLow, C::kHigh))
        return cudaErrorInvalidConfiguration;
    const int splits = plan<C, GATED>(p.e.M, p.e.N, p.e.K).splits;
    cudaLaunchAttribute attrs[1];
    cudaLaunchConfig_t cfg = config<C, GATED>(splits, attrs);
    cfg.gridDim = dim3(splits, tile_pairs<GATED>(p.e.N), (p.e.M + C::NT - 1) / C::NT);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, gemm_act_few_kernel<C, GATED>, p);
}

template <class C>
cudaError_t launch_rows(const ActParams &p, cudaStream_t st)
{
    return p.e.gated ? launch_typed<C, true>(p, st) : launch_typed<C, false>(p, st);
}

}  // namespace

int gemm_act_few_rows(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }

int64_t gemm_act_few_ns(int M, int N, int K, bool gated)
{
    if ((M + 63) / 64 > 65535)
        return INT64_MAX;   // more chunks than a grid's third dimension has
    switch (gemm_act_few_rows(M)) {
    case 16: return (gated ? plan<Rows16, true>(M, N, K) : plan<Rows16, false>(M, N, K)).ns;
    case 32: return (gated ? plan<Rows32, true>(M, N, K) : plan<Rows32, false>(M, N, K)).ns;
    default: return (gated ? plan<Rows64, true>(M, N, K) : plan<Rows64, false>(M, N, K)).ns;
    }
}

cudaError_t launch_gemm_act_few(const ActParams &p, cudaStream_t st)
{
    switch (gemm_act_few_rows(p.e.M)) {
    case 16: return launch_rows<Rows16>(p, st);
    case 32: return launch_rows<Rows32>(p, st);
    default: return launch_rows<Rows64>(p, st);
    }
}

}  // namespace gemmar

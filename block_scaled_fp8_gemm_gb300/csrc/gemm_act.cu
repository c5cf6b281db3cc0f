// gemm_act.cu -- the block-scaled e4m3 GEMM with bias, activation (gated or not), residual
// and quantisation in its epilogue (gemm_blockscale_act), for many rows.
//
//   z = A B^T + bias,  out = residual + act(z)               columns n0 .. n0+255 of a tile
//   or  z_g, z_u,      out = residual + act(z_g) * z_u       columns n0 .. n0+127 of both halves
//
// Bound by the tensor cores and, before them, by the promotion: the block scales change every
// 128 of K, so each of a tile's 128 x 256 sums is read from TMEM and multiplied-added in fp32
// once per K-block.  The kernel is laid out for that as gemm_blockscale.cu is: one persistent
// CTA per SM, a TMA producer warp, an MMA warp, two TMEM accumulators, and eight epilogue
// warps whose threads keep one row and 128 columns in registers.  A gated tile holds 128
// columns of each half, and a thread the same 64 of both, so the gate needs nothing from
// another thread.  What follows the product never leaves the registers except as the
// call's outputs.
#include <algorithm>

#include "activation.cuh"
#include "e4m3_encode.cuh"
#include "epilogue.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kThreads = 384;
constexpr int kStages = 4;
constexpr int kABytes = 128 * 128;
constexpr int kBBytes = 256 * 128;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpiWarps = 8;
constexpr int kOffB = kStages * kABytes;
constexpr int kOffStaging = kOffB + kStages * kBBytes;   // 4 KB per epilogue warp
constexpr int kOffMax = kOffStaging + kEpiWarps * 4096;  // a gated row's maximum, per column half
constexpr int kOffBar = kOffMax + 2 * 128 * 4;
constexpr int kNumBars = 2 * kStages + 5 + 4;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kSmemBytes = kOffMisc + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr int kRegsLow = 56;     // warps 0-3 after setmaxnreg.dec
constexpr int kRegsHigh = 224;   // epilogue warps after setmaxnreg.inc
constexpr int kRegsNeeded = 128 * kRegsLow + 256 * kRegsHigh;
constexpr int kGroupM = 16;      // row tiles that share their columns of B while they are in L2

struct Tile {
    int m0, n0;
};

__device__ __forceinline__ Tile decode(int t, int mt_total, int ntiles, int bn)
{
    const int per_group = kGroupM * ntiles;
    const int m_first = (t / per_group) * kGroupM;
    const int idx = t % per_group;
    const int gm = min(kGroupM, mt_total - m_first);
    return {(m_first + idx % gm) * 128, (idx / gm) * bn};
}

// The reverse of store_chunk: each thread gets UNITS 16-byte units of its own row, which the
// warp reads row-contiguously.  Rows past rows_valid read as zero.
template <int UNITS>
__device__ __forceinline__ void load_chunk(uint32_t stage, uint4 (&v)[UNITS], const char *gsrc, int64_t row_stride_bytes,
                                           int rows_valid)
{
    constexpr int ROWB = UNITS * 16, RPI = 32 / UNITS;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int r = i * RPI + lane / UNITS, u = lane % UNITS;
        const int rsw = (UNITS == 8) ? (r & 7) : ((r >> 1) & 3);
        uint4 val = make_uint4(0, 0, 0, 0);
        if (r < rows_valid)
            val = *reinterpret_cast<const uint4 *>(gsrc + r * row_stride_bytes + u * 16);
        st_shared_v4(stage + r * ROWB + ((u ^ rsw) * 16), val);
    }
    __syncwarp();
    const int sw = (UNITS == 8) ? (lane & 7) : ((lane >> 1) & 3);
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
        v[u] = ld_shared_v4(stage + lane * ROWB + ((u ^ sw) * 16));
    __syncwarp();
}

// 32 columns of a thread's row to global memory, as bf16 or fp32.
__device__ __forceinline__ void store_cols32(uint32_t staging, const float *a, bool bf16, char *dst, int64_t stride,
                                             int rows_valid)
{
    if (bf16) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            v[u] = make_uint4(bf16x2_from_f32(a[8 * u], a[8 * u + 1]), bf16x2_from_f32(a[8 * u + 2], a[8 * u + 3]),
                              bf16x2_from_f32(a[8 * u + 4], a[8 * u + 5]), bf16x2_from_f32(a[8 * u + 6], a[8 * u + 7]));
        store_chunk<4>(staging, v, dst, stride * 2, rows_valid);
    } else {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = make_uint4(__float_as_uint(a[4 * u]), __float_as_uint(a[4 * u + 1]), __float_as_uint(a[4 * u + 2]),
                              __float_as_uint(a[4 * u + 3]));
        store_chunk<8>(staging, v, dst, stride * 4, rows_valid);
    }
}

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 1) gemm_act_kernel(const __grid_constant__ ActParams prm)
{
    constexpr int BN = GATED ? 128 : 256;   // output columns of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;   // [2]
    uint64_t *tempty = tfull + 2;        // [2]
    uint64_t *final_bar = tempty + 2;
    uint64_t *max_bar = final_bar + 1;   // [4], per lane quarter: both halves' maxima written, then both read
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffMisc + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ActEpilogue &e = prm.e;
    const int KB = e.K / 128, mt = (e.M + 127) / 128, nt = (e.N + BN - 1) / BN, tiles = mt * nt;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull + b, 1);
            mbar_init(tempty + b, kEpiWarps);
        }
        mbar_init(final_bar, 1);
        for (int i = 0; i < 4; ++i)
            mbar_init(max_bar + i, 2);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&prm.tmA);
        prefetch_tmap(&prm.tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < 4) {
        setmaxnreg_dec<kRegsLow>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile c = decode(t, mt, nt, BN);
                const int nb = GATED ? e.N + c.n0 : c.n0 + 128;   // the tile's second 128 rows of B
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(empty + stage, ph ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_PRODUCER_EMPTY)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full + stage, kStageBytes);
                    uint8_t *b = smem + kOffB + stage * kBBytes;
                    tma_load_2d(smem + stage * kABytes, &prm.tmA, full + stage, kb * 128, c.m0);
                    tma_load_2d(b, &prm.tmB, full + stage, kb * 128, c.n0);
                    tma_load_2d(b + 128 * 128, &prm.tmB, full + stage, kb * 128, nb);   // zeros past the last row
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        ph ^= 1;
                    }
                }
            }
            if (*abort_flag)
                drain_loads(full, kStages, issued, prm.timeout_ns);
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            const uint32_t idesc = idesc_f8_e4m3(128, 256);
            int stage = 0;
            uint32_t ph = 0, n = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                for (int kb = 0; kb < KB; ++kb, ++n) {
                    const uint32_t buf = n & 1, tph = (n >> 1) & 1;
                    if (!mbar_wait(tempty + buf, tph ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_TMEM_EMPTY) ||
                        !mbar_wait(full + stage, ph, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = desc_kmajor_sw128(smem_u32(smem + stage * kABytes));
                    const uint64_t bd = desc_kmajor_sw128(smem_u32(smem + kOffB + stage * kBBytes));
#pragma unroll
                    for (int k = 0; k < 4; ++k)   // 4 x 32 of K = one 128-byte swizzle row
                        mma_f8(tmem_base + buf * 256, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
                    tc_commit(empty + stage);
                    tc_commit(tfull + buf);
                    if (++stage == kStages) {
                        stage = 0;
                        ph ^= 1;
                    }
                }
            }
            tc_commit(final_bar);
            wait_teardown(final_bar, prm.status, prm.timeout_ns);
        }
    } else {
        setmaxnreg_inc<kRegsHigh>();
        // ---------------------------------------------------- epilogue
        const int ew = warp - 4, q = warp & 3, h = ew >> 2;   // lane quarter, column half
        const int row = q * 32 + lane;
        const uint32_t staging = smem_u32(smem + kOffStaging + ew * 4096);
        float *maxima = reinterpret_cast<float *>(smem + kOffMax);   // [2][128]
        uint32_t groups = 0;   // tiles whose maxima were exchanged
        // the thread's two runs of 64 columns in the accumulator, and the same columns in B's rows
        const int col0 = GATED ? h * 64 : h * 128, col1 = GATED ? 128 + h * 64 : h * 128 + 64;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
        uint32_t n = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile c = decode(t, mt, nt, BN);
            const int64_t mrow = min(c.m0 + row, e.M - 1);
            const float *sa_row = prm.sa + mrow * KB;
            // a tile past the last column block (an odd number of them) has no scales to read
            const int last_block = (GATED ? 2 * e.N : e.N) / 128 - 1;
            const float *sb0 = prm.sb + (int64_t)min(last_block, (c.n0 + (GATED ? 0 : h * 128)) / 128) * KB;
            const float *sb1 = GATED ? prm.sb + (int64_t)((e.N + c.n0) / 128) * KB : sb0;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j)
                acc[j] = 0.0f;
            float a_next = __ldg(sa_row), b0_next = __ldg(sb0), b1_next = __ldg(sb1);
            for (int kb = 0; kb < KB; ++kb, ++n) {
                const float s0 = a_next * b0_next, s1 = a_next * b1_next;
                if (kb + 1 < KB) {
                    a_next = __ldg(sa_row + kb + 1);
                    b0_next = __ldg(sb0 + kb + 1);
                    b1_next = __ldg(sb1 + kb + 1);
                }
                const uint32_t buf = n & 1, tph = (n >> 1) & 1;
                if (!mbar_wait(tfull + buf, tph, abort_flag, prm.status, prm.timeout_ns, SITE_EPI_TMEM_FULL)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = lane_base + buf * 256;
                // 16-column loads, the next one issued before the current one's promotions
                uint32_t ra[16], rb[16];
                tmem_ld_x16(taddr + col0, ra);
                tmem_wait_ld(ra);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t(&cur)[16] = (i & 1) ? rb : ra;
                    uint32_t(&nxt)[16] = (i & 1) ? ra : rb;
                    if (i + 1 < 8)
                        tmem_ld_x16(taddr + (i + 1 < 4 ? col0 + (i + 1) * 16 : col1 + (i - 3) * 16), nxt);
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        fma2(acc[i * 16 + j], acc[i * 16 + j + 1], i < 4 ? s0 : s1, cur[j], cur[j + 1]);
                    if (i + 1 < 8) {
                        tmem_wait_ld(nxt);
                        if (i + 2 == 8) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(tempty + buf);
                        }
                    }
                }
            }
            if (!ok)
                break;
            // -------- what follows the product
            const int m_warp = c.m0 + q * 32;
            const int cols0 = c.n0 + (GATED ? h * 64 : h * 128);   // the thread's first output column
            const bool inside = cols0 < e.N;                       // warp-uniform
            const int rows_valid = inside ? max(0, min(32, e.M - m_warp)) : 0;
            const int P = GATED ? 2 * e.N : e.N;
            if (e.bias != nullptr && inside) {
                const float4 *b0 = reinterpret_cast<const float4 *>(e.bias + cols0);
                const float4 *b1 = reinterpret_cast<const float4 *>(e.bias + (GATED ? e.N + cols0 : cols0 + 64));
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float4 b = __ldg(j < 16 ? b0 + j : b1 + (j - 16));
                    acc[4 * j] += b.x;
                    acc[4 * j + 1] += b.y;
                    acc[4 * j + 2] += b.z;
                    acc[4 * j + 3] += b.w;
                }
            }
            if (e.z != nullptr) {
                char *z = reinterpret_cast<char *>(e.z) + ((int64_t)m_warp * P + cols0) * 2;
                const int64_t second = GATED ? e.N : 64;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    store_cols32(staging, &acc[i * 32], true, z + (i < 2 ? i * 32 : second + (i - 2) * 32) * 2, P, rows_valid);
            }
            constexpr int W = GATED ? 64 : 128;   // output columns of a thread
            with_act(e.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    acc[j] = act_value<decltype(act)::value>(acc[j]);
                    if (GATED)
                        acc[j] *= acc[(64 + j) & 127];
                }
            });
            if (e.res != nullptr) {
                const int bytes = e.r_bf16 ? 2 : 4;
                const char *r = static_cast<const char *>(e.res) + ((int64_t)m_warp * e.rs + cols0) * bytes;
#pragma unroll
                for (int i = 0; i < W / 32; ++i) {
                    if (e.r_bf16) {
                        uint4 v[4];
                        load_chunk<4>(staging, v, r + i * 64, e.rs * 2, rows_valid);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                acc[i * 32 + u * 8 + 2 * j] += bf16_lo(w[j]);
                                acc[i * 32 + u * 8 + 2 * j + 1] += bf16_hi(w[j]);
                            }
                        }
                    } else {
                        uint4 v[8];
                        load_chunk<8>(staging, v, r + i * 128, e.rs * 4, rows_valid);
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            acc[i * 32 + u * 4] += __uint_as_float(v[u].x);
                            acc[i * 32 + u * 4 + 1] += __uint_as_float(v[u].y);
                            acc[i * 32 + u * 4 + 2] += __uint_as_float(v[u].z);
                            acc[i * 32 + u * 4 + 3] += __uint_as_float(v[u].w);
                        }
                    }
                }
            }
            if (e.C != nullptr) {
                const int bytes = e.c_bf16 ? 2 : 4;
                char *out = static_cast<char *>(e.C) + ((int64_t)m_warp * e.cs + cols0) * bytes;
#pragma unroll
                for (int i = 0; i < W / 32; ++i)
                    store_cols32(staging, &acc[i * 32], e.c_bf16, out + i * 32 * bytes, e.cs, rows_valid);
            }
            if (e.q != nullptr) {
                // one scale per row and 128 columns: a gated thread has half of them
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < W; ++j)
                    m = fmaxf(m, fabsf(acc[j]));   // skips NaN
                if (GATED) {
                    // the barrier's phases alternate: both warps have written, both have read
                    if ((groups > 0 && !mbar_wait(max_bar + q, 1, abort_flag, prm.status, prm.timeout_ns, SITE_ROW_MAX))) {
                        ok = false;
                        break;
                    }
                    maxima[h * 128 + row] = m;
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(max_bar + q);
                    if (!mbar_wait(max_bar + q, 0, abort_flag, prm.status, prm.timeout_ns, SITE_ROW_MAX)) {
                        ok = false;
                        break;
                    }
                    ++groups;
                    m = fmaxf(m, maxima[(h ^ 1) * 128 + row]);
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(max_bar + q);
                }
                const float scale = __fdiv_rn(m, 448.0f);
                const Enc enc(scale);
                uint8_t *codes = e.q + (int64_t)m_warp * e.N + cols0;
#pragma unroll
                for (int i = 0; i < W / 64; ++i) {
                    uint32_t w[16];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float(&x)[16] = *reinterpret_cast<float(*)[16]>(&acc[i * 64 + u * 16]);
                        uint32_t(&o)[4] = *reinterpret_cast<uint32_t(*)[4]>(&w[u * 4]);
                        enc.codes(x, o);
                    }
                    const uint4 v[4] = {make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]),
                                        make_uint4(w[8], w[9], w[10], w[11]), make_uint4(w[12], w[13], w[14], w[15])};
                    store_chunk<4>(staging, v, reinterpret_cast<char *>(codes) + i * 64, e.N, rows_valid);
                }
                if (lane < rows_valid && (!GATED || h == 0))
                    e.scales[(int64_t)(m_warp + lane) * (e.N / 128) + cols0 / 128] = scale;
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, 512);
}

}  // namespace

bool gemm_act_split_ok()
{
    cudaFuncAttributes a, b;
    return cudaFuncGetAttributes(&a, gemm_act_kernel<false>) == cudaSuccess &&
           cudaFuncGetAttributes(&b, gemm_act_kernel<true>) == cudaSuccess &&
           std::min(a.numRegs, b.numRegs) * kThreads >= kRegsNeeded;
}

cudaError_t launch_gemm_act(const ActParams &p, int num_sms, cudaStream_t st)
{
    const bool gated = p.e.gated;
    const void *kernel = gated ? reinterpret_cast<const void *>(gemm_act_kernel<true>)
                               : reinterpret_cast<const void *>(gemm_act_kernel<false>);
    const cudaError_t e = ensure_dynamic_smem(kernel, kSmemBytes);
    if (e != cudaSuccess)
        return e;
    const int bn = gated ? 128 : 256;
    const int64_t tiles = (int64_t)((p.e.M + 127) / 128) * ((p.e.N + bn - 1) / bn);
    const int grid = (int)std::min<int64_t>(tiles, num_sms);
    if (gated)
        gemm_act_kernel<true><<<grid, kThreads, kSmemBytes, st>>>(p);
    else
        gemm_act_kernel<false><<<grid, kThreads, kSmemBytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace gemmar

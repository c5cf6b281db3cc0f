// gemm_act.cu -- the block-scaled e4m3 GEMM with bias, activation (gated or not), residual
// and quantisation in its epilogue (gemm_blockscale_act), for many rows.
//
//   z = A B^T + bias,  out = residual + act(z)               columns n0 .. n0+255 of a tile
//   or  z_g, z_u,      out = residual + act(z_g) * z_u       columns n0 .. n0+127 of both halves
//
// Bound by the tensor cores and, before them, by the promotion: the block scales change every
// 128 of K, so each of a tile's 128 x 256 sums is read from TMEM and multiplied-added in fp32
// once per K-block.  A K-block takes about 900 cycles, 512 of MMA, whose accumulators share TMEM's
// bandwidth with those reads (755 in the same pipeline without them): 16384 x 7168 x 2048 to
// bf16 in 215 us, 0.59 of the MMA's rate; with bias and residual 250 us; gated 7168 -> 2 x 2048 to
// codes and z, 4096 rows, 113 us.  One persistent CTA per SM, 16 warps:
//   warp 0      TMA producer: A tile 128x128 and B rows 2 x 128 per 128-K stage
//   warp 1      MMA issuer, 128 x 256 x 32 each into one of two TMEM buffers (two MMAs of 128
//               columns with two buffers each, for a finer overlap, ran at 0.69 of the rate)
//   warps 4-11  promotion: a thread keeps one row and 128 columns in registers; at tile end they
//               go back into the TMEM buffer of the last K-block (a "park").  While it is parked
//               the next tile's K-blocks run in the other buffer, one by one, so the MMA warp
//               takes for each the buffer that is free and leaves on record which
//   warps 12-15 finish: one per TMEM lane quarter, a thread per row.  They take a parked tile 32
//               columns at a time through bias, activation, gate, residual and the stores, while
//               the next tile is promoted.  A thread writes its own row in whole 32-byte sectors,
//               with no staging; the residual, which they would wait for, is asked for ahead
#include <algorithm>

#include "activation.cuh"
#include "e4m3_encode.cuh"
#include "epilogue.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kThreads = 512;
constexpr int kABytes = 128 * 128;
constexpr int kBBytes = 256 * 128;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kSteps = 4;        // K-steps whose buffer is on record: more than can be under way
constexpr int kResBytes = 16 * 1024;
// An ungated tile takes K in three stages as fast as in four, and has the room for its residual's rows on
// their way (16384 x 7168 x 2048 with a bf16 residual 240 us, with 64 columns of it in registers 276; fp32
// 302 and 381).  A gated one, 3% slower with three, keeps 64 columns in registers.
template <bool GATED>
struct Smem {
    static constexpr int kStages = GATED ? 4 : 3;
    static constexpr int kOffB = kStages * kABytes;
    static constexpr int kOffBias = kOffB + kStages * kBBytes;   // [4 finish warps][256] of the tile's columns
    static constexpr int kOffRes = kOffBias + 4 * 1024;          // [4 finish warps] rows of the residual
    static constexpr int kOffBar = kOffRes + (GATED ? 0 : 4 * kResBytes);
    static constexpr int kNumBars = 2 * kStages + kSteps + 5;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kBytes = kOffMisc + 8 + 4 * kSteps + 8 + 1024;
    static_assert(kBytes <= 232448, "shared memory budget");
};
// setmaxnreg: warps 0-3, promotion, finish, of 128 a thread.  Neither role of any form spills.  Promotion
// with the eight more that an ungated finish without gelu leaves: 16384 x 7168 x 2048 213 us, without 224.
constexpr int kRegsLow = 40;
template <bool GATED, bool GELU> constexpr int kRegsPromote = GATED || GELU ? 176 : 184;
template <bool GATED, bool GELU> constexpr int kRegsFinish = GATED || GELU ? 120 : 104;
template <bool GATED, bool GELU> constexpr int kRegsNeeded = 128 * kRegsLow + 256 * kRegsPromote<GATED, GELU> + 128 * kRegsFinish<GATED, GELU>;
static_assert(kRegsNeeded<true, false> <= 65536 && kRegsNeeded<false, true> <= 65536 && kRegsNeeded<false, false> <= 65536, "register split");
static_assert(kRegsPromote<true, false> >= 128 && kRegsFinish<true, false> <= 128 && kRegsPromote<false, false> >= 128 && kRegsFinish<false, false> <= 128,
              "raised and lowered from 128");
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

// 32 bytes of a row at a 16-byte boundary; `whole`: at a 32-byte one
__device__ __forceinline__ void load32(const char *p, bool whole, uint32_t *r)
{
    if (whole)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p)
                     : "memory");
    else {
        const uint4 a = ld_after_v4(p), b = ld_after_v4(p + 16);
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
        r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
    }
}

__device__ __forceinline__ void store32(char *p, bool whole, const uint32_t *r)
{
    if (whole)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                     "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

// 16 columns of a thread's row as bf16
__device__ __forceinline__ void store_bf16x16(char *p, bool whole, const float *v)
{
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        r[j] = bf16x2_from_f32(v[2 * j], v[2 * j + 1]);
    store32(p, whole, r);
}

// 32 columns as bf16 or fp32
__device__ __forceinline__ void store_cols(char *p, bool whole, bool bf16, const float *v)
{
    if (bf16) {
        store_bf16x16(p, whole, v);
        store_bf16x16(p + 32, whole, v + 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store32(p + 32 * i, whole, reinterpret_cast<const uint32_t *>(v + 8 * i));
    }
}

// v += the W values at p in shared memory
template <int W>
__device__ __forceinline__ void add_bias(float (&v)[W], uint32_t p)
{
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
        const uint4 b = ld_shared_v4(p + j * 16);
        v[4 * j] += __uint_as_float(b.x);
        v[4 * j + 1] += __uint_as_float(b.y);
        v[4 * j + 2] += __uint_as_float(b.z);
        v[4 * j + 3] += __uint_as_float(b.w);
    }
}

__device__ __forceinline__ uint32_t (&bits(float (&v)[32]))[32] { return *reinterpret_cast<uint32_t(*)[32]>(&v); }

__device__ __forceinline__ bool whole32(const void *p, int64_t row_bytes)
{
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)row_bytes) & 31) == 0;
}

// GELU: an ungated tile's activation is gelu, whose code is the longest: two copies of it, as the others have,
// and instructions that wait for one another cost 8192 x 1920 x 1152 70 us, this form 49; the others lose 5% to one copy.
template <bool GATED, bool GELU>
__global__ void __launch_bounds__(kThreads, 1) gemm_act_kernel(const __grid_constant__ ActParams prm)
{
    constexpr int BN = GATED ? 128 : 256;   // output columns of a tile
    using S = Smem<GATED>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kOffBar);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;   // [kSteps], by K-step
    uint64_t *tempty = tfull + kSteps;   // [2], by buffer
    uint64_t *park_full = tempty + 2;    // [2], by tile: its sums are in TMEM
    uint64_t *final_bar = park_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
    volatile int *step_buf = abort_flag + 1;          // [kSteps] buffer of a K-step
    volatile int *park_buf = step_buf + kSteps;       // [2] buffer of a tile's park

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const ActEpilogue &e = prm.e;
    const int KB = e.K / 128, mt = (e.M + 127) / 128, nt = (e.N + BN - 1) / BN, tiles = mt * nt;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int i = 0; i < kSteps; ++i)
            mbar_init(tfull + i, 2);   // the MMAs, and the record of their buffer
        for (int b = 0; b < 2; ++b) {
            mbar_init(tempty + b, 8);
            mbar_init(park_full + b, 8);
        }
        mbar_init(final_bar, 1);
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
                    uint8_t *b = smem + S::kOffB + stage * kBBytes;
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
            drain_loads(full, kStages, issued, prm.timeout_ns);
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            constexpr uint32_t idesc = idesc_f8_e4m3(128, 256);
            int stage = 0, buf = 1;
            uint32_t ph = 0, step = 0, use0 = 0, use1 = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                for (int kb = 0; kb < KB; ++kb, ++step) {
                    // the other buffer than the last step's, or the first of the two that is free
                    buf ^= 1;
                    uint64_t t0 = 0;
                    for (uint32_t tries = 1; !mbar_test_wait(tempty + buf, ((buf ? use1 : use0) & 1) ^ 1); ++tries) {
                        buf ^= 1;
                        if (tries % 256 != 0)
                            continue;
                        const uint64_t now = globaltimer();
                        t0 = t0 == 0 ? now : t0;
                        if (*abort_flag || now - t0 > prm.timeout_ns) {
                            if (!*abort_flag) {
                                *abort_flag = 1;
                                report(prm.status, kErrTimeout, SITE_MMA_TMEM_EMPTY);
                            }
                            ok = false;
                            break;
                        }
                    }
                    if (!ok || !mbar_wait(full + stage, ph, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_FULL)) {
                        ok = false;
                        break;
                    }
                    use0 += buf ? 0u : 1u;
                    use1 += buf ? 1u : 0u;
                    tc_fence_after();
                    const uint64_t ad = desc_kmajor_sw128(smem_u32(smem + stage * kABytes));
                    const uint64_t bd = desc_kmajor_sw128(smem_u32(smem + S::kOffB + stage * kBBytes));
#pragma unroll
                    for (int k = 0; k < 4; ++k)   // 4 x 32 of K = one 128-byte swizzle row
                        mma_f8(tmem_base + buf * 256, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
                    tc_commit(empty + stage);
                    tc_commit(tfull + step % kSteps);
                    step_buf[step % kSteps] = buf;
                    mbar_arrive(tfull + step % kSteps);   // for what this thread wrote
                    if (++stage == kStages) {
                        stage = 0;
                        ph ^= 1;
                    }
                }
            }
            tc_commit(final_bar);
            wait_teardown(final_bar, prm.status, prm.timeout_ns);
        }
    } else if (warp < 12) {
        setmaxnreg_inc<kRegsPromote<GATED, GELU>>();
        // ---------------------------------------------------- promotion
        const int q = warp & 3, h = (warp - 4) >> 2;   // lane quarter, half of the accumulator's columns
        const int row = q * 32 + lane;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16) + h * 128;
        // a tile past the last column block (an odd number of them) has no scales to read
        const int last_block = (GATED ? 2 * e.N : e.N) / 128 - 1;
        uint32_t step = 0, tile = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++tile) {
            const Tile c = decode(t, mt, nt, BN);
            const float *sa_row = prm.sa + (int64_t)min(c.m0 + row, e.M - 1) * KB;
            const float *sb = prm.sb + (int64_t)min(last_block, (GATED ? h * e.N + c.n0 : c.n0 + h * 128) / 128) * KB;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j)
                acc[j] = 0.0f;
            float a_next = __ldg(sa_row), b_next = __ldg(sb);
            for (int kb = 0; kb < KB; ++kb, ++step) {
                const float s = a_next * b_next;
                if (kb + 1 < KB) {
                    a_next = __ldg(sa_row + kb + 1);
                    b_next = __ldg(sb + kb + 1);
                }
                if (!mbar_wait(tfull + step % kSteps, step / kSteps & 1, abort_flag, prm.status, prm.timeout_ns, SITE_EPI_TMEM_FULL)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int buf = step_buf[step % kSteps];
                const uint32_t taddr = lane_base + buf * 256;
                const bool parks = kb == KB - 1;
                // 16-column loads, the next one issued before the current one's promotions
                uint32_t ra[16], rb[16];
                tmem_ld_x16(taddr, ra);
                tmem_wait_ld(ra);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t(&cur)[16] = (i & 1) ? rb : ra;
                    uint32_t(&nxt)[16] = (i & 1) ? ra : rb;
                    if (i + 1 < 8)
                        tmem_ld_x16(taddr + (i + 1) * 16, nxt);
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        fma2(acc[i * 16 + j], acc[i * 16 + j + 1], s, cur[j], cur[j + 1]);
                    if (i + 1 < 8) {
                        tmem_wait_ld(nxt);
                        if (i + 2 == 8 && !parks) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(tempty + buf);
                        }
                    }
                }
                if (parks) {
                    // the finish warps read them from here and release the buffer
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        tmem_st_x32(taddr + i * 32, &acc[i * 32]);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (warp == 4)
                            park_buf[tile & 1] = buf;
                        mbar_arrive(park_full + (tile & 1));
                    }
                }
            }
        }
    } else {
        setmaxnreg_dec<kRegsFinish<GATED, GELU>>();
        // ---------------------------------------------------- finish
        const int q = warp & 3;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
        const int P = GATED ? 2 * e.N : e.N;
        const int r_bytes = e.r_bf16 ? 2 : 4, c_bytes = e.c_bf16 ? 2 : 4;
        const bool r_whole = whole32(e.res, e.rs * r_bytes), c_whole = whole32(e.C, e.cs * c_bytes);
        const bool z_whole = whole32(e.z, 0), q_whole = whole32(e.q, 0);   // N is a multiple of 128
        const uint32_t bias = smem_u32(smem + S::kOffBias + q * 1024);   // the warp's own copy
        const uint32_t res_ring = smem_u32(smem + S::kOffRes + q * kResBytes);   // ungated
        uint32_t parked = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++parked) {
            const Tile c = decode(t, mt, nt, BN);
            const int64_t m = c.m0 + q * 32 + lane;
            const bool inside = m < e.M;
            const int cols = min(BN, e.N - c.n0);   // a multiple of 128
            // Gated: the residual's columns, 64 ahead of their use as bf16 and 32 as fp32: blocks of 32 go to
            // the two halves of these registers in turn, or fill both.
            const char *res = static_cast<const char *>(e.res) + (m * e.rs + c.n0) * r_bytes;
            const bool has_res = e.res != nullptr && inside;
            uint32_t ahead[32];
            auto fetch_residual = [&](int col, int half) {   // half is a constant where it is used
                if (!has_res || col >= cols)
                    return;
                if (e.r_bf16) {
                    load32(res + col * 2, r_whole, ahead + 16 * half);
                    load32(res + col * 2 + 32, r_whole, ahead + 16 * half + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        load32(res + col * 4 + 32 * i, r_whole, ahead + 8 * i);
                }
            };
            // Ungated: 64 columns at a time, in shared memory: a bf16 tile's four such blocks, or two of an fp32
            // one's.  Unit u of row r lies at u ^ (r % 8), so that the rows that eight lanes read lie in different
            // banks.
            const int block_bytes = 32 * 64 * r_bytes, blocks = kResBytes / block_bytes, units = 4 * r_bytes;
            auto stage_residual = [&](int col) {
                if (e.res != nullptr && col < cols) {
                    const uint32_t to = res_ring + col / 64 % blocks * block_bytes;
                    const int u = lane % units;
                    const char *from = static_cast<const char *>(e.res) + ((m - lane) * e.rs + c.n0 + col) * r_bytes + u * 16;
                    for (int row = lane / units; row < 32; row += 32 / units)
                        if (m - lane + row < e.M)
                            cp_async_cg16(to + row * 64 * r_bytes + (u ^ row % 8) * 16, from + row * e.rs * r_bytes);
                }
                cp_async_commit();
            };
            if constexpr (GATED) {
                fetch_residual(0, 0);
                if (e.r_bf16)
                    fetch_residual(32, 1);
            } else {
                for (int i = 0; i < blocks; ++i)
                    stage_residual(i * 64);
            }
            if (e.bias != nullptr) {
                // 256 sums' bias: a tile's columns, or 128 of both halves
                __syncwarp();   // every lane is through with the last tile's
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = lane + 32 * i, n = c.n0 + (GATED ? k % 32 : k) * 4;   // four columns
                    float4 b = make_float4(0, 0, 0, 0);
                    if (n < e.N)
                        b = __ldg(reinterpret_cast<const float4 *>(e.bias + (GATED && i ? e.N : 0) + n));
                    st_shared_v4(bias + k * 16, make_uint4(__float_as_uint(b.x), __float_as_uint(b.y), __float_as_uint(b.z), __float_as_uint(b.w)));
                }
                __syncwarp();
            }
            if (GATED && e.res != nullptr) {
                // the next tile's rows of it into L2
                const Tile d = decode(min(t + (int)gridDim.x, tiles - 1), mt, nt, BN);
                const int64_t row = d.m0 + q * 32 + lane;
                if (row < e.M)
                    for (int i = 0; i < min(BN, e.N - d.n0) * r_bytes; i += 128)
                        prefetch_l2(static_cast<const char *>(e.res) + (row * e.rs + d.n0) * r_bytes + i);
            }
            if (!mbar_wait(park_full + (parked & 1), parked / 2 & 1, abort_flag, prm.status, prm.timeout_ns, SITE_PARK_FULL))
                break;
            tc_fence_after();
            const int buf = park_buf[parked & 1];
            const uint32_t park = lane_base + buf * 256;
            float top = 0.0f;
            // 32 columns of out from their sums v
            auto block = [&](float (&v)[32], int col, int half) {
                const int n0 = c.n0 + col;
                if (e.bias != nullptr)
                    add_bias(v, bias + col * 4);
                char *z = reinterpret_cast<char *>(e.z) + (m * P + n0) * 2;
                if (e.z != nullptr && inside)
                    store_cols(z, z_whole, true, v);
                if constexpr (GELU) {
                    gelu_values(v);
                } else {
                    with_act(e.act, [&](auto act) {
                        constexpr int ACT = decltype(act)::value;
                        if constexpr (ACT != ACT_NONE && (GATED || ACT != ACT_GELU)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                v[i] = act_value<ACT>(v[i]);
                        }
                    });
                }
                if (GATED) {
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        float u[16];
                        uint32_t(&r)[16] = *reinterpret_cast<uint32_t(*)[16]>(&u);
                        tmem_ld_x16(park + 128 + col + i, r);
                        tmem_wait_ld(r);
                        if (e.bias != nullptr)
                            add_bias(u, bias + 512 + (col + i) * 4);
                        if (e.z != nullptr && inside)
                            store_bf16x16(z + ((int64_t)e.N + i) * 2, z_whole, u);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[i + j] *= u[j];
                    }
                }
                if (!GATED && e.res != nullptr) {
                    const uint32_t row = res_ring + col / 64 % blocks * block_bytes + lane * 64 * r_bytes;
                    const int u = half * 2 * r_bytes, turn = lane % 8;
                    if (e.r_bf16) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 a = ld_shared_v4(row + ((u + i) ^ turn) * 16);
                            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[8 * i + 2 * j] += bf16_lo(w[j]);
                                v[8 * i + 2 * j + 1] += bf16_hi(w[j]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 a = ld_shared_v4(row + ((u + i) ^ turn) * 16);
                            v[4 * i] += __uint_as_float(a.x);
                            v[4 * i + 1] += __uint_as_float(a.y);
                            v[4 * i + 2] += __uint_as_float(a.z);
                            v[4 * i + 3] += __uint_as_float(a.w);
                        }
                    }
                }
                if (GATED && has_res) {
                    if (e.r_bf16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            v[2 * i] += bf16_lo(ahead[16 * half + i]);
                            v[2 * i + 1] += bf16_hi(ahead[16 * half + i]);
                        }
                        fetch_residual(col + 64, half);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] += __uint_as_float(ahead[i]);
                        fetch_residual(col + 32, 0);
                    }
                }
                if (e.C != nullptr && inside)
                    store_cols(static_cast<char *>(e.C) + (m * e.cs + n0) * c_bytes, c_whole, e.c_bf16, v);
                if (e.q != nullptr) {
                    // one scale per row and 128 columns: they wait in the park for it
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        top = fmaxf(top, fabsf(v[i]));   // skips NaN
                    tmem_st_x32(park + col, v);
                }
            };
            auto finish_codes = [&](int col0) {   // of 128 columns whose values wait in the park
                tmem_wait_st();
                const float scale = __fdiv_rn(top, 448.0f);
                const Enc enc(scale);
#pragma unroll 1
                for (int i = col0; i < col0 + 128; i += 32) {
                    float v[32];
                    tmem_ld_x32(park + i, bits(v));
                    tmem_wait_ld(bits(v));
                    uint32_t o[8];
                    enc.codes(v, o);
                    if (inside)
                        store32(reinterpret_cast<char *>(e.q) + m * e.N + c.n0 + i, q_whole, o);
                }
                if (inside)
                    e.scales[m * (e.N / 128) + (c.n0 + col0) / 128] = scale;
                top = 0.0f;
            };
            if constexpr (!GELU) {
#pragma unroll 1
                for (int col = 0; col < cols; col += 64) {
                    float v[32], w[32];
                    tmem_ld_x32(park + col, bits(v));
                    tmem_wait_ld(bits(v));
                    if (!GATED)   // under way while the first block is taken through
                        tmem_ld_x32(park + col + 32, bits(w));
                    if (!GATED && e.res != nullptr) {
                        if (e.r_bf16)
                            cp_async_wait<3>();   // all but what has been asked for since
                        else
                            cp_async_wait<1>();
                        __syncwarp();
                    }
                    block(v, col, 0);
                    if (GATED)
                        tmem_ld_x32(park + col + 32, bits(w));
                    tmem_wait_ld(bits(w));
                    block(w, col + 32, 1);
                    if (!GATED) {
                        __syncwarp();   // the residual's block is read
                        stage_residual(col + 64 * blocks);
                    }
                    if (e.q != nullptr && col % 128 == 64)
                        finish_codes(col - 64);
                }
            } else {
                // the next block's sums are under way in w while v is taken through
                float v[32], w[32];
                tmem_ld_x32(park, bits(w));
                tmem_wait_ld(bits(w));
#pragma unroll 1
                for (int col = 0; col < cols; col += 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = w[i];
                    if (col + 32 < cols)
                        tmem_ld_x32(park + col + 32, bits(w));
                    if (e.res != nullptr && col % 64 == 0) {
                        if (e.r_bf16)
                            cp_async_wait<3>();   // all but what has been asked for since
                        else
                            cp_async_wait<1>();
                        __syncwarp();
                    }
                    block(v, col, col / 32 & 1);
                    if (e.res != nullptr && col % 64 == 32) {
                        __syncwarp();   // the residual's block is read
                        stage_residual(col - 32 + 64 * blocks);
                    }
                    tmem_wait_ld(bits(w));
                    if (e.q != nullptr && col % 128 == 96)
                        finish_codes(col - 96);
                }
            }
            // the park is read: the MMA may refill the buffer.  Two of the eight arrivals it waits for
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(tempty + buf);
                mbar_arrive(tempty + buf);
            }
        }
        cp_async_wait<0>();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, 512);
}

}  // namespace

template <bool GATED, bool GELU>
static bool split_ok()
{
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, gemm_act_kernel<GATED, GELU>) == cudaSuccess && a.numRegs * kThreads >= kRegsNeeded<GATED, GELU>;
}

bool gemm_act_split_ok() { return split_ok<true, false>() && split_ok<false, true>() && split_ok<false, false>(); }

// How long a launch takes, about: 0.45 us per 128 of K and 5 us per tile that a CTA does one after
// another, and 3 us (measured: 31 us at one tile of K = 7168, 14.5 at 2048, 12.4 at 1152).
int64_t gemm_act_tiles_ns(int M, int N, int K, bool gated, int num_sms)
{
    const int bn = gated ? 128 : 256;
    const int64_t tiles = (int64_t)((M + 127) / 128) * ((N + bn - 1) / bn);
    return (tiles + num_sms - 1) / num_sms * (450 * (K / 128) + 5000) + 3000;
}

template <bool GATED, bool GELU>
static cudaError_t launch_typed(const ActParams &p, int num_sms, cudaStream_t st)
{
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(gemm_act_kernel<GATED, GELU>), Smem<GATED>::kBytes);
    if (e != cudaSuccess)
        return e;
    const int bn = GATED ? 128 : 256;
    const int64_t tiles = (int64_t)((p.e.M + 127) / 128) * ((p.e.N + bn - 1) / bn);
    gemm_act_kernel<GATED, GELU><<<(int)std::min<int64_t>(tiles, num_sms), kThreads, Smem<GATED>::kBytes, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_gemm_act(const ActParams &p, int num_sms, cudaStream_t st)
{
    if (p.e.gated)
        return launch_typed<true, false>(p, num_sms, st);
    return p.e.act == ACT_GELU ? launch_typed<false, true>(p, num_sms, st) : launch_typed<false, false>(p, num_sms, st);
}

}  // namespace gemmar

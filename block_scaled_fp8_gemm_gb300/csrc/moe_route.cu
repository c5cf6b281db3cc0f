// moe_route.cu -- which experts a token goes to, and with which weights (moe_route).
//
//   l[t,e] = sum_h x[t,h] w[e,h];   p = softmax(l) or sigmoid(l);   the k largest of p + bias
//
// For few tokens it reads the router once and is bound by latency, and from some tens of tokens
// on by fp32 FMAs (the sums must tell neighbours in the order apart, so they are no tensor-core
// sums).  Up to 8 tokens a CTA computes the logits of a few of them and of few experts with
// all its threads along h, and the one that finishes last chooses, a warp per token.  More go by
// tiles of 32 tokens and 32 experts, h cut into as many parts as fill the SMs (96 tokens, 256
// experts, h = 7168: 9 000 cycles of FMAs an SM at best), and a second launch adds the parts and
// chooses.  One token of 64 experts takes 4.7 us, 8 of 256 11 us, 96 of 256 18.8 us.
//
// The order of two experts whose scores agree to fp32's rounding would depend on how the
// sums are split.  Such tokens are decided in 64 bits: the logits in question are summed
// again with what their roundings lost (20 us for a pair at h = 7168, for about one token in two
// thousand).
// Without a bias the order is the logits' own, which neither saturates nor underflows.
#include <algorithm>

#include "e4m3_encode.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 8;        // tokens of the first form: one warp chooses for each
static_assert(kTokens == kWarps, "a warp per token");
constexpr int kMaxExperts = 1024;

// 8 values of a row of the router
template <bool BF>
__device__ __forceinline__ void load8(const void *row, int h, float (&v)[8])
{
    if (BF) {
        const uint4 r = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + h));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + h);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

__device__ __forceinline__ const void *router_row(const RouteArgs &a, int e)
{
    return static_cast<const char *>(a.w) + (int64_t)e * a.H * (a.w_bf16 ? 2 : 4);
}

// A number as an unsigned one of the same order, never 0 but for a NaN.  The warp's largest is then
// one instruction, and 0 what is not to be chosen.
__device__ __forceinline__ uint32_t key_of(float s)
{
    const uint32_t b = __float_as_uint(s);
    return s == s ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float score_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); }

// x[t] . w[e] by the whole warp, every product and sum with its rounding error carried along
// (error-free sums and products by the published methods of Knuth and Dekker): about 2^-45 of the
// terms' sizes, on the fp32 units, as those for fp64 are few.
__device__ double logit64(const RouteArgs &a, int t, int e)
{
    const int lane = threadIdx.x & 31;
    const uint16_t *x = a.x + (int64_t)t * a.xs;
    const void *w = router_row(a, e);
    float hi = 0.0f, lo = 0.0f;
    for (int h = lane * 8; h < a.H; h += 256) {
        float xv[8], wv[8];
        load8<true>(x, h, xv);
        if (a.w_bf16)
            load8<true>(w, h, wv);
        else
            load8<false>(w, h, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = __fmul_rn(xv[i], wv[i]), pe = __fmaf_rn(xv[i], wv[i], -p);
            const float s = __fadd_rn(hi, p), b = __fsub_rn(s, hi);
            lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(p, b)), pe));
            hi = s;
        }
    }
    double s = (double)hi + (double)lo;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

// What orders the experts, in double: the logit, or the score with its bias.
struct Order64 {
    bool soft, biased;
    double top, sum;      // of the softmax
    __device__ double of(double logit, double bias) const
    {
        if (!biased)
            return logit;
        return (soft ? exp(logit - top) / sum : 1.0 / (1.0 + exp(-logit))) + bias;
    }
};

// The first k in double of the experts whose fp32 order value is at least `least`, for the rare
// token where fp32 cannot tell: lane j gets the j-th.  value: the fp32 order values, in shared
// memory; zero: every logit of the token is exactly 0.
// Only experts with another one twice `tol` away or nearer need it: between the others fp32 can tell.
__device__ __noinline__ int decide64(const RouteArgs &a, int t, const float *value, float least, float tol, int k, Order64 o, bool zero)
{
    const int lane = threadIdx.x & 31;
    double mine = -INFINITY;   // lane j: the j-th best so far, and whose
    int mine_e = -1, count = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const float f = e0 + lane < a.E ? value[e0 + lane] : -INFINITY;
        unsigned todo = __ballot_sync(0xffffffffu, f >= least && e0 + lane < a.E);
        while (todo) {
            const int who = __ffs(todo) - 1, e = e0 + who;
            todo &= todo - 1;
            const float mine32 = __shfl_sync(0xffffffffu, f, who), near = 2.0f * (tol + (o.biased ? 0x1p-21f * fabsf(mine32) : 0.0f));
            bool alone = true;
            for (int i = lane; i < a.E; i += 32)
                alone = alone && (i == e || !(fabsf(value[i] - mine32) <= near));
            double d = mine32;
            if (!__all_sync(0xffffffffu, alone)) {
                const double x = zero ? 0.0 : logit64(a, t, e);
                if (x > -INFINITY && x < INFINITY)   // an infinite logit's fp32 value is exact
                    d = o.of(x, o.biased ? (double)__ldg(a.bias + e) : 0.0);
            }
            // its place behind the ones that are not smaller (equal ones have lower numbers)
            const int place = __popc(__ballot_sync(0xffffffffu, lane < count && mine >= d));
            const double up = __shfl_up_sync(0xffffffffu, mine, 1);
            const int up_e = __shfl_up_sync(0xffffffffu, mine_e, 1);
            if (lane >= place) {
                mine = lane == place ? d : up;
                mine_e = lane == place ? e : up_e;
            }
            count = min(count + 1, 32);
        }
    }
    return lane < k ? mine_e : -1;
}

// Weights over their sum where the scores of all chosen are too small for fp32 (a bias that takes
// out the experts before them; a sigmoid of logits far below 0): both scores are then e^l but for a factor
// that the sum takes out.  Lane j < chosen has the j-th expert and gets its weight.
__device__ __noinline__ float tiny_weights(const RouteArgs &a, int t, int mine, int chosen)
{
    const int lane = threadIdx.x & 31;
    double logit = -INFINITY;
    for (int j = 0; j < chosen; ++j) {
        const double x = logit64(a, t, __shfl_sync(0xffffffffu, mine, j));
        logit = lane == j ? x : logit;
    }
    double top = logit;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
    const double w = logit > -INFINITY ? exp(logit - top) : 0.0;
    double all = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        all += __shfl_xor_sync(0xffffffffu, all, d);
    return all > 0.0 ? (float)(w / all) : 0.0f;
}

// One warp chooses token t's experts from its logits in global memory, which other CTAs wrote, in
// `parts` to be added.  score: [2 E] in shared memory, the warp's own.  PER: experts of a lane
// (E <= 32 PER), lane + 32 i.
template <int PER>
__device__ __forceinline__ void choose(const RouteArgs &a, int t, const float *logits, int parts, float *score)
{
    const int lane = threadIdx.x & 31;
    const bool soft = a.score == 0;
    float *order = score + a.E;
    float v[PER], bias[PER];             // logits, then scores without the bias
    float top = -INFINITY, big = 0.0f;   // largest logit, largest size of one
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        bias[i] = e < a.E && a.bias != nullptr ? __ldg(a.bias + e) : 0.0f;
        v[i] = e < a.E ? __ldcg(logits + (int64_t)t * a.E + e) : -INFINITY;
    }
    // many loads under way: a lane's experts of four parts
    const float *from = logits + (int64_t)t * a.E + lane;
#pragma unroll(PER <= 8 ? 4 : 1)
    for (int p = 1; p < parts; ++p) {
        from += (int64_t)a.T * a.E;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < a.E)
                v[i] += __ldcg(from + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        top = fmaxf(top, v[i]);          // skips NaN
        if (fabsf(v[i]) < INFINITY)
            big = fmaxf(big, fabsf(v[i]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
    // exponentials to be divided by their sum, or sigmoids
    const bool biased = a.bias != nullptr;
    uint32_t key[PER];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = lane + 32 * i < a.E ? key_of(v[i]) : 0u;   // the order without a bias
        // of the softmax's both may be infinite; a NaN logit is no expert's
        const float x = soft && v[i] == top ? 1.0f : expf(soft ? v[i] - top : -v[i]);
        const float p = soft ? x : __fdividef(1.0f, 1.0f + x);
        if (lane + 32 * i < a.E) {
            score[lane + 32 * i] = p;
            order[lane + 32 * i] = v[i];
            sum += p >= 0.0f ? p : 0.0f;
        }
        v[i] = p;
    }
    float scale = 1.0f;
    if (soft) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        scale = 1.0f / sum;
    }
    // how far fp32's rounding may move what orders: the logits' sums to 2^-20 of the largest
    // logit (twenty times the spread of such sums), scores besides by a few units in the last place
    float tol = 0x1p-20f * big;
    if (biased) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float s = v[i] * scale + bias[i];
            if (lane + 32 * i < a.E) {
                key[i] = s > -INFINITY ? key_of(s) : 0u;
                order[lane + 32 * i] = s;
            }
        }
        tol = tol * (soft ? scale : 0.25f) + 0x1p-21f * scale;
    }
    bool close = false;                  // whether neighbours in the order are too close to tell
    int mine = -1, chosen = 0;           // lane j keeps the j-th choice (k <= 16)
    float last = INFINITY, cut = -INFINITY;
#pragma unroll 1
    for (int j = 0; j <= a.k; ++j) {     // one past the last, to see how near it is
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best == 0)
            break;
        const float s = score_of(best);
        close = close || last - s <= tol + (biased ? 0x1p-21f * fabsf(s) : 0.0f);   // no two infinities
        last = s;
        if (j == a.k)
            break;
        int e = INT32_MAX;               // of equal ones the lowest
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            e = key[i] == best ? lane + 32 * i : e;
        e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            key[i] = e == lane + 32 * i ? 0u : key[i];
        cut = s;
        ++chosen;
        if (lane == j)
            mine = e;
    }
    __syncwarp();
    if (close && chosen > 0) {
        double sum64 = 1.0;
        if (soft && biased) {
            sum64 = 0.0;
            for (int e = lane; e < a.E; e += 32)
                sum64 += score[e] >= 0.0f ? (double)score[e] : 0.0;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                sum64 += __shfl_xor_sync(0xffffffffu, sum64, d);
        }
        const float near = 2.0f * (tol + (biased ? 0x1p-21f * fabsf(cut) : 0.0f));
        mine = decide64(a, t, order, near > 0.0f ? cut - near : cut, tol, chosen, Order64{soft, biased, (double)top, sum64}, big == 0.0f);
    }
    float w = mine >= 0 ? score[mine] * scale : 0.0f, all = w;
    if (a.renorm) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            all += __shfl_xor_sync(0xffffffffu, all, d);
        w = all < 0x1p-100f && chosen > 0 ? tiny_weights(a, t, mine, chosen) : w / all;
    }
    if (lane < a.k) {
        a.ids[(int64_t)t * a.k + lane] = mine;
        a.weights[(int64_t)t * a.k + lane] = mine >= 0 ? w * a.factor : 0.0f;
    }
}

__device__ __forceinline__ void choose_token(const RouteArgs &a, int t, const float *logits, int parts, float *score)
{
    if (a.E <= 64)
        choose<2>(a, t, logits, parts, score);
    else if (a.E <= 256)
        choose<8>(a, t, logits, parts, score);
    else
        choose<32>(a, t, logits, parts, score);
}

// At most kTokens tokens.  grid: experts / EB; logits fp32 [T,E]; done: zero before and after.
template <int TB, int EB, bool BF>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a, float *logits, uint32_t *done)
{
    __shared__ float part[kWarps][TB * EB];
    extern __shared__ __align__(16) uint8_t smem[];
    float *scores = reinterpret_cast<float *>(smem);   // [kWarps][2 E]
    __shared__ bool chooses;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.x * EB;
    for (int t0 = 0; t0 < a.T; t0 += TB) {
        float acc[TB * EB] = {};
        for (int h = threadIdx.x * 8; h < a.H; h += kThreads * 8) {
            float x[TB][8];
#pragma unroll
            for (int i = 0; i < TB; ++i)
                load8<true>(a.x + (int64_t)min(t0 + i, a.T - 1) * a.xs, h, x[i]);
#pragma unroll
            for (int j = 0; j < EB; ++j) {
                float w[8];
                load8<BF>(router_row(a, min(e0 + j, a.E - 1)), h, w);
#pragma unroll
                for (int i = 0; i < TB; ++i)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[i * EB + j] = fmaf(x[i][c], w[c], acc[i * EB + j]);
            }
        }
#pragma unroll
        for (int i = 0; i < TB * EB; ++i) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            if (lane == 0)
                part[warp][i] = acc[i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < TB * EB; i += kThreads) {
            float s = part[0][i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                s += part[w][i];
            const int t = t0 + i / EB, e = e0 + i % EB;
            if (t < a.T && e < a.E)
                __stcg(logits + (int64_t)t * a.E + e, s);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        chooses = add_acq_rel(done, 1u) == gridDim.x - 1;   // then all CTAs' logits are visible
        if (chooses)
            *done = 0;
    }
    __syncthreads();
    if (chooses && warp < a.T)
        choose_token(a, warp, logits, 1, scores + warp * 2 * a.E);
}

// ---- tiles of 32 tokens x 32 experts

constexpr int kTile = 32, kChunk = 256, kStages = 4, kMaxParts = 16;   // kChunk: columns of a stage

// Rows of the two operands in shared memory, a 16-byte unit longer than a chunk: the rows that
// the lanes of a warp read at a time then lie in different banks.
template <bool BF>
struct TileSmem {
    static constexpr int kXRow = kChunk * 2 + 16, kWRow = kChunk * (BF ? 2 : 4) + 16;
    static constexpr int kStage = kTile * (kXRow + kWRow);
    static constexpr int kBytes = kStages * kStage;
    static_assert(kBytes >= kWarps * kTile * kTile * 4, "the warps' sums lie in the stages");
    static_assert(kBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }

// four bf16 as two pairs of fp32
__device__ __forceinline__ void widen4(uint2 v, uint64_t (&p)[2])
{
    p[0] = pair_of(v.x << 16, v.x & 0xFFFF0000u);
    p[1] = pair_of(v.y << 16, v.y & 0xFFFF0000u);
}

__device__ __forceinline__ void fma_pair(uint64_t &c, uint64_t a, uint64_t b)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

// grid: (parts of h, experts / 32, tokens / 32); out fp32 [part][T][E].  A warp computes the whole
// tile over every eighth run of 32 columns, a lane 4 tokens x 8 experts of it.
template <bool BF>
__global__ void __launch_bounds__(kThreads, 1) route_tile_kernel(const RouteArgs a, float *out)
{
    using S = TileSmem<BF>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.y * kTile, t0 = blockIdx.z * kTile;
    const int part = (a.H + 8 * (int)gridDim.x - 1) / (8 * (int)gridDim.x) * 8;
    const int h0 = min((int)blockIdx.x * part, a.H), h1 = min(h0 + part, a.H);
    const int chunks = (h1 - h0 + kChunk - 1) / kChunk;
    grid_launch_next();   // it waits for this grid's end before it reads
    // a thread copies the same 16 bytes of columns of every 8th row (of w's fp32 rows two such)
    constexpr int PER = BF ? 8 : 4, WU = kChunk / PER / 32;   // columns of 16 bytes of w; units of a thread
    const int u = lane, r0 = warp;
    const uint16_t *xp = a.x + h0 + u * 8;
    const char *wp = static_cast<const char *>(a.w) + (int64_t)(h0 + u * PER) * (16 / PER);
    int64_t xrow[kTile / 8], wrow[kTile / 8];
#pragma unroll
    for (int i = 0; i < kTile / 8; ++i) {
        xrow[i] = (int64_t)min(t0 + r0 + 8 * i, a.T - 1) * a.xs;
        wrow[i] = (int64_t)min(e0 + r0 + 8 * i, a.E - 1) * a.H * (16 / PER);
    }
    auto copy = [&](int c) {
        if (c < chunks) {
            const uint32_t st = smem_u32(smem + c % kStages * S::kStage) + u * 16;
            const uint32_t x = st + r0 * S::kXRow, w = st + kTile * S::kXRow + r0 * S::kWRow;
            const int left = h1 - h0 - c * kChunk;   // columns of the part from this chunk on
            const bool ok = u * 8 < left;
#pragma unroll
            for (int i = 0; i < kTile / 8; ++i)
                cp_async_cg16_or_zero(x + 8 * i * S::kXRow, ok ? xp + xrow[i] + c * kChunk : a.x, ok);
#pragma unroll
            for (int j = 0; j < WU; ++j) {
                const bool in = (u + 32 * j) * PER < left;
#pragma unroll
                for (int i = 0; i < kTile / 8; ++i)
                    cp_async_cg16_or_zero(w + 8 * i * S::kWRow + 512 * j,
                                          in ? wp + wrow[i] + (c * kChunk + 32 * j * PER) * (16 / PER) : static_cast<const char *>(a.w), in);
            }
        }
        cp_async_commit();
    };
    for (int c = 0; c < kStages - 1; ++c)
        copy(c);
    // tokens ti + 8 i, experts ei + 4 j
    const int ti = lane >> 2, ei = lane & 3;
    uint64_t acc[4][8] = {};   // sums over the even and the odd columns
    for (int c = 0; c < chunks; ++c) {
        cp_async_wait<kStages - 2>();
        __syncthreads();   // everyone's copies of chunk c are there, and chunk c - 1 is read
        copy(c + kStages - 1);
        const uint32_t x = smem_u32(smem + c % kStages * S::kStage) + ti * S::kXRow;
        const uint32_t w = smem_u32(smem + c % kStages * S::kStage) + kTile * S::kXRow + ei * S::kWRow;
#pragma unroll 4
        for (int col = warp * 32; col < warp * 32 + 32; col += 4) {
            uint64_t xv[4][2], wv[2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                widen4(ld_shared_v2(x + 8 * i * S::kXRow + col * 2), xv[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (BF) {
                    widen4(ld_shared_v2(w + 4 * j * S::kWRow + col * 2), wv);
                } else {
                    const uint4 r = ld_shared_v4(w + 4 * j * S::kWRow + col * 4);
                    wv[0] = pair_of(r.x, r.y);
                    wv[1] = pair_of(r.z, r.w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    fma_pair(acc[i][j], xv[i][0], wv[0]);
                    fma_pair(acc[i][j], xv[i][1], wv[1]);
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem);   // [warp][token][expert]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sums[(warp * kTile + ti + 8 * i) * kTile + ei + 4 * j] =
                __uint_as_float((uint32_t)acc[i][j]) + __uint_as_float((uint32_t)(acc[i][j] >> 32));
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kTile; i += kThreads) {
        float s = sums[i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            s += sums[w * kTile * kTile + i];
        const int t = t0 + i / kTile, e = e0 + i % kTile;
        if (t < a.T && e < a.E)
            __stcg(out + ((int64_t)blockIdx.x * a.T + t) * a.E + e, s);
    }
}

// a warp per token
__global__ void __launch_bounds__(128) route_choose_kernel(const RouteArgs a, const float *logits, int parts)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
    grid_wait();
    if (t < a.T)
        choose_token(a, t, logits, parts, reinterpret_cast<float *>(smem) + (threadIdx.x >> 5) * 2 * a.E);
}

// The number of parts that ends soonest: waves of CTAs, each as long as a part and two chunks
// more (its first copies, and adding the sums).
int tile_parts(const RouteArgs &a, int num_sms)
{
    const int tiles = ((a.E + kTile - 1) / kTile) * ((a.T + kTile - 1) / kTile);
    int best = 1;
    int64_t least = INT64_MAX;
    for (int p = 1; p <= std::min(kMaxParts, (a.H + kChunk - 1) / kChunk); ++p) {
        const int64_t cost = (int64_t)((tiles * p + num_sms - 1) / num_sms) * ((a.H + p - 1) / p + 2 * kChunk);
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return best;
}

template <int TB, int EB, bool BF>
cudaError_t launch_typed(const RouteArgs &a, float *ws, uint32_t *counter, cudaStream_t st)
{
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(route_kernel<TB, EB, BF>), kWarps * kMaxExperts * 8);
    if (e != cudaSuccess)
        return e;
    route_kernel<TB, EB, BF><<<(a.E + EB - 1) / EB, kThreads, a.T * a.E * 8, st>>>(a, ws, counter);
    return cudaGetLastError();
}

template <bool BF>
cudaError_t launch_tiles(const RouteArgs &a, float *ws, int num_sms, cudaStream_t st)
{
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(route_tile_kernel<BF>), TileSmem<BF>::kBytes);
    if (e != cudaSuccess)
        return e;
    const cudaError_t c = ensure_dynamic_smem(reinterpret_cast<const void *>(route_choose_kernel), 4 * kMaxExperts * 8);
    if (c != cudaSuccess)
        return c;
    const int parts = tile_parts(a, num_sms);
    route_tile_kernel<BF><<<dim3(parts, (a.E + kTile - 1) / kTile, (a.T + kTile - 1) / kTile), kThreads, TileSmem<BF>::kBytes, st>>>(a, ws);
    return launch(route_choose_kernel, dim3((a.T + 3) / 4), 128, (size_t)4 * a.E * 8, 1, true, st, a, static_cast<const float *>(ws), parts);
}

}  // namespace

int64_t route_ws_floats(const RouteArgs &a, int num_sms)
{
    return (int64_t)a.T * a.E * (a.T <= kTokens ? 1 : tile_parts(a, num_sms));
}

cudaError_t launch_route(const RouteArgs &a, float *ws, uint32_t *counter, int num_sms, cudaStream_t st)
{
    if (a.T == 1)
        return a.w_bf16 ? launch_typed<1, 1, true>(a, ws, counter, st) : launch_typed<1, 1, false>(a, ws, counter, st);
    if (a.T <= kTokens)
        return a.w_bf16 ? launch_typed<4, 4, true>(a, ws, counter, st) : launch_typed<4, 4, false>(a, ws, counter, st);
    return a.w_bf16 ? launch_tiles<true>(a, ws, num_sms, st) : launch_tiles<false>(a, ws, num_sms, st);
}

}  // namespace gemmar

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
// chooses, a CTA per token.  One token of 64 experts takes 5.6 us, 8 of 256 11 to 12 us, 96 of 256 19.5 us.
//
// An fp32 sum of n roundings is off by n 2^-24 sum_h |x w| at most, and that sum is at most |x| |w| of
// the rows' norms.  Norms are summed beside the logits; a token with two of its first k + 1 experts
// nearer than such sums can tell is decided in 64 bits, by all warps of its CTA: the logits in question are
// summed again with what their roundings lost.  At h = 7168 and 256 experts that is one token in 25 or so and
// takes 5 to 7 us, of up to 8 tokens one after another: 96 tokens 25 to 26 us, 8 of them 15 on average.
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

// The warps' sums in pairs: three roundings
template <typename F>
__device__ __forceinline__ float sum8(F of)
{
    static_assert(kWarps == 8, "one each");
    return ((of(0) + of(1)) + (of(2) + of(3))) + ((of(4) + of(5)) + (of(6) + of(7)));
}

__device__ __forceinline__ const void *router_row(const RouteArgs &a, int e)
{
    return static_cast<const char *>(a.w) + (int64_t)e * a.H * (a.w_bf16 ? 2 : 4);
}

// What the choice starts from: `parts` sums [T,E] of logits to be added, then the parts' sums of squares of the tokens'
// rows [parts,T], and of each tile of experts the largest sum [parts,tiles].
struct Sums {
    float *at;
    int parts, tiles;
    float slack;      // times both norms: what an fp32 logit may be off by
    __device__ float *logit(const RouteArgs &a, int part, int t, int e) const { return at + ((int64_t)part * a.T + t) * a.E + e; }
    __device__ float *x2(const RouteArgs &a, int part, int t) const { return logit(a, parts, 0, 0) + part * a.T + t; }
    __device__ float *largest_w2(const RouteArgs &a, int i) const { return x2(a, parts, 0) + i; }
    __device__ float *largest_w2(const RouteArgs &a, int part, int tile) const { return largest_w2(a, part * tiles + tile); }
};

int64_t sums_floats(int64_t T, int64_t E, int64_t parts, int64_t tiles) { return parts * (T * E + T + tiles); }

// n roundings in a row, and 2% for second orders and the norms' own.
inline float slack_of(int64_t n) { return 1.02f * 0x1p-24f * (float)n; }
// Squares that fp32 loses, of a row of 65536: added to every sum of squares.
constexpr float kLostSquares = 0x1p-110f;

// A number as an unsigned one of the same order, never 0 but for a NaN.  The warp's largest is then
// one instruction, and 0 what is not to be chosen.
__device__ __forceinline__ uint32_t key_of(float s)
{
    const uint32_t b = __float_as_uint(s);
    return s == s ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float score_of(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key); }

// A thread's share of x . w, `threads` of them side by side, 8 columns at a time: every product and sum with its
// rounding error carried along (error-free sums and products by the published methods of Knuth and Dekker), on
// the fp32 units, as those for fp64 are few.  The errors of 56 terms are added in fp32 and their sums in
// fp64: about 2^-44 of the terms' sizes is lost, and products below 2^-100 lose digits.
template <bool BF>
__device__ __forceinline__ double share64(const uint16_t *x, const void *w, int H, int thread, int threads)
{
    constexpr int kAhead = 7;   // loads under way
    float hi = 0.0f;
    double lost = 0.0;
    for (int h0 = thread * 8; h0 < H; h0 += kAhead * threads * 8) {
        float xv[kAhead][8], wv[kAhead][8];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = h0 + u * threads * 8;
            if (h < H) {
                load8<true>(x, h, xv[u]);
                load8<BF>(w, h, wv[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    xv[u][i] = wv[u][i] = 0.0f;
            }
        }
        float lo = 0.0f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = __fmul_rn(xv[u][i], wv[u][i]), pe = __fmaf_rn(xv[u][i], wv[u][i], -p);
                const float s = __fadd_rn(hi, p), b = __fsub_rn(s, hi);
                lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(p, b)), pe));
                hi = s;
            }
        }
        lost += (double)lo;
    }
    return (double)hi + lost;
}

__device__ __forceinline__ double warp_sum(double s)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}

// One of `warps` warps' part of x[t] . w[e]
__device__ __noinline__ double part64(const RouteArgs &a, int t, int e, int warp, int warps)
{
    const uint16_t *x = a.x + (int64_t)t * a.xs;
    const void *w = router_row(a, e);
    const int thread = warp * 32 + (threadIdx.x & 31);
    return warp_sum(a.w_bf16 ? share64<true>(x, w, a.H, thread, warps * 32) : share64<false>(x, w, a.H, thread, warps * 32));
}

// Weights over their sum where the scores of all chosen are too small for fp32 (a bias that takes
// out the experts before them; a sigmoid of logits far below 0): both scores are then e^l but for a factor
// that the sum takes out.  Lane j < chosen has the j-th expert and gets its weight.
__device__ __noinline__ float tiny_weights(const RouteArgs &a, int t, int mine, int chosen)
{
    const int lane = threadIdx.x & 31;
    double logit = -INFINITY;
    for (int j = 0; j < chosen; ++j) {
        const double x = part64(a, t, __shfl_sync(0xffffffffu, mine, j), 0, 1);
        logit = lane == j ? x : logit;
    }
    double top = logit;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
    const double w = logit > -INFINITY ? exp(logit - top) : 0.0, all = warp_sum(w);
    return all > 0.0 ? (float)(w / all) : 0.0f;
}

// Lane j has the j-th of `chosen` experts: their weights, and both outputs.
__device__ __forceinline__ void finish(const RouteArgs &a, int t, int mine, int chosen, const float *score, float scale)
{
    const int lane = threadIdx.x & 31;
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

// What fp32 knows of a token's order.
struct Choice {
    bool close;       // two of the first k + 1 are too near to tell
    int chosen;
    float tol;        // how near that is, besides 2^-21 of a score with its bias
    float cut;        // the last one's
    float top, err;   // the largest logit, and what a logit may be off by
    float scale;      // of the scores
    bool zero;        // the token's row squares to nothing
};

__device__ __forceinline__ float nearness(const RouteArgs &a, const Choice &c, float s)
{
    return c.tol + (a.bias != nullptr ? 0x1p-21f * fabsf(s) : 0.0f);
}

// One warp chooses token t's experts from its logits' sums, which other CTAs wrote, and is done with
// it unless the choice is close.  score: [2 E] in shared memory: scores without the bias, to be multiplied by
// `scale`, then what orders.  PER: experts of a lane (E <= 32 PER), lane + 32 i.
template <int PER>
__device__ __forceinline__ void choose(const RouteArgs &a, int t, const Sums &sums, float *score, Choice &out)
{
    const int lane = threadIdx.x & 31;
    const bool soft = a.score == 0;
    float *order = score + a.E;
    float v[PER], bias[PER];             // logits, then scores without the bias
    float top = -INFINITY;               // largest logit
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        bias[i] = e < a.E && a.bias != nullptr ? __ldg(a.bias + e) : 0.0f;
        v[i] = e < a.E ? __ldcg(sums.logit(a, 0, t, e)) : -INFINITY;
    }
    // of the router's rows the parts' largest, as if in one row
    float w2 = 0.0f, x2 = lane < sums.parts ? __ldcg(sums.x2(a, lane, t)) : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        w2 = fmaxf(w2, lane + 32 * i < sums.parts * sums.tiles ? __ldcg(sums.largest_w2(a, lane + 32 * i)) : 0.0f);
    w2 *= (float)sums.parts;
    // many loads under way: a lane's experts of four parts
    const float *from = sums.logit(a, 0, t, lane);
#pragma unroll(PER <= 8 ? 4 : 1)
    for (int p = 1; p < sums.parts; ++p) {
        from += (int64_t)a.T * a.E;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i < a.E)
                v[i] += __ldcg(from + 32 * i);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        top = fmaxf(top, v[i]);          // skips NaN
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        x2 += __shfl_xor_sync(0xffffffffu, x2, d);
    }
    w2 = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(w2)));
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
    Choice c;
    c.top = top;
    c.scale = 1.0f;
    if (soft) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        c.scale = 1.0f / sum;
    }
    // How near two values are that may stand in either order: each logit is off by err.  A sigmoid's slope is
    // at most 1/4, and it is off by 2^-21 and one rounding besides.  Of a softmax's score the exponential and the
    // sum are off by a factor of exp(err) each, and by two units in the last place an exponential (four roundings),
    // PER + 5 additions, the quotient and the product.
    c.err = sums.slack * sqrtf(x2 + kLostSquares) * sqrtf(w2 + kLostSquares);
    c.tol = 2.0f * c.err;
    if (biased) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float s = v[i] * c.scale + bias[i];
            if (lane + 32 * i < a.E) {
                key[i] = s > -INFINITY ? key_of(s) : 0u;
                order[lane + 32 * i] = s;
            }
        }
        c.tol = soft ? 2.02f * c.scale * (expm1f(2.0f * c.err) + (PER + 16) * 0x1p-24f) : 0.5f * c.err + 0x1p-19f;
    }
    c.zero = x2 == 0.0f;
    c.close = false;
    c.chosen = 0;
    c.cut = -INFINITY;
    int mine = -1;                       // lane j keeps the j-th choice (k <= 16)
    float last = INFINITY;
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
        c.close = c.close || last - s <= nearness(a, c, s);   // no two infinities
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
        c.cut = s;
        ++c.chosen;
        if (lane == j)
            mine = e;
    }
    __syncwarp();
    c.close = c.close && c.chosen > 0;
    if (!c.close)
        finish(a, t, mine, c.chosen, score, c.scale);
    if (lane == 0)
        out = c;
}

__device__ __forceinline__ void choose_token(const RouteArgs &a, int t, const Sums &sums, float *score, Choice &out)
{
    if (a.E <= 64)
        choose<2>(a, t, sums, score, out);
    else if (a.E <= 256)
        choose<8>(a, t, sums, score, out);
    else
        choose<32>(a, t, sums, score, out);
}

// Shared memory of the decisions in 64 bits: [E] doubles and two lists of experts.
constexpr int kWideBytes = 16;   // an expert
// Rounding may move a softmax's sum by this much before its exponentials are taken in 64 bits as well: E logits
// instead of a few (96 tokens of 256 experts 0.3 ms).  Centred rows of 7168 with logits of a standard deviation below
// 20 stay under it.
constexpr float kSumSlack = 0x1p-8f;

// An integer of the same order; both zeros have one.
__device__ __forceinline__ int64_t key64(double v)
{
    const int64_t b = __double_as_longlong(v);
    return b < 0 ? INT64_MIN - b : b;
}

// Decides a close choice in 64 bits, with all of the CTA's warps.  Only experts whose fp32 value is near
// another's need it: twice the nearness away, fp32 can tell.  wide: [E] of shared memory and the lists behind it.
template <int WARPS>
__device__ __noinline__ void decide64(const RouteArgs &a, int t, const Choice &c, const float *score, double *wide)
{
    __shared__ int listed, candidates, best[32];
    __shared__ double part[WARPS];
    int *list = reinterpret_cast<int *>(wide + a.E), *candidate = list + a.E;
    const float *order = score + a.E;
    const int E = a.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool soft = a.score == 0, biased = a.bias != nullptr;
    const bool whole = soft && biased && c.err > kSumSlack;
    const float near = 2.0f * nearness(a, c, c.cut), least = c.cut < INFINITY ? c.cut - near : c.cut;
    if (threadIdx.x == 0)
        listed = candidates = 0;
    bool zero = false;   // a padded row: its logits are all 0
    if (c.zero) {
        uint32_t some = 0;
        const uint16_t *x = a.x + (int64_t)t * a.xs;
        for (int h = threadIdx.x * 8; h < a.H; h += WARPS * 32 * 8) {
            const uint4 r = __ldg(reinterpret_cast<const uint4 *>(x + h));
            some |= (r.x | r.y | r.z | r.w) & 0x7FFF7FFFu;
        }
        zero = !__syncthreads_or(some != 0);
    } else {
        __syncthreads();
    }
    // which may be among the chosen, and which of them are near another
    for (int e0 = warp * 32; e0 < E; e0 += WARPS * 32) {
        const int e = e0 + lane;
        const float f = e < E ? order[e] : NAN;
        bool sum = whole && e < E && score[e] >= 0.0f;
        unsigned todo = __ballot_sync(0xffffffffu, f >= least);
        while (todo) {
            const int who = __ffs(todo) - 1;
            todo &= todo - 1;
            const float mine = __shfl_sync(0xffffffffu, f, who), reach = 2.0f * nearness(a, c, mine);
            int others = 0;   // itself among them, unless it is infinite
#pragma unroll 8
            for (int i = lane; i < E; i += 32)
                others += fabsf(order[i] - mine) <= reach ? 1 : 0;
            others = __reduce_add_sync(0xffffffffu, others);
            if (lane == who)
                sum = sum || others > 1;
        }
        if (e < E)
            wide[e] = zero && sum ? 0.0 : (double)f;
        if (f >= least)
            candidate[atomicAdd(&candidates, 1)] = e;
        if (sum)
            list[atomicAdd(&listed, 1)] = e;
    }
    __syncthreads();
    // their logits: an expert by as many warps as there are for it, all by the same number
    const int n = zero ? 0 : listed, each = max(1, WARPS / max(n, 1)), at_once = WARPS / each;
    for (int i0 = 0; i0 < n; i0 += at_once) {
        const int i = i0 + warp / each;
        const bool has = warp / each < at_once && i < n;
        const double l = has ? part64(a, t, list[i], warp % each, each) : 0.0;
        if (lane == 0)
            part[warp] = l;
        if (each > 1)
            __syncthreads();   // one round
        if (has && warp % each == 0 && lane == 0) {
            double all = l;
            for (int w = 1; w < each; ++w)
                all += part[warp + w];
            wide[list[i]] = all;
        }
    }
    __syncthreads();
    // what orders those; where the logit is infinite, or the bias, fp32's value is exact
    double sum = 0.0;
    if (soft && biased) {
        for (int e = lane; e < E; e += 32)
            if (score[e] >= 0.0f)
                sum += whole && fabs(wide[e]) < INFINITY ? exp(wide[e] - (double)c.top) : (double)score[e];
        sum = warp_sum(sum);
        __syncthreads();
    }
    for (int i = threadIdx.x; i < listed; i += WARPS * 32) {
        const int e = list[i];
        const double l = wide[e];
        if (!(fabsf(order[e]) < INFINITY && fabs(l) < INFINITY))
            wide[e] = order[e];
        else if (biased)
            wide[e] = (soft ? exp(l - (double)c.top) / sum : 1.0 / (1.0 + exp(-l))) + (double)__ldg(a.bias + e);
    }
    __syncthreads();
    // a candidate's place: the larger ones, and of equal ones those before it (as integers of the same order)
    for (int i = threadIdx.x; i < candidates; i += WARPS * 32) {
        const int e = candidate[i];
        const int64_t mine = key64(wide[e]);
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < candidates; ++j) {
            const int other = candidate[j];
            const int64_t v = key64(wide[other]);
            place += v > mine || (v == mine && other < e) ? 1 : 0;
        }
        if (place < c.chosen)
            best[place] = e;
    }
    __syncthreads();
    if (warp == 0)
        finish(a, t, lane < c.chosen ? best[lane] : -1, c.chosen, score, c.scale);
}

// At most kTokens tokens.  grid: experts / EB; done: zero before and after.
template <int TB, int EB, bool BF>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a, const Sums sums, uint32_t *done)
{
    constexpr int kSums = TB * EB + EB + TB;   // products, then the squares of the router's rows and of the tokens'
    __shared__ float part[kWarps][kSums];
    extern __shared__ __align__(16) uint8_t smem[];
    float *scores = reinterpret_cast<float *>(smem);   // [T][2 E]
    __shared__ bool chooses;
    __shared__ Choice choice[kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e0 = blockIdx.x * EB;
    for (int t0 = 0; t0 < a.T; t0 += TB) {
        const bool first = t0 == 0, squares = blockIdx.x == 0;   // once for each row
        float acc[kSums] = {};
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
                for (int i = 0; i < TB; ++i) {
                    float eight = x[i][0] * w[0];   // by themselves: fewer roundings in a row
#pragma unroll
                    for (int c = 1; c < 8; ++c)
                        eight = fmaf(x[i][c], w[c], eight);
                    acc[i * EB + j] += eight;
                }
                if (first)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[TB * EB + j] = fmaf(w[c], w[c], acc[TB * EB + j]);
            }
            if (squares)
#pragma unroll
                for (int i = 0; i < TB; ++i)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        acc[TB * EB + EB + i] = fmaf(x[i][c], x[i][c], acc[TB * EB + EB + i]);
        }
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            if (i >= TB * EB && !(i < TB * EB + EB ? first : squares))
                continue;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            if (lane == 0)
                part[warp][i] = acc[i];
        }
        __syncthreads();
        if (threadIdx.x < kSums) {
            const int i = threadIdx.x;
            const float s = sum8([&](int w) { return part[w][i]; });
            const int t = t0 + i / EB, e = e0 + i % EB, tx = t0 + i - TB * EB - EB;
            if (i < TB * EB) {
                if (t < a.T && e < a.E)
                    __stcg(sums.logit(a, 0, t, e), s);
            } else if (i < TB * EB + EB) {
                if (first)
                    part[0][i] = s;
            } else if (squares && tx < a.T) {
                __stcg(sums.x2(a, 0, tx), s);
            }
        }
        if (first) {
            __syncthreads();
            if (threadIdx.x == 0) {
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < EB; ++j)
                    m = fmaxf(m, part[0][TB * EB + j]);   // skips NaN
                __stcg(sums.largest_w2(a, 0, blockIdx.x), m);
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        chooses = add_acq_rel(done, 1u) == gridDim.x - 1;   // then all CTAs' sums are visible
        if (chooses)
            *done = 0;
    }
    __syncthreads();
    if (!chooses)
        return;
    if (warp < a.T)
        choose_token(a, warp, sums, scores + warp * 2 * a.E, choice[warp]);
    __syncthreads();
    for (int t = 0; t < a.T; ++t)
        if (choice[t].close) {
            decide64<kWarps>(a, t, choice[t], scores + t * 2 * a.E, reinterpret_cast<double *>(scores + a.T * 2 * a.E));
            __syncthreads();
        }
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

__device__ __forceinline__ void add_pair(uint64_t &c, uint64_t a) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(c) : "l"(a)); }

__device__ __forceinline__ float sum_of(uint64_t v) { return __uint_as_float((uint32_t)v) + __uint_as_float((uint32_t)(v >> 32)); }

// += the squares of 32 values at p in shared memory
template <bool BF>
__device__ __forceinline__ void add_squares(uint64_t &c, uint32_t p)
{
#pragma unroll
    for (int i = 0; i < (BF ? 4 : 8); ++i) {
        const uint4 r = ld_shared_v4(p + i * 16);
        if (BF) {
            uint64_t v[4];
            widen4(make_uint2(r.x, r.y), *reinterpret_cast<uint64_t(*)[2]>(&v[0]));
            widen4(make_uint2(r.z, r.w), *reinterpret_cast<uint64_t(*)[2]>(&v[2]));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                fma_pair(c, v[j], v[j]);
        } else {
            fma_pair(c, pair_of(r.x, r.y), pair_of(r.x, r.y));
            fma_pair(c, pair_of(r.z, r.w), pair_of(r.z, r.w));
        }
    }
}

// grid: (parts of h, experts / 32, tokens / 32).  A warp computes the whole tile over every eighth run of
// 32 columns, a lane 4 tokens x 8 experts of it.  The 16 products of a run are added up by themselves
// before they join the other runs', which keeps a sum's roundings in a row few.
template <bool BF>
__global__ void __launch_bounds__(kThreads, 1) route_tile_kernel(const RouteArgs a, const Sums out)
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
    uint64_t total[4][8] = {};   // sums over the even and the odd columns
    uint64_t x2 = 0, w2 = 0;     // squares of token t0 + lane and expert e0 + lane
    for (int c = 0; c < chunks; ++c) {
        uint64_t acc[4][8] = {};
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
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                add_pair(total[i][j], acc[i][j]);
        // once for each row
        const uint32_t st = smem_u32(smem + c % kStages * S::kStage);
        if (blockIdx.y == 0)
            add_squares<true>(x2, st + lane * S::kXRow + warp * 64);
        if (blockIdx.z == 0)
            add_squares<BF>(w2, st + kTile * S::kXRow + lane * S::kWRow + warp * (BF ? 64 : 128));
    }
    cp_async_wait<0>();
    __syncthreads();
    __shared__ float squares[2][kWarps][32];
    squares[0][warp][lane] = sum_of(x2);
    squares[1][warp][lane] = sum_of(w2);
    float *sums = reinterpret_cast<float *>(smem);   // [warp][token][expert]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            sums[(warp * kTile + ti + 8 * i) * kTile + ei + 4 * j] = sum_of(total[i][j]);
    __syncthreads();
    if (warp < 2 && (warp == 0 ? blockIdx.y : blockIdx.z) == 0) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            s += squares[warp][w][lane];
        if (warp == 0) {
            if (t0 + lane < a.T)
                __stcg(out.x2(a, blockIdx.x, t0 + lane), s);
        } else {
            s = fmaxf(0.0f, s);   // a NaN is no expert's
            s = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(s)));
            if (lane == 0)
                __stcg(out.largest_w2(a, blockIdx.x, blockIdx.y), s);
        }
    }
    for (int i = threadIdx.x; i < kTile * kTile; i += kThreads) {
        const float s = sum8([&](int w) { return sums[w * kTile * kTile + i]; });
        const int t = t0 + i / kTile, e = e0 + i % kTile;
        if (t < a.T && e < a.E)
            __stcg(out.logit(a, blockIdx.x, t, e), s);
    }
}

// a CTA per token: one warp chooses, the others help where it is close
constexpr int kChooseWarps = 8;
__global__ void __launch_bounds__(kChooseWarps * 32) route_choose_kernel(const RouteArgs a, const Sums sums)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Choice choice;
    float *score = reinterpret_cast<float *>(smem);
    const int t = blockIdx.x;
    grid_wait();
    if (threadIdx.x < 32)
        choose_token(a, t, sums, score, choice);
    __syncthreads();
    if (choice.close)
        decide64<kChooseWarps>(a, t, choice, score, reinterpret_cast<double *>(score + 2 * a.E));
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
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(route_kernel<TB, EB, BF>), kMaxExperts * (kTokens * 8 + kWideBytes));
    if (e != cudaSuccess)
        return e;
    const int ctas = (a.E + EB - 1) / EB;
    // eight products, a thread's such sums, the shuffles and the warps
    const Sums sums{ws, 1, ctas, slack_of(8 + (a.H + 8 * kThreads - 1) / (8 * kThreads) + 5 + 3)};
    route_kernel<TB, EB, BF><<<ctas, kThreads, a.E * (a.T * 8 + kWideBytes), st>>>(a, sums, counter);
    return cudaGetLastError();
}

template <bool BF>
cudaError_t launch_tiles(const RouteArgs &a, float *ws, int num_sms, cudaStream_t st)
{
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(route_tile_kernel<BF>), TileSmem<BF>::kBytes);
    if (e != cudaSuccess)
        return e;
    const int parts = tile_parts(a, num_sms), tiles = (a.E + kTile - 1) / kTile;
    const int chunks = ((a.H + parts - 1) / parts + 8 + kChunk - 1) / kChunk;
    // the products of a run, the runs, both halves, the warps and the parts
    const Sums sums{ws, parts, tiles, slack_of(16 + chunks + 1 + 3 + parts)};
    route_tile_kernel<BF><<<dim3(parts, tiles, (a.T + kTile - 1) / kTile), kThreads, TileSmem<BF>::kBytes, st>>>(a, sums);
    return launch(route_choose_kernel, dim3(a.T), kChooseWarps * 32, (size_t)a.E * (8 + kWideBytes), 1, true, st, a, sums);
}

}  // namespace

int64_t route_ws_floats(const RouteArgs &a, int num_sms)
{
    if (a.T == 1)
        return sums_floats(a.T, a.E, 1, a.E);
    if (a.T <= kTokens)
        return sums_floats(a.T, a.E, 1, (a.E + 3) / 4);
    return sums_floats(a.T, a.E, tile_parts(a, num_sms), (a.E + kTile - 1) / kTile);
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

// moe.cu -- the experts' layer for a few tokens (moe_apply), in one launch.
//
//   out[t] = y[t] + sum_s w[t,s] W2[e] (act(G[e] x[t]) * (U[e] x[t])),   e = the expert of slot s
//
// Bound by HBM: every expert that has a token gives up its 3 H I bytes once, for a handful of
// tokens each.  So the weights are the MMA's M operand, 128 rows a tile, and the tokens its N:
// a CTA streams pairs of weight tiles, 32 KB per 128 of K, and their sums cost the tensor
// cores next to nothing.
//
// One persistent CTA per SM (a cooperative launch), 12 warps:
//   warp 0     TMA of the weights, for both products without a pause
//   warp 1     MMA issuer
//   warp 2     TMA of the tokens' codes (first product) and of the hidden values' (second)
//   warp 3     the grid's barriers
//   warps 4-11 promotion: a thread keeps one weight row of one of the two tiles, for all tokens;
//              between the products they form the hidden values, and at the end the rows of out
// The work of a product is a line of units (expert, tile pair, 128 of K), cut into equal
// shares, so that all SMs read the same number of bytes whatever the experts' number; a tile
// whose K is cut leaves a partial sum per share in the workspace ("planes"), added in their
// order.  Hidden values wait for the whole first product, at two barriers of the grid; the
// weights of the second keep coming meanwhile, as deep as the ring is (160 to 210 KB per SM,
// about 4 us of HBM).
//
// The first product takes every token as a column for every expert and keeps the columns of
// the tokens that chose it: no gather, and the columns are free.  The second one's columns are
// an expert's own hidden rows, in chunks of 8 GROUPS.  They enter as three e4m3 parts of one
// fp32 value under the scale of its 128 (h / s = c0 + c1 / 16 + c2 / 512): 448 is coded to 16,
// 16 times that remainder to 8, 32 times the next to 8, so the error is below
// 2^-14 of the largest of the 128 (or of 2^-100), where one e4m3 rounding would cost each value 2^-4.
//
// Experts of 7168 x 2048, bytes of the weights that are needed: one token of 8 experts 70.5 us (5.0
// TB/s; of 16 123 us, so what streams does at 6.7), 64 tokens that meet 64 experts 454 us (6.2), 96 that
// meet 128 879 us (6.4).  Up to 18 us are launch, plan, hidden values and rows of out.
#include <algorithm>

#include "activation.cuh"
#include "e4m3_encode.cuh"
#include "epilogue.cuh"
#include "few_rows.cuh"

namespace gemmar {
using namespace ptx;

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxSlots = 16;

// NT: token columns of the first product; GROUPS: groups of 8 tokens in a chunk of the second.
template <int NT_, int GROUPS_, int STAGES_, int BUFS_>
struct Cfg {
    static constexpr int NT = NT_, GROUPS = GROUPS_, kStages = STAGES_, kBufs = BUFS_;
    static constexpr int kXRows = NT > 24 * GROUPS ? NT : 24 * GROUPS;
    static constexpr int kStageBytes = 2 * kTileBytes + kXRows * 128;
    static constexpr int kCols = NT > (24 * GROUPS + 15) / 16 * 16 ? NT : (24 * GROUPS + 15) / 16 * 16;   // per tile
    static constexpr int kBufCols = kCols <= 32 ? 64 : kCols <= 64 ? 128 : 256;   // both tiles
    static constexpr int kTmemCols = kBufCols * kBufs;
    static constexpr int kSparse = NT >= 64 ? 32 : 16;   // tokens of an expert up to which its columns are picked
    static constexpr int kAcc = NT > 8 * GROUPS ? NT : 8 * GROUPS;
    static constexpr int kPairs = NT * kMaxSlots;
    static constexpr int kActive = kPairs < kMaxExperts ? kPairs : kMaxExperts;
    static constexpr int kChunks = kActive + kPairs / (8 * GROUPS);
    static constexpr int kOffScale = kStages * kStageBytes;            // [8 warps][2][kAcc] token scales
    static constexpr int kOffActive = kOffScale + 8 * 2 * kAcc * 4;    // u32 e | first pair << 10, and a last one
    static constexpr int kOffChunk = kOffActive + (kActive + 1) * 4;   // u32 e | first pair << 10 | pairs << 22
    static constexpr int kOffPair = kOffChunk + kChunks * 4;           // u32 token | active << 7 | chunk << 17
    static constexpr int kOffSlot = kOffPair + kPairs * 4;             // u16 pair of a token's slot
    static constexpr int kOffBar = (kOffSlot + kPairs * 2 + 7) / 8 * 8;
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 5;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmemBytes = kOffMisc + 96 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
    static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM budget");
    // the plan's scratch lies in the ring
    static_assert(kStages * kStageBytes >= kMaxExperts * (16 + 4 + 4) + kPairs * 2, "scratch of the plan");
};

using Few8 = Cfg<16, 1, 6, 4>;     // at most 8 tokens
using Few32 = Cfg<32, 2, 5, 4>;
using Few64 = Cfg<64, 3, 5, 2>;
using Few128 = Cfg<128, 5, 4, 2>;

__device__ __forceinline__ int expert_of(const MoeArgs &a, int slot)
{
    int e = __ldg(a.ids + slot);
    if (a.place != nullptr)
        e = e >= 0 && e < a.places ? __ldg(a.place + e) : -1;
    return e >= 0 && e < a.E ? e : -1;
}

// A product's units in a line: item (tile pair of an expert) by item, KB each, `per` to a CTA.
struct Line {
    int KB, per, first, end;   // first, end: this CTA's
    __device__ __forceinline__ Line(int items, int KB_) : KB(KB_)
    {
        const int units = items * KB;
        per = max((units + (int)gridDim.x - 1) / (int)gridDim.x, (KB + 7) / 8);   // no item in more than 9 shares
        first = min(units, (int)blockIdx.x * per);
        end = min(units, first + per);
    }
    // the shares an item's units are in, and the place of this CTA's among them
    __device__ __forceinline__ int planes(int item) const
    {
        const uint32_t u = (uint32_t)(item * KB);
        int n = 1;
        for (int left = (int)(u % (uint32_t)per) + KB - 1; left >= per; left -= per)
            ++n;
        return n;
    }
    __device__ __forceinline__ int plane(int item) const { return (int)blockIdx.x - item * KB / per; }
};

// A CTA's way along its share.  step() goes on to the next item's first unit; stay() to the next unit
// of this one, false where there is none.
struct Walk {
    const Line &l;
    int u, item, kb;
    __device__ __forceinline__ explicit Walk(const Line &line) : l(line), u(line.first), item(line.first / line.KB), kb(line.first - item * line.KB) {}
    __device__ __forceinline__ bool last_of_item() const { return kb + 1 == l.KB || u + 1 == l.end; }
    __device__ __forceinline__ bool stay()
    {
        if (last_of_item())
            return false;
        ++u;
        ++kb;
        return true;
    }
    __device__ __forceinline__ void step()
    {
        ++u;
        ++item;
        kb = 0;
    }
    __device__ __forceinline__ void advance()
    {
        if (!stay())
            step();
    }
};

// Who goes where, computed by every CTA for itself from the ids: experts that have tokens in
// ascending order, each one's tokens in ascending order ("pairs"; a token that names an expert
// twice is one pair, with both weights).
template <class C>
__device__ void make_plan(const MoeArgs &a, uint8_t *smem, int &active, int &chunks, int &pairs)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem);             // [E][4] tokens of an expert
    uint32_t *place = mask + kMaxExperts * 4, *base = place + kMaxExperts;   // [E] first pair | active << 12; first chunk
    int16_t *expert = reinterpret_cast<int16_t *>(base + kMaxExperts);       // [T k] of a slot
    uint32_t *act = reinterpret_cast<uint32_t *>(smem + C::kOffActive);
    uint32_t *chk = reinterpret_cast<uint32_t *>(smem + C::kOffChunk);
    uint32_t *pair = reinterpret_cast<uint32_t *>(smem + C::kOffPair);
    uint16_t *slot = reinterpret_cast<uint16_t *>(smem + C::kOffSlot);
    uint32_t *sums = reinterpret_cast<uint32_t *>(smem + C::kOffScale);      // [12][2] of the scan
    const int slots = a.T * a.k;
    for (int i = tid; i < a.E * 4; i += kThreads)
        mask[i] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += kThreads) {
        const int e = expert_of(a, i), t = i / a.k;
        expert[i] = (int16_t)e;
        if (e >= 0)
            atomicOr(mask + e * 4 + (t >> 5), 1u << (t & 31));
    }
    __syncthreads();
    // three experts in a row to a thread; sums of pairs, and of experts with tokens and chunks
    constexpr int PER = (kMaxExperts + kThreads - 1) / kThreads, CH = 8 * C::GROUPS;
    uint32_t n[PER], mine0 = 0, mine1 = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid * PER + j;
        n[j] = 0;
        if (e < a.E) {
            const uint4 m = *reinterpret_cast<const uint4 *>(mask + e * 4);
            n[j] = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
        }
        mine0 += n[j];
        mine1 += (n[j] > 0 ? 1u : 0u) | ((n[j] + CH - 1) / CH) << 16;
    }
    uint32_t s0 = mine0, s1 = mine1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o0 = __shfl_up_sync(0xffffffffu, s0, d), o1 = __shfl_up_sync(0xffffffffu, s1, d);
        if (lane >= d) {
            s0 += o0;
            s1 += o1;
        }
    }
    if (lane == 31) {
        sums[warp * 2] = s0;
        sums[warp * 2 + 1] = s1;
    }
    __syncthreads();
    uint32_t all0 = 0, all1 = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) {
            s0 += all0;
            s1 += all1;
        }
        all0 += sums[w * 2];
        all1 += sums[w * 2 + 1];
    }
    s0 -= mine0;
    s1 -= mine1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid * PER + j;
        if (n[j] == 0)
            continue;
        const uint32_t ia = s1 & 0xFFFFu, ic = s1 >> 16;
        act[ia] = (uint32_t)e | s0 << 10;
        place[e] = s0 | ia << 12;
        base[e] = ic;
        for (uint32_t c = 0; c * CH < n[j]; ++c)
            chk[ic + c] = (uint32_t)e | (s0 + c * CH) << 10 | min(n[j] - c * CH, (uint32_t)CH) << 22;
        s0 += n[j];
        s1 += 1u | ((n[j] + CH - 1) / CH) << 16;
    }
    pairs = (int)all0;
    active = (int)(all1 & 0xFFFFu);
    chunks = (int)(all1 >> 16);
    if (tid == 0)
        act[active] = all0 << 10;
    __syncthreads();
    for (int i = tid; i < slots; i += kThreads) {
        const int e = expert[i], t = i / a.k;
        bool first = e >= 0;
        for (int j = t * a.k; j < i; ++j)
            first = first && expert[j] != e;
        uint32_t at = 0xFFFFu;
        if (first) {
            uint32_t rank = __popc(mask[e * 4 + (t >> 5)] & ((1u << (t & 31)) - 1));
            for (int w = 0; w < (t >> 5); ++w)
                rank += __popc(mask[e * 4 + w]);
            at = (place[e] & 0xFFFu) + rank;
            pair[at] = (uint32_t)t | (place[e] >> 12) << 7 | (base[e] + rank / CH) << 17;
        }
        slot[i] = (uint16_t)at;
    }
    fence_async_shared();   // the ring's first copies come after this scratch
}

__device__ __forceinline__ float max4(const float4 &v) { return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))); }

__device__ __forceinline__ float4 ld4(const float *p) { return __ldcg(reinterpret_cast<const float4 *>(p)); }

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b)
{
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// four codes of v, and what is left of it
__device__ __forceinline__ uint32_t code4(float (&v)[4])
{
    const uint32_t lo = e4m3x2_from_f32(v[0], v[1]), hi = e4m3x2_from_f32(v[2], v[3]);
    const float2 a = f32x2_from_e4m3x2((uint16_t)lo), b = f32x2_from_e4m3x2((uint16_t)hi);
    v[0] -= a.x;
    v[1] -= a.y;
    v[2] -= b.x;
    v[3] -= b.y;
    return lo | hi << 16;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ MoeParams prm)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *empty = full + C::kStages;
    uint64_t *tfull = empty + C::kStages;
    uint64_t *tempty = tfull + C::kBufs;
    uint64_t *final_bar = tempty + C::kBufs;
    uint64_t *epi_bar = final_bar + 1;     // the promotion warps have written what the grid waits for
    uint64_t *grid_bar = epi_bar + 1;      // [3], once each: so have those of all CTAs
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

    const MoeArgs &a = prm.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full + s, 2);   // weights and tokens
            mbar_init(empty + s, 1);
        }
        for (int b = 0; b < C::kBufs; ++b) {
            mbar_init(tfull + b, 1);
            mbar_init(tempty + b, 8);
        }
        mbar_init(final_bar, 1);
        mbar_init(epi_bar, 8);
        for (int b = 0; b < 3; ++b)
            mbar_init(grid_bar + b, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&prm.tmX);
        prefetch_tmap(&prm.tmW13);
        prefetch_tmap(&prm.tmW2);
        prefetch_tmap(&prm.tmParts);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kTmemCols);
        tmem_relinquish();
    }
    int active, chunks, pairs;
    make_plan<C>(a, smem, active, chunks, pairs);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t *act = reinterpret_cast<const uint32_t *>(smem + C::kOffActive);
    const uint32_t *chk = reinterpret_cast<const uint32_t *>(smem + C::kOffChunk);
    const uint32_t *pair = reinterpret_cast<const uint32_t *>(smem + C::kOffPair);
    const uint16_t *slot = reinterpret_cast<const uint16_t *>(smem + C::kOffSlot);

    const int IB = a.I / 128, HB = a.H / 128, J2 = (HB + 1) / 2;
    const Line l1(active * IB, HB);        // items (expert, 128 hidden values: their gate and up rows)
    const Line l2(J2 * chunks, IB);        // items (256 columns of out, chunk)
    const int n1 = (a.T + 15) / 16 * 16;   // columns of the first product
    const int64_t rows3 = (int64_t)a.T * a.k + 8;   // hidden rows of one part

    if (warp < 4) {
        setmaxnreg_dec<kRegsLow>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ weights: they pass through L2 without
            // pushing out what the launch comes back to, its later steps' code among it
            const uint64_t once = l2_evict_first();
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto load = [&](const CUtensorMap *tm, int row0, int row1, int kb) {
                ok = mbar_wait(empty + stage, ph ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_PRODUCER_EMPTY);
                if (!ok)
                    return;
                uint8_t *w = smem + stage * C::kStageBytes;
                mbar_arrive_expect_tx(full + stage, 2 * kTileBytes);
                tma_load_2d(w, tm, full + stage, kb * 128, row0, once);
                tma_load_2d(w + kTileBytes, tm, full + stage, kb * 128, row1, once);
                if (++stage == C::kStages) {
                    stage = 0;
                    ph ^= 1;
                }
            };
            for (Walk w(l1); w.u < l1.end && ok; w.step()) {
                const int ia = w.item / IB, r = (int)(act[ia] & 1023) * 2 * a.I + (w.item - ia * IB) * 128;
                const int r1 = r + a.I;
                for (bool same = true; same && ok; same = w.stay())
                    load(&prm.tmW13, r, r1, w.kb);
            }
            for (Walk w(l2); w.u < l2.end && ok; w.step()) {
                // the second tile of an odd last pair holds other rows, or none: nobody reads its sums
                const int j = w.item / chunks, r = (int)(chk[w.item - j * chunks] & 1023) * a.H + j * 256;
                for (bool same = true; same && ok; same = w.stay())
                    load(&prm.tmW2, r, r + 128, w.kb);
            }
        } else if (warp == 1 && lane == 0) {
            // ------------------------------------------------ MMA issuer
            int stage = 0, buf = 0;
            uint32_t ph = 0, tph = 0;
            bool ok = true;
            auto issue = [&](int n) {
                ok = mbar_wait(tempty + buf, tph ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_TMEM_EMPTY) &&
                     mbar_wait(full + stage, ph, abort_flag, prm.status, prm.timeout_ns, SITE_MMA_FULL);
                if (!ok)
                    return;
                tc_fence_after();
                const uint32_t idesc = idesc_f8_e4m3(128, n);
                const uint32_t w = smem_u32(smem + stage * C::kStageBytes);
                const uint64_t xd = desc_kmajor_sw128(w + 2 * kTileBytes);
#pragma unroll
                for (int tile = 0; tile < 2; ++tile) {
                    const uint64_t wd = desc_kmajor_sw128(w + tile * kTileBytes);
                    const uint32_t d = tmem_base + buf * C::kBufCols + tile * (C::kBufCols / 2);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8(d, wd + 2 * k, xd + 2 * k, idesc, k > 0 ? 1u : 0u);
                }
                tc_commit(empty + stage);
                tc_commit(tfull + buf);
                if (++stage == C::kStages) {
                    stage = 0;
                    ph ^= 1;
                }
                if (++buf == C::kBufs) {
                    buf = 0;
                    tph ^= 1;
                }
            };
            for (int u = l1.first; u < l1.end && ok; ++u)
                issue(n1);
            for (Walk w(l2); w.u < l2.end && ok; w.step()) {
                const int groups = (int)((chk[w.item % chunks] >> 22) + 7) / 8;
                const int n2 = (24 * groups + 15) / 16 * 16;   // columns past the parts hold anything, and are not read
                for (bool same = true; same && ok; same = w.stay())
                    issue(n2);
            }
            tc_commit(final_bar);
            wait_teardown(final_bar, prm.status, prm.timeout_ns);
        } else if (warp == 2 && lane == 0) {
            // ------------------------------------------------ tokens
            int stage = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto next = [&] {
                if (++stage == C::kStages) {
                    stage = 0;
                    ph ^= 1;
                }
            };
            for (Walk w(l1); w.u < l1.end && ok; w.advance(), next()) {
                ok = mbar_wait(empty + stage, ph ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_PRODUCER_EMPTY);
                if (ok) {
                    mbar_arrive_expect_tx(full + stage, n1 * 128);
                    tma_load_2d(smem + stage * C::kStageBytes + 2 * kTileBytes, &prm.tmX, full + stage, w.kb * 128, 0);
                }
            }
            // the hidden values of all CTAs, written through the generic proxy
            ok = ok && mbar_wait(grid_bar + 1, 0, abort_flag, prm.status, prm.timeout_ns, SITE_GRID);
            fence_async_all();
            for (Walk w(l2); w.u < l2.end && ok; w.step()) {
                const uint32_t c = chk[w.item % chunks];
                const int groups = (int)((c >> 22) + 7) / 8, first = (int)(c >> 10 & 0xFFF);
                for (bool same = true; same && ok; same = w.stay(), next()) {
                    ok = mbar_wait(empty + stage, ph ^ 1, abort_flag, prm.status, prm.timeout_ns, SITE_PRODUCER_EMPTY);
                    if (!ok)
                        break;
                    uint8_t *x = smem + stage * C::kStageBytes + 2 * kTileBytes;
                    mbar_arrive_expect_tx(full + stage, 3 * groups * 1024);
                    for (int part = 0; part < 3; ++part)
                        for (int i = 0; i < groups; ++i)
                            tma_load_2d(x + (part * groups + i) * 1024, &prm.tmParts, full + stage, w.kb * 128,
                                        (int)(part * rows3) + first + i * 8);
                }
            }
        } else if (warp == 3 && lane == 0) {
            // ------------------------------------------------ the grid's barriers
            bool ok = true;
            for (int b = 0; b < 3 && ok; ++b) {
                ok = mbar_wait(epi_bar, b & 1, abort_flag, prm.status, prm.timeout_ns, SITE_GRID);
                if (!ok)
                    break;
                red_release_add(prm.counters, 1u);   // releases what the promotion warps wrote before they arrived
                const uint32_t want = (uint32_t)(b + 1) * gridDim.x;
                const uint64_t t0 = globaltimer();
                while (ld_acquire(prm.counters) < want) {
                    if (*abort_flag || globaltimer() - t0 > prm.timeout_ns) {
                        if (!*abort_flag) {
                            *abort_flag = 1;
                            report(prm.status, kErrTimeout, SITE_GRID);
                        }
                        ok = false;
                        break;
                    }
                }
                if (ok)
                    mbar_arrive(grid_bar + b);
            }
            // the last CTA that is done with the barriers, whether it passed them or gave up, leaves the counters as the
            // next call expects them
            if (add_acq_rel(prm.counters + 1, 1u) == gridDim.x - 1) {
                prm.counters[0] = 0;
                prm.counters[1] = 0;
            }
        }
    } else {
        setmaxnreg_inc<kRegsHigh>();
        // ------------------------------------------------ promotion
        const int q = warp & 3, h = (warp - 4) >> 2;   // lane quarter, tile of the pair
        const int row = q * 32 + lane;
        float *ts = reinterpret_cast<float *>(smem + C::kOffScale) + (warp - 4) * 2 * C::kAcc;
        const uint32_t taddr0 = tmem_base + ((uint32_t)(q * 32) << 16) + h * (C::kBufCols / 2);
        int buf = 0;
        uint32_t tph = 0;
        bool ok = true;
        float acc[C::kAcc];
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tempty + buf);
            if (++buf == C::kBufs) {
                buf = 0;
                tph ^= 1;
            }
        };
        auto everyone = [&](int b) {   // the b-th barrier of the grid
            __syncwarp();
            if (lane == 0)
                mbar_arrive(epi_bar);
            ok = mbar_wait(grid_bar + b, 0, abort_flag, prm.status, prm.timeout_ns, SITE_GRID);
        };
        // Scales of the tokens, a unit ahead: column lane + 32 i at from + at[i] + kb, the weights' at
        // from_sw + kb.  The product of both goes to the warp's own shared memory, from where each
        // thread reads all of them.
        constexpr int PER = (C::kAcc + 31) / 32;
        const float *from = a.sx, *from_sw = nullptr;
        int at[PER];   // -1: no token at this column
        float next_ts[PER], next_sw = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            at[i] = -1;
            next_ts[i] = 0.0f;
        }
        auto fetch = [&](int kb) {
            next_sw = __ldg(from_sw + kb);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                next_ts[i] = at[i] >= 0 ? ld_after_f32(from + at[i] + kb) : 0.0f;
        };
        auto stage_scales = [&](int u) {
            float *now = ts + (u & 1) * C::kAcc;   // read last two units back
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 32 * i < C::kAcc)
                    now[lane + 32 * i] = next_sw * next_ts[i];
            return now;
        };

        // -------- first product.  Of an expert with few tokens only their columns are read, the
        // j-th token's sum in acc[j]; of one with more all, a token's in acc[token].  Where there
        // are 8 tokens at most, all.
        constexpr bool kAll = C::NT <= 16;
        constexpr int kDense = kAll ? 8 : C::NT;
        constexpr int kPick = kAll ? 8 : C::kSparse;
        int first = 0, n = 0;
        bool sparse = false;
        uint32_t column[kPick];
        auto point1 = [&](int item) {
            const int ia = item / IB;
            const uint32_t e = act[ia];
            from_sw = a.s13 + ((int64_t)(e & 1023) * 2 * IB + h * IB + (item - ia * IB)) * HB;
            const int begin = (int)(e >> 10), count = (int)(act[ia + 1] >> 10) - begin;
            if (!kAll && count <= C::kSparse) {
                at[0] = lane < count ? (int)(pair[begin + lane] & 127) * HB : -1;
#pragma unroll
                for (int i = 1; i < PER; ++i)
                    at[i] = -1;
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    at[i] = lane + 32 * i < a.T ? (lane + 32 * i) * HB : -1;
            }
        };
        auto enter1 = [&](int item) {
            const int ia = item / IB;
            first = (int)(act[ia] >> 10);
            n = (int)(act[ia + 1] >> 10) - first;
            if (!kAll) {
                sparse = n <= C::kSparse;
                const int list = lane < n ? (int)(pair[first + lane] & 127) : 0;
#pragma unroll
                for (int j = 0; j < kPick; ++j)   // past the last token: a column nobody asked for, unused
                    column[j] = taddr0 + __shfl_sync(0xffffffffu, list, j);
            }
#pragma unroll
            for (int j = 0; j < C::kAcc; ++j)
                acc[j] = 0.0f;
        };
        Walk w1(l1);
        if (w1.u < l1.end) {
            point1(w1.item);
            fetch(w1.kb);
        }
        for (bool fresh = true; w1.u < l1.end; w1.advance()) {
            if (fresh)
                enter1(w1.item);
            const float *now = stage_scales(w1.u);
            const bool last = fresh = w1.last_of_item();
            if (!last) {
                fetch(w1.kb + 1);
            } else if (w1.u + 1 < l1.end) {
                point1(w1.item + 1);
                fetch(0);
            }
            ok = mbar_wait(tfull + buf, tph, abort_flag, prm.status, prm.timeout_ns, SITE_EPI_TMEM_FULL);
            if (!ok)
                break;
            __syncwarp();
            tc_fence_after();
            if (sparse) {
                uint32_t r[kPick];
#pragma unroll
                for (int c = 0; c < kPick; c += 8)
                    if (c < n) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            tmem_ld_x1(column[c + j] + buf * C::kBufCols, r[c + j]);
                    }
#pragma unroll
                for (int c = 0; c < kPick; c += 8)
                    if (c < n) {
                        uint32_t(&v)[8] = *reinterpret_cast<uint32_t(*)[8]>(&r[c]);
                        tmem_wait_ld(v);
                        promote8(acc + c, v, now + c);
                    }
            } else if (kAll) {
                uint32_t r[8];
                tmem_ld_x8(taddr0 + buf * C::kBufCols, r);
                tmem_wait_ld(r);
                promote8(acc, r, now);
            } else {
#pragma unroll
                for (int c = 0; c < kDense; c += 16)
                    if (c < a.T) {
                        uint32_t r[16];
                        tmem_ld_x16(taddr0 + buf * C::kBufCols + c, r);
                        tmem_wait_ld(r);
                        promote8(acc + c, *reinterpret_cast<uint32_t(*)[8]>(&r[0]), now + c);
                        promote8(acc + c + 8, *reinterpret_cast<uint32_t(*)[8]>(&r[8]), now + c + 8);
                    }
            }
            release();
            if (last) {
                const int ia = w1.item / IB, jb = w1.item - ia * IB;
                float *to = prm.pieces + ((int64_t)l1.plane(w1.item) * pairs + first) * (2 * a.I) + h * a.I + jb * 128 + row;
                if (sparse) {
#pragma unroll
                    for (int j = 0; j < kPick; ++j)
                        if (j < n)
                            __stcg(to + (int64_t)j * 2 * a.I, acc[j]);
                } else {
                    uint32_t mask[(kDense + 31) / 32] = {};
                    for (int i = 0; i < n; i += 32) {
                        const uint32_t t = i + lane < n ? pair[first + i + lane] & 127 : 0xFFFFu;
#pragma unroll
                        for (int w = 0; w < (kDense + 31) / 32; ++w)
                            mask[w] |= __reduce_or_sync(0xffffffffu, t >> 5 == (uint32_t)w ? 1u << (t & 31) : 0u);
                    }
#pragma unroll
                    for (int j = 0; j < kDense; ++j)
                        if (mask[j >> 5] >> (j & 31) & 1) {
                            __stcg(to, acc[j]);
                            to += 2 * a.I;
                        }
                }
            }
        }
        // -------- hidden values: a warp takes 128 of a pair at a time
        if (ok)
            everyone(0);
        if (ok) {
            const int groups = pairs * IB;
            for (int i = (warp - 4) * gridDim.x + blockIdx.x; i < groups; i += gridDim.x * 8) {
                const int p = i / IB, jb = i % IB;
                const uint32_t info = pair[p];
                const int t = (int)(info & 127), ia = (int)(info >> 7 & 1023), e = (int)(act[ia] & 1023);
                const int planes = l1.planes(ia * IB + jb);
                const float *from = prm.pieces + (int64_t)p * 2 * a.I + jb * 128 + lane * 4;
                const int64_t plane = (int64_t)pairs * 2 * a.I;
                float4 zg = ld4(from), zu = ld4(from + a.I);
                if (planes > 1) {
                    const float4 g1 = ld4(from + plane), u1 = ld4(from + plane + a.I);
                    zg = add4(zg, g1);
                    zu = add4(zu, u1);
                }
                for (int pl = 2; pl < planes; ++pl) {
                    zg = add4(zg, ld4(from + pl * plane));
                    zu = add4(zu, ld4(from + pl * plane + a.I));
                }
                float w = 0.0f;
                if (lane < a.k) {
                    const float v = __ldg(a.weights + t * a.k + lane);
                    w = expert_of(a, t * a.k + lane) == e ? v : 0.0f;
                }
#pragma unroll
                for (int d = kMaxSlots / 2; d > 0; d >>= 1)
                    w += __shfl_xor_sync(0xffffffffu, w, d);
                w = __shfl_sync(0xffffffffu, w, 0);
                float4 hv;
                with_act(a.act, [&](auto kind) {
                    constexpr int ACT = decltype(kind)::value;
                    hv = make_float4(act_value<ACT>(zg.x) * zu.x * w, act_value<ACT>(zg.y) * zu.y * w,
                                     act_value<ACT>(zg.z) * zu.z * w, act_value<ACT>(zg.w) * zu.w * w);
                });
                // not below 2^-100, so that a scale's reciprocal stays in range
                const float m = fmaxf(0x1p-100f, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(max4(hv)))));
                // s times the parts is h to 2^-21, whichever way the two quotients round; no s comes near
                // 2^126, from where __fdividef gives 0
                const float s = m * (1.0f / 448.0f), inv = __fdividef(1.0f, s);
                float v[4] = {hv.x * inv, hv.y * inv, hv.z * inv, hv.w * inv};
                uint8_t *o = prm.parts + (int64_t)p * a.I + jb * 128 + lane * 4;
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    *reinterpret_cast<uint32_t *>(o + part * rows3 * a.I) = code4(v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] *= part == 0 ? 16.0f : 32.0f;
                }
                if (lane == 0)
                    __stcg(prm.hidden_scale + (int64_t)p * IB + jb, s);
            }
            fence_async_all();   // other SMs read the parts through their async proxy
            everyone(1);
        }
        // -------- second product
        auto point2 = [&](int item) {
            const int j = item / chunks;
            const uint32_t c = chk[item - j * chunks];
            from_sw = a.s2 + ((int64_t)(c & 1023) * HB + min(j * 2 + h, HB - 1)) * IB;
            const int begin = (int)(c >> 10 & 0xFFF), count = (int)(c >> 22);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                at[i] = lane + 32 * i < count ? (begin + lane + 32 * i) * IB : -1;
        };
        from = prm.hidden_scale;
        __syncwarp();
        Walk w2(l2);
        if (ok && w2.u < l2.end) {
            point2(w2.item);
            fetch(w2.kb);
        }
        int groups = 0;
        for (bool fresh = true; w2.u < l2.end && ok; w2.advance()) {
            if (fresh) {
                const uint32_t c = chk[w2.item % chunks];
                first = (int)(c >> 10 & 0xFFF);
                n = (int)(c >> 22);
                groups = (n + 7) / 8;
#pragma unroll
                for (int j = 0; j < 8 * C::GROUPS; ++j)
                    acc[j] = 0.0f;
            }
            const float *now = stage_scales(w2.u);
            const bool last = fresh = w2.last_of_item();
            if (!last) {
                fetch(w2.kb + 1);
            } else if (w2.u + 1 < l2.end) {
                point2(w2.item + 1);
                fetch(0);
            }
            ok = mbar_wait(tfull + buf, tph, abort_flag, prm.status, prm.timeout_ns, SITE_EPI_TMEM_FULL);
            if (!ok)
                break;
            __syncwarp();
            tc_fence_after();
            const uint32_t taddr = taddr0 + buf * C::kBufCols;
#pragma unroll
            for (int i = 0; i < C::GROUPS; ++i)
                if (i < groups) {
                    uint32_t r0[8], r1[8], r2[8], d[8];
                    tmem_ld_x8(taddr + i * 8, r0);
                    tmem_ld_x8(taddr + (groups + i) * 8, r1);
                    tmem_ld_x8(taddr + (2 * groups + i) * 8, r2);
                    tmem_wait_ld(r0, r1);
                    tmem_wait_ld(r2);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        d[j] = __float_as_uint(fmaf(__uint_as_float(r2[j]), 0x1p-9f, fmaf(__uint_as_float(r1[j]), 0x1p-4f, __uint_as_float(r0[j]))));
                    promote8(acc + i * 8, d, now + i * 8);
                }
            release();
            const int block = w2.item / chunks * 2 + h;
            if (last && block < HB) {
                float *to = prm.pieces + ((int64_t)l2.plane(w2.item) * pairs + first) * a.H + block * 128 + row;
#pragma unroll
                for (int j = 0; j < 8 * C::GROUPS; ++j)
                    if (j < n)
                        __stcg(to + (int64_t)j * a.H, acc[j]);
            }
        }
        // rows of out: a lane takes four columns and every fourth of the token's slots, eight lanes in a
        // row 32 columns.  A tight loop: its code is fetched while the weights fill the memory's queues
        const uint32_t octs = a.H / 32, oct0 = (warp - 4) * gridDim.x + blockIdx.x;
        const int oct_lane = lane & 7, share = lane >> 3;
        if (a.y != nullptr && oct0 < a.T * octs && share == 0)
            prefetch_l2(a.y + oct0 / octs * a.ys + (oct0 % octs * 32 + oct_lane * 4));
        if (ok)
            everyone(2);
        if (ok) {
            const int64_t plane = (int64_t)pairs * a.H;
#pragma unroll 1
            for (uint32_t i = oct0; i < a.T * octs; i += gridDim.x * 8) {
                const int t = (int)(i / octs), col = (int)(i - t * octs) * 32 + oct_lane * 4;
                float4 sum = make_float4(0, 0, 0, 0);
                if (share == 0 && a.y != nullptr) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(a.y + t * a.ys + col);
                    sum = make_float4(bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y));
                }
#pragma unroll 1
                for (int s = share; s < a.k; s += 4) {
                    const uint32_t p = slot[t * a.k + s];
                    if (p == 0xFFFFu)
                        continue;
                    const float *from = prm.pieces + (int64_t)p * a.H + col;
#pragma unroll 1
                    for (int planes = l2.planes(col / 256 * chunks + (int)(pair[p] >> 17)); planes > 0; --planes, from += plane)
                        sum = add4(sum, ld4(from));
                }
                __syncwarp();
#pragma unroll
                for (int d = 8; d < 32; d *= 2)
                    sum = add4(sum, make_float4(__shfl_xor_sync(0xffffffffu, sum.x, d), __shfl_xor_sync(0xffffffffu, sum.y, d),
                                                __shfl_xor_sync(0xffffffffu, sum.z, d), __shfl_xor_sync(0xffffffffu, sum.w, d)));
                if (share == 0)
                    *reinterpret_cast<uint2 *>(a.out + t * a.os + col) =
                        make_uint2(bf16x2_from_f32(sum.x, sum.y), bf16x2_from_f32(sum.z, sum.w));
            }
        }
    }

    __syncwarp();
    if (*abort_flag) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < kAbortGraceNs) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem_base, C::kTmemCols);
}

template <class C>
cudaError_t launch_typed(const MoeParams &p, int num_sms, cudaStream_t st)
{
    const void *kernel = reinterpret_cast<const void *>(moe_kernel<C>);
    static std::atomic<bool> split_ok{false};
    if (!few_rows_split_ok(split_ok, kernel))
        return cudaErrorInvalidConfiguration;
    const cudaError_t e = ensure_dynamic_smem(kernel, C::kSmemBytes);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // its CTAs wait for one another
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3(num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_kernel<C>, p);
}

}  // namespace

// Sums of both products: an item's units lie in at most 9 shares and at most sms / items + 2, and
// there are at least as many experts as a token's slots name, so the planes of all pairs are at
// most T (sms / tile pairs + 2 k) rows, and 9 T k.
MoeLayout moe_layout(const MoeArgs &a, int num_sms)
{
    MoeLayout l;
    const int64_t IB = a.I / 128, J2 = (a.H / 128 + 1) / 2, slots = (int64_t)a.T * a.k;
    const int64_t rows1 = std::min<int64_t>(9 * a.k, num_sms / IB + 1 + 2 * a.k), rows2 = std::min<int64_t>(9 * a.k, num_sms / J2 + 1 + 2 * a.k);
    l.hidden_scale = a.T * std::max(rows1 * 2 * a.I, rows2 * a.H);
    l.parts = l.hidden_scale + (slots * IB + 3) / 4 * 4;
    l.part_rows = 3 * (slots + 8);
    l.floats = l.parts + l.part_rows * a.I / 4;
    return l;
}

int moe_columns(int T) { return (T + 15) / 16 * 16; }

cudaError_t launch_moe(const MoeParams &p, int num_sms, cudaStream_t st)
{
    if (p.a.T <= 8)
        return launch_typed<Few8>(p, num_sms, st);
    if (p.a.T <= 32)
        return launch_typed<Few32>(p, num_sms, st);
    if (p.a.T <= 64)
        return launch_typed<Few64>(p, num_sms, st);
    return launch_typed<Few128>(p, num_sms, st);
}

}  // namespace gemmar

// gemmar.cu -- the C ABI of libgemmar (declared in include/gemmar.h): context
// and workspace, argument and shape validation, TMA tensor maps, launches,
// the device status word and the closed-form self-test.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <set>
#include <utility>
#include <vector>

#include "gemmar.h"
#include "kernels.h"
#include "spans.h"

#define GEMMAR_API extern "C" __attribute__((visibility("default")))

using namespace gemmar;

struct gemmar_ctx {
    int device = -1;
    int num_sms = 0;
    int64_t max_M = 0, N = 0, K = 0;
    int max_P = 0;
    uint32_t flags = 0;
    uint64_t timeout_ns = 0;
    float *W = nullptr;               // fp32 partials, max_P * (max_M + 128 * max_P) * N (tile-blocked), or 256 * max_M
    int64_t W_floats = 0;
    uint32_t *band_done = nullptr;    // kMaxBands retire counters, then as many claim counters
    ptx::DevStatus *status = nullptr;
    uint8_t *sfa = nullptr;           // mx repack images of A scales
    int64_t sfa_bytes = 0;
    uint8_t *sfb = nullptr;           // mx repack images of B scales
    int64_t sfb_bytes = 0;
    uint8_t *wire_q = nullptr;        // fp8-wire codes, max_M * N
    float *wire_s = nullptr;          // fp8-wire row scales, max_M
    uint32_t *counters = nullptr;     // kCounters arrival counters, zero between calls
    int disabled = 0;
    int64_t total_bytes = 0;
    // the last fused band-path call, for gemmar_overlap_stats
    int ov_bands = 0;                 // bands whose claim counters it used (0: no in-kernel reduce)
    int64_t ov_bpb = 0;               // 32 x 32 blocks per band
    int64_t ov_total = 0;             // blocks of the call
    // phase timing: one set of GEMMAR_NUM_PHASES + 1 events per recorded call
    int timing = 0;
    std::vector<cudaEvent_t> events;
    int recorded = 0;
};

namespace gemmar {

cudaError_t ensure_dynamic_smem(const void *kernel, int bytes)
{
    static std::mutex mu;
    static std::set<std::pair<const void *, int>> done;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    std::lock_guard<std::mutex> lock(mu);
    if (done.count({kernel, dev}))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.insert({kernel, dev});
    return e;
}

}  // namespace gemmar

namespace {

constexpr int kMaxTimedCalls = 65536;
constexpr int kCounters = 64;      // moe_route's, and moe_apply's in a cache line of their own
constexpr int kMoeCounters = 32;
constexpr int kEventsPerCall = GEMMAR_NUM_PHASES + 1;

// Event marking the start of phase `ph` (ph == GEMMAR_NUM_PHASES: the end) of
// the current recorded call, or nullptr when timing is off or the record is full.
cudaEvent_t phase_event(gemmar_ctx *ctx, int ph)
{
    if (!ctx->timing || ctx->recorded >= kMaxTimedCalls)
        return nullptr;
    const size_t idx = (size_t)ctx->recorded * kEventsPerCall + ph;
    while (ctx->events.size() <= idx) {
        cudaEvent_t e;
        if (cudaEventCreate(&e) != cudaSuccess)
            return nullptr;
        ctx->events.push_back(e);
    }
    return ctx->events[idx];
}

void mark(gemmar_ctx *ctx, int ph, cudaStream_t st)
{
    cudaEvent_t e = phase_event(ctx, ph);
    if (e)
        cudaEventRecord(e, st);
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool load_encode()
{
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// 2-D uint8 tensor [rows, cols] (cols contiguous), box {128 bytes, box_rows},
// 128-byte swizzle; rows past the end read as zero.
bool make_tmap_u8(CUtensorMap *tm, const void *base, int64_t rows, int64_t cols, int box_rows)
{
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols};
    cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = g_encode(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

int check_ctx(gemmar_ctx *ctx)
{
    if (ctx == nullptr)
        return GEMMAR_ERR_ARG;
    if (ctx->disabled)
        return GEMMAR_ERR_DISABLED;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return GEMMAR_ERR_CUDA;
    if (dev != ctx->device)
        return GEMMAR_ERR_DEVICE;
    return GEMMAR_OK;
}

int shape_rules(int P, int64_t M, int64_t N, int64_t K, int bands, int scale_kind)
{
    if (P < 1 || P > kMaxP || M < 1 || N < 1 || K < 1 || bands < 1)
        return GEMMAR_ERR_ARG;
    if (bands > kMaxBands || bands > M || M % bands != 0)
        return GEMMAR_ERR_SHAPE;
    // N is tiled by 256/128 (blockscale: also the B-scale block; ptpc) or 224/128 (mx)
    const bool n_ok = scale_kind == GEMMAR_SCALE_MX32 ? (N % 128 == 0 || N % 224 == 0) : (N % 128 == 0);
    if (!n_ok || K % 128 != 0)
        return GEMMAR_ERR_SHAPE;
    if (N > 65536 || K > 65536 || M > (int64_t(1) << 24))
        return GEMMAR_ERR_SHAPE;
    return GEMMAR_OK;
}

int mx_tile_n(int64_t N) { return (N % 224 == 0) ? 224 : 128; }
int ptpc_tile_n(int64_t N) { return (N % 256 == 0) ? 256 : 128; }

bool known_scale_kind(int k)
{
    return k == GEMMAR_SCALE_BLOCK128 || k == GEMMAR_SCALE_MX32 || k == GEMMAR_SCALE_PTPC;
}

TileGrid make_grid(int P, int64_t M, int64_t N, int64_t K, int bands, int bn, int slice_loop = 0)
{
    TileGrid g;
    if (slice_loop)
        bands = 1;
    g.P = P;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.bands = bands;
    g.rows_per_band = (int)(M / bands);
    g.mt_per_band = (g.rows_per_band + 127) / 128;
    g.ntiles_n = (int)(N / bn);
    g.slice_loop = slice_loop;
    g.num_tiles = (slice_loop ? 1 : P) * bands * g.mt_per_band * g.ntiles_n;
    return g;
}

// The blockscale kernel splits 65536 registers between its warp roles with
// setmaxnreg; that split needs the kernel to have been built for 128 per thread
// (512 threads).
bool register_split_ok(int bn)
{
    return gemm_blockscale_split_ok(bn);
}

int64_t mx_sfa_bytes(int P, int64_t M, int64_t K, int bands)
{
    const int64_t rpb = M / bands, mtpb = (rpb + 127) / 128;
    return (int64_t)P * bands * mtpb * (K / 128) * 512;
}

int64_t mx_sfb_bytes(int P, int64_t N, int64_t K, int bn) { return (int64_t)P * (N / bn) * (K / 128) * 1024; }

#define CUDA_OK(x)                          \
    do {                                    \
        if ((x) != cudaSuccess)             \
            return GEMMAR_ERR_CUDA;         \
    } while (0)

// One GEMM launch over P slices.  scale_kind selects the kernel; o says where
// the result goes.
int run_gemm(gemmar_ctx *ctx, int P, const uint8_t *const *A, const void *const *sa, const uint8_t *const *B,
             const void *const *sb, int scale_kind, int64_t M, int64_t N, int64_t K, int bands, const GemmOut &o,
             cudaStream_t st, int slice_loop = 0)
{
    if (!load_encode())
        return GEMMAR_ERR_CUDA;
    if (scale_kind == GEMMAR_SCALE_BLOCK128) {
        // slice_loop 2 (partials summed on chip) exists on the CTA-pair kernel only
        const BsPlan pl = plan_blockscale(P, M, N, K, bands, slice_loop, ctx->num_sms,
                                          (slice_loop == 2 || (ctx->flags & GEMMAR_CTA_PAIR)) ? 1 : 0);
        if (slice_loop == 2 && !pl.pair)
            return GEMMAR_ERR_DEVICE;
        if (!pl.pair && !register_split_ok(pl.bn))
            return GEMMAR_ERR_DEVICE;
        BsParams prm;
        std::memset(&prm, 0, sizeof(prm));
        for (int p = 0; p < P; ++p) {
            if (!make_tmap_u8(&prm.tmA[p], A[p], M, K, 128) || !make_tmap_u8(&prm.tmB[p], B[p], N, K, pl.box_b_rows))
                return GEMMAR_ERR_CUDA;
            prm.sa[p] = static_cast<const float *>(sa[p]);
            prm.sb[p] = static_cast<const float *>(sb[p]);
        }
        prm.g = pl.g;
        prm.o = o;
        prm.status = ctx->status;
        prm.timeout_ns = ctx->timeout_ns;
        CUDA_OK(launch_blockscale(prm, pl, st));
    } else if (scale_kind == GEMMAR_SCALE_PTPC) {
        // one fp32 scale per row of A and of B: whole-K accumulation, scaled in the epilogue
        const int bn = ptpc_tile_n(N);
        if (slice_loop)
            bands = 1;
        if (!gemm_mx_split_ok(gemm_ptpc_num_regs(bn)))
            return GEMMAR_ERR_DEVICE;
        MxParams prm;
        std::memset(&prm, 0, sizeof(prm));
        for (int p = 0; p < P; ++p) {
            if (!make_tmap_u8(&prm.tmA[p], A[p], M, K, 128) || !make_tmap_u8(&prm.tmB[p], B[p], N, K, bn))
                return GEMMAR_ERR_CUDA;
            prm.pa[p] = static_cast<const float *>(sa[p]);
            prm.pb[p] = static_cast<const float *>(sb[p]);
        }
        prm.g = make_grid(P, M, N, K, bands, bn, slice_loop);
        prm.o = o;
        prm.status = ctx->status;
        prm.timeout_ns = ctx->timeout_ns;
        const int grid = std::min(prm.g.num_tiles, ctx->num_sms);
        CUDA_OK(launch_gemm_ptpc(prm, bn, grid, st));
    } else {
        const int bn = mx_tile_n(N);
        if (slice_loop)
            bands = 1;
        if (!gemm_mx_split_ok(gemm_mx_num_regs(bn)))
            return GEMMAR_ERR_DEVICE;
        if (mx_sfa_bytes(P, M, K, bands) > ctx->sfa_bytes || mx_sfb_bytes(P, N, K, bn) > ctx->sfb_bytes)
            return GEMMAR_ERR_WORKSPACE;
        CUDA_OK(launch_mx_repack(reinterpret_cast<const uint8_t *const *>(sa),
                                 reinterpret_cast<const uint8_t *const *>(sb), P, (int)M, (int)N, (int)K, bands, bn,
                                 ctx->sfa, ctx->sfb, st));
        MxParams prm;
        std::memset(&prm, 0, sizeof(prm));
        for (int p = 0; p < P; ++p)
            if (!make_tmap_u8(&prm.tmA[p], A[p], M, K, 128) || !make_tmap_u8(&prm.tmB[p], B[p], N, K, bn))
                return GEMMAR_ERR_CUDA;
        prm.sfa = ctx->sfa;
        prm.sfb = ctx->sfb;
        prm.g = make_grid(P, M, N, K, bands, bn, slice_loop);
        prm.o = o;
        prm.status = ctx->status;
        prm.timeout_ns = ctx->timeout_ns;
        const int grid = std::min(prm.g.num_tiles, ctx->num_sms);
        CUDA_OK(launch_gemm_mx(prm, bn, grid, st));
    }
    return GEMMAR_OK;
}

int gemm_single(gemmar_ctx *ctx, const uint8_t *A, const void *sa, const uint8_t *B, const void *sb, void *C,
                int c_dtype, int64_t M, int64_t N, int64_t K, int scale_kind, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!A || !sa || !B || !sb || !C || (c_dtype != GEMMAR_DTYPE_F32 && c_dtype != GEMMAR_DTYPE_BF16))
        return GEMMAR_ERR_ARG;
    if ((rc = shape_rules(1, M, N, K, 1, scale_kind)))
        return rc;
    if (!aligned16(A) || !aligned16(B) || !aligned16(C) || !aligned16(sa) || !aligned16(sb))
        return GEMMAR_ERR_ALIGN;
    GemmOut o{C, nullptr, c_dtype == GEMMAR_DTYPE_BF16 ? OUT_BF16 : OUT_F32, -1};
    return run_gemm(ctx, 1, &A, &sa, &B, &sb, scale_kind, M, N, K, 1, o, as_stream(stream));
}

}  // namespace

// ============================================================================ ABI

GEMMAR_API int gemmar_supports(int P, int64_t M, int64_t N, int64_t K, int bands, int scale_kind)
{
    if (!known_scale_kind(scale_kind))
        return GEMMAR_ERR_ARG;
    return shape_rules(P, M, N, K, bands, scale_kind);
}

GEMMAR_API int64_t gemmar_workspace_bytes(const gemmar_ctx *ctx) { return ctx ? ctx->total_bytes : 0; }

GEMMAR_API int gemmar_status(gemmar_ctx *ctx, int *detail)
{
    if (ctx == nullptr)
        return GEMMAR_ERR_ARG;
    ptx::DevStatus st{0, 0};
    if (cudaMemcpy(&st, ctx->status, sizeof(st), cudaMemcpyDeviceToHost) != cudaSuccess)
        return GEMMAR_ERR_CUDA;
    if (detail)
        *detail = st.detail;
    if (st.code != 0)
        ctx->disabled = 1;
    return st.code;
}

GEMMAR_API int gemmar_overlap_stats(gemmar_ctx *ctx, int64_t *overlapped, int64_t *total)
{
    if (ctx == nullptr || overlapped == nullptr || total == nullptr)
        return GEMMAR_ERR_ARG;
    *overlapped = 0;
    *total = ctx->ov_total;
    if (ctx->ov_bands == 0)
        return GEMMAR_OK;
    std::vector<uint32_t> claimed((size_t)ctx->ov_bands);
    if (cudaMemcpy(claimed.data(), ctx->band_done + ctx->ov_bands, sizeof(uint32_t) * claimed.size(),
                   cudaMemcpyDeviceToHost) != cudaSuccess)
        return GEMMAR_ERR_CUDA;
    for (uint32_t c : claimed)   // a counter can pass the band's block count by the claims that found it empty
        *overlapped += std::min<int64_t>(c, ctx->ov_bpb);
    return GEMMAR_OK;
}

GEMMAR_API int gemmar_destroy(gemmar_ctx *ctx)
{
    if (ctx == nullptr)
        return GEMMAR_ERR_ARG;
    int prev = -1;
    cudaGetDevice(&prev);
    if (ctx->device >= 0)
        cudaSetDevice(ctx->device);
    cudaDeviceSynchronize();
    cudaFree(ctx->W);
    cudaFree(ctx->band_done);
    cudaFree(ctx->status);
    cudaFree(ctx->sfa);
    cudaFree(ctx->sfb);
    cudaFree(ctx->wire_q);
    cudaFree(ctx->wire_s);
    cudaFree(ctx->counters);
    for (cudaEvent_t e : ctx->events)
        cudaEventDestroy(e);
    if (prev >= 0)
        cudaSetDevice(prev);
    delete ctx;
    return GEMMAR_OK;
}

GEMMAR_API int gemm_blockscale_fp8(gemmar_ctx *ctx, const uint8_t *A, const float *sa, const uint8_t *B,
                                   const float *sb, void *C, int c_dtype, int64_t M, int64_t N, int64_t K,
                                   void *stream)
{
    return gemm_single(ctx, A, sa, B, sb, C, c_dtype, M, N, K, GEMMAR_SCALE_BLOCK128, stream);
}

GEMMAR_API int gemm_ptpc_fp8(gemmar_ctx *ctx, const uint8_t *A, const float *sa, const uint8_t *B, const float *sb,
                             void *C, int c_dtype, int64_t M, int64_t N, int64_t K, void *stream)
{
    return gemm_single(ctx, A, sa, B, sb, C, c_dtype, M, N, K, GEMMAR_SCALE_PTPC, stream);
}

GEMMAR_API int gemm_mxfp8(gemmar_ctx *ctx, const uint8_t *A, const uint8_t *ea, const uint8_t *B, const uint8_t *eb,
                          void *C, int c_dtype, int64_t M, int64_t N, int64_t K, void *stream)
{
    return gemm_single(ctx, A, ea, B, eb, C, c_dtype, M, N, K, GEMMAR_SCALE_MX32, stream);
}

GEMMAR_API int band_reduce(gemmar_ctx *ctx, const float *W, int P, int64_t M, int64_t N, int bands, uint16_t *out,
                           void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!W || !out)
        return GEMMAR_ERR_ARG;
    if (P < 1 || P > kMaxP || M < 1 || N < 1 || bands < 1)
        return GEMMAR_ERR_ARG;
    if (M % bands != 0 || N % 8 != 0 || bands > kMaxBands)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(W) || !aligned16(out))
        return GEMMAR_ERR_ALIGN;
    CUDA_OK(launch_band_reduce(W, out, P, M, N, bands, nullptr, 0, ctx->status, ctx->timeout_ns, ctx->num_sms,
                               as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int rowquant_e4m3(gemmar_ctx *ctx, const void *x, int x_dtype, int64_t M, int64_t N, uint8_t *q,
                             float *row_scale, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!x || !q || !row_scale || (x_dtype != GEMMAR_DTYPE_F32 && x_dtype != GEMMAR_DTYPE_BF16) || M < 1 || N < 1)
        return GEMMAR_ERR_ARG;
    if (N % 16 != 0)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(row_scale))
        return GEMMAR_ERR_ALIGN;
    CUDA_OK(launch_rowquant(x, x_dtype == GEMMAR_DTYPE_BF16, M, N, q, row_scale, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int rowdequant_e4m3(gemmar_ctx *ctx, const uint8_t *q, const float *row_scale, int64_t M, int64_t N,
                               uint16_t *y, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!q || !row_scale || !y || M < 1 || N < 1)
        return GEMMAR_ERR_ARG;
    if (N % 16 != 0)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(q) || !aligned16(row_scale) || !aligned16(y))
        return GEMMAR_ERR_ALIGN;
    CUDA_OK(launch_rowdequant(q, row_scale, M, N, y, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int quant_blockscale_e4m3(gemmar_ctx *ctx, const void *x, int x_dtype, int64_t R, int64_t C,
                                     int group_rows, uint8_t *q, float *scales, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!x || !q || !scales || R < 1 || C < 1 || (group_rows != 1 && group_rows != 128) ||
        (x_dtype != GEMMAR_DTYPE_F32 && x_dtype != GEMMAR_DTYPE_BF16))
        return GEMMAR_ERR_ARG;
    if (C % 128 != 0)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(scales))
        return GEMMAR_ERR_ALIGN;
    CUDA_OK(launch_quant_blockscale(x, x_dtype == GEMMAR_DTYPE_BF16, R, C, group_rows, q, scales, ctx->num_sms,
                                    as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int quant_mx_e4m3(gemmar_ctx *ctx, const void *x, int x_dtype, int64_t R, int64_t C, uint8_t *q,
                             uint8_t *e8m0, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!x || !q || !e8m0 || R < 1 || C < 1 || (x_dtype != GEMMAR_DTYPE_F32 && x_dtype != GEMMAR_DTYPE_BF16))
        return GEMMAR_ERR_ARG;
    if (C % 32 != 0)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q) || !aligned16(e8m0))
        return GEMMAR_ERR_ALIGN;
    CUDA_OK(launch_quant_mx(x, x_dtype == GEMMAR_DTYPE_BF16, R, C, q, e8m0, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int fused_gemm_reduce(gemmar_ctx *ctx, int P, const uint8_t *const *A, const void *const *sa,
                                 const uint8_t *const *B, const void *const *sb, int scale_kind, int64_t M,
                                 int64_t N, int64_t K, int bands, uint32_t flags, uint16_t *out, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!A || !sa || !B || !sb || !out || !known_scale_kind(scale_kind))
        return GEMMAR_ERR_ARG;
    if (bands == 0)
        bands = P;
    if ((rc = shape_rules(P, M, N, K, bands, scale_kind)))
        return rc;
    for (int p = 0; p < P; ++p) {
        if (!A[p] || !sa[p] || !B[p] || !sb[p])
            return GEMMAR_ERR_ARG;
        if (!aligned16(A[p]) || !aligned16(sa[p]) || !aligned16(B[p]) || !aligned16(sb[p]))
            return GEMMAR_ERR_ALIGN;
    }
    if (!aligned16(out))
        return GEMMAR_ERR_ALIGN;
    // on-chip partial sums: mx on the mx kernel, blockscale on the CTA-pair kernel
    // (N % 256 == 0); other blockscale shapes take the band path, whose bits they reproduce
    // ptpc applies its scales after the whole K of a slice, so its only in-tile
    // reduction is the on-chip one (GEMMAR_FUSE_SLICES takes it too)
    const bool onchip = ((flags & GEMMAR_FUSE_ONCHIP) ||
                         (scale_kind == GEMMAR_SCALE_PTPC && (flags & GEMMAR_FUSE_SLICES))) &&
                        (scale_kind != GEMMAR_SCALE_BLOCK128 || plan_blockscale(P, M, N, K, bands, 2, ctx->num_sms, 1).pair);
    const bool slices = onchip || ((flags & GEMMAR_FUSE_SLICES) != 0 && !(flags & GEMMAR_FUSE_ONCHIP));
    if (!slices && blocked_partial_floats(P, M, bands, N) > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    if ((flags & GEMMAR_FP8_WIRE) && (M > ctx->max_M || M * N > ctx->max_M * ctx->N))   // row scales, codes
        return GEMMAR_ERR_WORKSPACE;
    cudaStream_t st = as_stream(stream);
    ctx->ov_bands = 0;
    ctx->ov_total = 0;
    // fp8 wire on the band path: the band reduce can quantise the rows itself
    const bool fuse_q = !slices && (flags & GEMMAR_FP8_WIRE) && (flags & GEMMAR_FUSE_QUANTIZE) &&
                        N <= kBandQuantMaxN;
    if (slices) {
        // every tile accumulates all P slices itself: no partials, no band reduce
        if (flags & GEMMAR_DEBUG_CANARY)
            CUDA_OK(cudaMemsetAsync(out, 0xFF, sizeof(uint16_t) * (size_t)(M * N), st));
        mark(ctx, GEMMAR_PHASE_GEMM, st);
        GemmOut os{out, nullptr, OUT_BF16, -1};
        if ((rc = run_gemm(ctx, P, A, sa, B, sb, scale_kind, M, N, K, 1, os, st, onchip ? 2 : 1)))
            return rc;
        mark(ctx, GEMMAR_PHASE_REDUCE, st);
    } else {
        int bn;
        uint32_t expected;   // every epilogue warp signals once per retired tile
        bool inkernel = false;   // the GEMM's reducer warps take the bands that retire while it runs
        if (scale_kind == GEMMAR_SCALE_BLOCK128) {
            const BsPlan pl = plan_blockscale(P, M, N, K, bands, 0, ctx->num_sms,
                                              (ctx->flags & GEMMAR_CTA_PAIR) ? 1 : 0);
            bn = pl.bn;
            expected = pl.band_signals;
            inkernel = !pl.pair && !(flags & GEMMAR_SERIAL_REDUCE);
        } else {
            bn = scale_kind == GEMMAR_SCALE_PTPC ? ptpc_tile_n(N) : mx_tile_n(N);
            const TileGrid g = make_grid(P, M, N, K, bands, bn);
            expected = (uint32_t)(g.mt_per_band * g.ntiles_n * P * 8);
            inkernel = !(flags & GEMMAR_SERIAL_REDUCE);
        }
        // band retire counters, then the reducer warps' per-band claim counters
        uint32_t *claim = ctx->band_done + bands;
        CUDA_OK(cudaMemsetAsync(ctx->band_done, 0, sizeof(uint32_t) * 2 * bands, st));
        if (flags & GEMMAR_DEBUG_CANARY) {
            CUDA_OK(cudaMemsetAsync(ctx->W, 0xFF, sizeof(float) * (size_t)blocked_partial_floats(P, M, bands, N), st));
            CUDA_OK(cudaMemsetAsync(out, 0xFF, sizeof(uint16_t) * (size_t)(M * N), st));
        }
        GemmOut o{ctx->W, ctx->band_done, OUT_PARTIAL_F32, (flags & GEMMAR_FAULT_SKIP_BAND) ? 0 : -1,
                  inkernel ? claim : nullptr, out, expected};
        {
            const int64_t mtpb = (M / bands + 127) / 128;
            ctx->ov_bpb = mtpb * (N / bn) * 4 * (bn / 32);
            ctx->ov_bands = inkernel ? bands : 0;
            ctx->ov_total = inkernel ? ctx->ov_bpb * bands : 0;
        }
        mark(ctx, GEMMAR_PHASE_GEMM, st);
        if ((rc = run_gemm(ctx, P, A, sa, B, sb, scale_kind, M, N, K, bands, o, st)))
            return rc;
        mark(ctx, GEMMAR_PHASE_REDUCE, st);
        if (fuse_q) {
            // the remaining blocks' sums go straight to the row quantiser
            CUDA_OK(launch_band_reduce_quant(ctx->W, out, P, M, N, bands, bn, ctx->band_done, expected,
                                             inkernel ? claim : nullptr, ctx->wire_q, ctx->wire_s, ctx->status,
                                             ctx->timeout_ns, st));
        } else {
            CUDA_OK(launch_band_reduce_blocked(ctx->W, out, P, M, N, bands, bn, ctx->band_done, expected,
                                               inkernel ? claim : nullptr, ctx->status, ctx->timeout_ns,
                                               ctx->num_sms, st));
        }
    }
    mark(ctx, GEMMAR_PHASE_QUANTIZE, st);
    if ((flags & GEMMAR_FP8_WIRE) && !fuse_q)
        CUDA_OK(launch_rowquant(out, 1, M, N, ctx->wire_q, ctx->wire_s, ctx->num_sms, st));
    mark(ctx, GEMMAR_PHASE_DEQUANTIZE, st);
    if (flags & GEMMAR_FP8_WIRE)
        CUDA_OK(launch_rowdequant(ctx->wire_q, ctx->wire_s, M, N, out, ctx->num_sms, st));
    mark(ctx, GEMMAR_NUM_PHASES, st);
    if (ctx->timing && ctx->recorded < kMaxTimedCalls)
        ++ctx->recorded;
    return GEMMAR_OK;
}

GEMMAR_API int gemmar_set_phase_timing(gemmar_ctx *ctx, int enable)
{
    if (ctx == nullptr)
        return GEMMAR_ERR_ARG;
    ctx->timing = enable ? 1 : 0;
    return GEMMAR_OK;
}

GEMMAR_API int gemmar_phase_times(gemmar_ctx *ctx, float *ms, int *calls)
{
    if (ctx == nullptr || ms == nullptr)
        return GEMMAR_ERR_ARG;
    for (int ph = 0; ph < GEMMAR_NUM_PHASES; ++ph)
        ms[ph] = 0.0f;
    for (int c = 0; c < ctx->recorded; ++c) {
        cudaEvent_t *ev = &ctx->events[(size_t)c * kEventsPerCall];
        if (cudaEventSynchronize(ev[GEMMAR_NUM_PHASES]) != cudaSuccess)
            return GEMMAR_ERR_CUDA;
        for (int ph = 0; ph < GEMMAR_NUM_PHASES; ++ph) {
            float t = 0.0f;
            if (cudaEventElapsedTime(&t, ev[ph], ev[ph + 1]) != cudaSuccess)
                return GEMMAR_ERR_CUDA;
            ms[ph] += t;
        }
    }
    if (calls)
        *calls = ctx->recorded;
    ctx->recorded = 0;
    return GEMMAR_OK;
}

// ---------------------------------------------------------------- residual stream and adapters

namespace {

bool known_dtype(int d) { return d == GEMMAR_DTYPE_F32 || d == GEMMAR_DTYPE_BF16; }

// A matrix of rows at a stride: 0 (one row for all) or at least the row's length.
int check_rows(const void *p, int64_t stride, int64_t cols, int elem_bytes, bool written = false)
{
    if (stride < 0 || (stride != 0 && stride < cols) || (written && stride == 0))
        return GEMMAR_ERR_ARG;
    if (!aligned16(p) || (stride * elem_bytes) % 16 != 0)
        return GEMMAR_ERR_ALIGN;
    return GEMMAR_OK;
}

// Do two bf16 matrices of T rows share elements?  Rows at one stride may lie between one
// another (columns of a wider matrix); at two strides only the same start counts.
bool rows_meet(const uint16_t *a, int64_t a_stride, int64_t a_cols, const uint16_t *b, int64_t b_stride, int64_t b_cols,
               int64_t T)
{
    if (a == b)
        return true;
    if (a_stride != b_stride && T > 1)
        return false;
    const int64_t d = ((intptr_t)b - (intptr_t)a) / 2, last = (T - 1) * a_stride;
    if (d >= last + a_cols || -d >= last + b_cols)
        return false;
    const int64_t off = a_stride > 0 && T > 1 ? ((d % a_stride) + a_stride) % a_stride : d;
    return T == 1 || a_stride == 0 || off < a_cols || a_stride - off < b_cols;
}

int norm_shape(int64_t M, int64_t N)
{
    if (M < 1 || N < 1)
        return GEMMAR_ERR_ARG;
    if (N % 8 != 0 || N > GEMMAR_NORM_MAX_N || M > (int64_t(1) << 24))
        return GEMMAR_ERR_SHAPE;
    return GEMMAR_OK;
}

// What lora_apply and lora_apply_bwd share.
int check_lora(const int32_t *order, const int32_t *offsets, const uint16_t *A, const uint16_t *B, const float *scales,
               const int32_t *ranks, int64_t T, int64_t K, int64_t N, int R, int r)
{
    if (!order || !offsets || !A || !B || !scales || T < 1 || K < 1 || N < 1 || R < 1 || r < 1)
        return GEMMAR_ERR_ARG;
    if (K % 8 != 0 || N % 8 != 0 || K > 65536 || N > 65536 || T > (int64_t(1) << 24) ||
        R > GEMMAR_LORA_MAX_ADAPTERS || r > GEMMAR_LORA_MAX_RANK)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(order) || !aligned16(offsets) || !aligned16(A) || !aligned16(B) || !aligned16(scales) ||
        !aligned16(ranks))
        return GEMMAR_ERR_ALIGN;
    return GEMMAR_OK;
}

}  // namespace

GEMMAR_API int norm_gate_residual(gemmar_ctx *ctx, const void *y, int y_dtype, int64_t y_stride, const void *h,
                                  int h_dtype, int64_t h_stride, const float *w_post, const float *w_pre,
                                  const uint16_t *gate, int64_t gate_stride, float alpha, float beta, float eps,
                                  int64_t M, int64_t N, void *t, uint16_t *u, uint8_t *q, float *scales, float *rstd,
                                  void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!y || !h || !t || !known_dtype(y_dtype) || !known_dtype(h_dtype) || (!w_pre && (u || q)) || (!q) != (!scales) ||
        !std::isfinite(alpha) || !std::isfinite(beta) || !std::isfinite(eps) || eps < 0.0f)
        return GEMMAR_ERR_ARG;
    if ((rc = norm_shape(M, N)))
        return rc;
    if (q && N % 128 != 0)
        return GEMMAR_ERR_SHAPE;
    if ((rc = check_rows(y, y_stride, N, y_dtype == GEMMAR_DTYPE_BF16 ? 2 : 4)) ||
        (rc = check_rows(h, h_stride, N, h_dtype == GEMMAR_DTYPE_BF16 ? 2 : 4)) ||
        (gate && (rc = check_rows(gate, gate_stride, N, 2))))
        return rc;
    if (!aligned16(w_post) || !aligned16(w_pre) || !aligned16(t) || !aligned16(u) || !aligned16(q) ||
        !aligned16(scales) || !aligned16(rstd))
        return GEMMAR_ERR_ALIGN;
    NormArgs a{y, h, y_dtype == GEMMAR_DTYPE_BF16, h_dtype == GEMMAR_DTYPE_BF16, y_stride, h_stride, w_post, w_pre,
               gate, gate_stride, alpha, beta, eps, M, (int)N, t, u, q, scales, rstd};
    CUDA_OK(launch_norm(a, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int norm_gate_residual_bwd(gemmar_ctx *ctx, const void *y, int y_dtype, int64_t y_stride, const void *h,
                                      int h_dtype, int64_t h_stride, const float *rstd, const float *w_post,
                                      const float *w_pre, const uint16_t *gate, int64_t gate_stride, float alpha,
                                      float beta, int64_t M, int64_t N, const void *dt, int64_t dt_stride,
                                      const uint16_t *du, int64_t du_stride, void *dy, void *dh, float *dw_post,
                                      float *dw_pre, void *dgate, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!y || !h || !rstd || !dy || !dh || !known_dtype(y_dtype) || !known_dtype(h_dtype) || (w_pre && !du) ||
        (dw_post && !w_post) || (dw_pre && !w_pre) || (dgate && !gate) || !std::isfinite(alpha) ||
        !std::isfinite(beta))
        return GEMMAR_ERR_ARG;
    if ((rc = norm_shape(M, N)))
        return rc;
    const int yb = y_dtype == GEMMAR_DTYPE_BF16 ? 2 : 4, hb = h_dtype == GEMMAR_DTYPE_BF16 ? 2 : 4;
    if ((rc = check_rows(y, y_stride, N, yb)) || (rc = check_rows(h, h_stride, N, hb)) ||
        (gate && (rc = check_rows(gate, gate_stride, N, 2))) || (dt && (rc = check_rows(dt, dt_stride, N, hb))) ||
        (w_pre && (rc = check_rows(du, du_stride, N, 2))))
        return rc;
    if (!aligned16(rstd) || !aligned16(w_post) || !aligned16(w_pre) || !aligned16(dy) || !aligned16(dh) ||
        !aligned16(dw_post) || !aligned16(dw_pre) || !aligned16(dgate))
        return GEMMAR_ERR_ALIGN;
    if (norm_bwd_ws_floats(M, (int)N, ctx->num_sms) > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    NormBwdArgs a{y, h, yb == 2, hb == 2, y_stride, h_stride, rstd, w_post, w_pre, gate, gate_stride, alpha, beta, M,
                  (int)N, dt, dt_stride, w_pre ? du : nullptr, du_stride, dy, dh, dw_post, dw_pre, dgate};
    CUDA_OK(launch_norm_bwd(a, ctx->W, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int lora_plan(gemmar_ctx *ctx, const int32_t *adapter_ids, int64_t T, int R, int32_t *order,
                         int32_t *offsets, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!adapter_ids || !order || !offsets || T < 1 || R < 1)
        return GEMMAR_ERR_ARG;
    if (T > (int64_t(1) << 24) || R > GEMMAR_LORA_MAX_ADAPTERS)
        return GEMMAR_ERR_SHAPE;
    if (!aligned16(adapter_ids) || !aligned16(order) || !aligned16(offsets))
        return GEMMAR_ERR_ALIGN;
    CUDA_OK(launch_lora_plan(adapter_ids, T, R, order, offsets, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int lora_apply(gemmar_ctx *ctx, const uint16_t *x, int64_t x_stride, const int32_t *order,
                          const int32_t *offsets, const uint16_t *A, const uint16_t *B, const float *scales,
                          const int32_t *ranks, int64_t T, int64_t K, int64_t N, int R, int r, const uint16_t *y,
                          int64_t y_stride, uint16_t *out, int64_t out_stride, float *v, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!x || !out || (y == out && y_stride != out_stride))
        return GEMMAR_ERR_ARG;
    if ((rc = check_lora(order, offsets, A, B, scales, ranks, T, K, N, R, r)) || (rc = check_rows(x, x_stride, K, 2)) ||
        (y && (rc = check_rows(y, y_stride, N, 2))) || (rc = check_rows(out, out_stride, N, 2, true)))
        return rc;
    if (!aligned16(v))
        return GEMMAR_ERR_ALIGN;
    const LoraArgs l{order, offsets, ranks, scales, T, R, r};
    if (lora_apply_floats(l) > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    cudaStream_t st = as_stream(stream);
    const LoraCall p{ctx->num_sms, ctx->status, ctx->timeout_ns};
    CUDA_OK(launch_lora_apply(l, p, x, x_stride, A, (int)K, B, (int)N, y, y_stride, out, out_stride, v, ctx->W, st));
    return GEMMAR_OK;
}

GEMMAR_API int lora_apply_bwd(gemmar_ctx *ctx, const uint16_t *x, int64_t x_stride, const uint16_t *dy,
                              int64_t dy_stride, const int32_t *order, const int32_t *offsets, const uint16_t *A,
                              const uint16_t *B, const float *scales, const int32_t *ranks, const float *v, int64_t T,
                              int64_t K, int64_t N, int R, int r, const uint16_t *dx0, int64_t dx0_stride,
                              uint16_t *dx, int64_t dx_stride, uint16_t *dA, uint16_t *dB, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!x || !dy || !v || !dx || !dA || !dB || (dx0 == dx && dx0_stride != dx_stride))
        return GEMMAR_ERR_ARG;
    if ((rc = check_lora(order, offsets, A, B, scales, ranks, T, K, N, R, r)) || (rc = check_rows(x, x_stride, K, 2)) ||
        (rc = check_rows(dy, dy_stride, N, 2)) || (dx0 && (rc = check_rows(dx0, dx0_stride, K, 2))) ||
        (rc = check_rows(dx, dx_stride, K, 2, true)))
        return rc;
    if (!aligned16(v) || !aligned16(dA) || !aligned16(dB))
        return GEMMAR_ERR_ALIGN;
    const int64_t na = (int64_t)R * r * K, nb = (int64_t)R * r * N;
    auto meet = [](const uint16_t *p, int64_t n, const uint16_t *q, int64_t m) { return rows_meet(p, n, n, q, m, m, 1); };
    if (rows_meet(dx, dx_stride, K, x, x_stride, K, T) || rows_meet(dx, dx_stride, K, dy, dy_stride, N, T) ||
        meet(dA, na, A, na) || meet(dA, na, B, nb) || meet(dB, nb, A, na) || meet(dB, nb, B, nb) || meet(dA, na, dB, nb))
        return GEMMAR_ERR_ARG;
    if (lora_grad_floats(T, r, (int)K, (int)N) > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    cudaStream_t st = as_stream(stream);
    const LoraArgs l{order, offsets, ranks, scales, T, R, r};
    const LoraCall p{ctx->num_sms, ctx->status, ctx->timeout_ns};
    CUDA_OK(launch_lora_apply_bwd(l, p, x, x_stride, dy, dy_stride, A, (int)K, B, (int)N, v, dx0, dx0_stride, dx, dx_stride,
                                  dA, dB, ctx->W, ctx->W_floats, st));
    return GEMMAR_OK;
}

// ---------------------------------------------------------------- feed-forward half

namespace {

bool known_act(int act) { return act >= GEMMAR_ACT_NONE && act <= GEMMAR_ACT_GELU_TANH; }

int elem_bytes(int dtype) { return dtype == GEMMAR_DTYPE_BF16 ? 2 : 4; }

}  // namespace

GEMMAR_API int gemm_blockscale_act(gemmar_ctx *ctx, const uint8_t *A, const float *sa, const uint8_t *B, const float *sb,
                                   int act, int gated, const float *bias, const void *residual, int r_dtype,
                                   int64_t r_stride, int64_t M, int64_t N, int64_t K, void *C, int c_dtype,
                                   int64_t c_stride, uint8_t *q, float *scales, uint16_t *z, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!A || !sa || !B || !sb || (!C && !q) || (!q) != (!scales) || !known_act(act) || (gated != 0 && gated != 1) ||
        (residual && !known_dtype(r_dtype)) || (C && !known_dtype(c_dtype)) ||
        (C && residual == C && (r_dtype != c_dtype || r_stride != c_stride)))
        return GEMMAR_ERR_ARG;
    if (N > 65536 || (rc = shape_rules(1, M, gated ? 2 * N : N, K, 1, GEMMAR_SCALE_BLOCK128)))
        return N > 65536 ? GEMMAR_ERR_SHAPE : rc;
    if (N % 128 != 0)
        return GEMMAR_ERR_SHAPE;
    if ((residual && (rc = check_rows(residual, r_stride, N, elem_bytes(r_dtype)))) ||
        (C && (rc = check_rows(C, c_stride, N, elem_bytes(c_dtype), true))))
        return rc;
    if (!aligned16(A) || !aligned16(B) || !aligned16(sa) || !aligned16(sb) || !aligned16(bias) || !aligned16(q) ||
        !aligned16(scales) || !aligned16(z))
        return GEMMAR_ERR_ALIGN;
    // an output over what is still being read; residual may be C itself
    const int64_t P = gated ? 2 * N : N;
    const int rb = elem_bytes(r_dtype), cb = elem_bytes(c_dtype);
    const Span c = span_rows(C, N * cb, c_stride * cb, M), res = span_rows(residual, N * rb, r_stride * rb, M);
    const Span qs = span(q, M * N), ss = span(scales, M * N / 32), zs = span(z, 2 * M * P);
    if (any_meet({c, qs, ss, zs}, {span(A, M * K), span(sa, M * K / 32), span(B, P * K), span(sb, P / 128 * (K / 128) * 4), span(bias, 4 * P)}) ||
        any_meet({qs, ss, zs}, {res}) || (C != residual && meet(c, res)))
        return GEMMAR_ERR_ARG;
    if (!load_encode())
        return GEMMAR_ERR_CUDA;
    // 128 gated rows at N = 2048, K = 7168: 13 us as few rows, 31 as tiles; 512: 35 and 31
    const bool few = gemm_act_few_ns((int)M, (int)N, (int)K, gated != 0) <= gemm_act_tiles_ns((int)M, (int)N, (int)K, gated != 0, ctx->num_sms);
    if (!few && !gemm_act_split_ok())
        return GEMMAR_ERR_DEVICE;
    ActParams p;
    std::memset(&p, 0, sizeof(p));
    if (!make_tmap_u8(&p.tmA, A, M, K, few ? gemm_act_few_rows((int)M) : 128) || !make_tmap_u8(&p.tmB, B, gated ? 2 * N : N, K, 128))
        return GEMMAR_ERR_CUDA;
    p.sa = sa;
    p.sb = sb;
    p.e = ActEpilogue{act, gated, (int)M, (int)N, (int)K, bias, residual, r_dtype == GEMMAR_DTYPE_BF16, r_stride,
                      C, c_dtype == GEMMAR_DTYPE_BF16, c_stride, q, scales, z};
    p.status = ctx->status;
    p.timeout_ns = ctx->timeout_ns;
    CUDA_OK(few ? launch_gemm_act_few(p, as_stream(stream)) : launch_gemm_act(p, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int gemm_blockscale_act_bwd(gemmar_ctx *ctx, const void *dout, int d_dtype, int64_t d_stride,
                                       const uint16_t *z, int act, int gated, int64_t M, int64_t N, uint16_t *dz,
                                       float *dbias, uint8_t *q, float *scales, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!dout || !z || (!dz && !q) || (!q) != (!scales) || !known_act(act) || (gated != 0 && gated != 1) ||
        !known_dtype(d_dtype) ||
        (dz && dz == dout && (gated || d_dtype != GEMMAR_DTYPE_BF16 || d_stride != N)))
        return GEMMAR_ERR_ARG;
    if (M < 1 || N < 1)
        return GEMMAR_ERR_ARG;
    if (N % 128 != 0 || N > (gated ? 32768 : 65536) || M > (int64_t(1) << 24))
        return GEMMAR_ERR_SHAPE;
    if ((rc = check_rows(dout, d_stride, N, elem_bytes(d_dtype))))
        return rc;
    if (!aligned16(z) || !aligned16(dz) || !aligned16(dbias) || !aligned16(q) || !aligned16(scales))
        return GEMMAR_ERR_ALIGN;
    // dz may be z itself, or dout
    const int64_t P = gated ? 2 * N : N, db = elem_bytes(d_dtype);
    const Span dzs = span(dz, 2 * M * P), bs = span(dbias, 4 * P), qs = span(q, M * P), ss = span(scales, M * P / 32);
    const Span zs = span(z, 2 * M * P), ds = span_rows(dout, N * db, d_stride * db, M);
    if (any_meet({dzs, bs, qs, ss}, {}) || any_meet({bs, qs, ss}, {zs, ds}) || (dz != z && meet(dzs, zs)) || (dz != dout && meet(dzs, ds)))
        return GEMMAR_ERR_ARG;
    if (dbias && act_bwd_ws_floats(M, (int)N, gated, ctx->num_sms) > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    const ActBwdArgs a{dout, d_dtype == GEMMAR_DTYPE_BF16, d_stride, z, act, gated, M, (int)N, dz, dbias, q, scales};
    CUDA_OK(launch_act_bwd(a, ctx->W, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int moe_route(gemmar_ctx *ctx, const uint16_t *x, int64_t x_stride, const void *w, int w_dtype,
                         const float *bias, int64_t T, int64_t H, int E, int k, int score, int renorm, float factor,
                         int32_t *ids, float *weights, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!x || !w || !ids || !weights || !known_dtype(w_dtype) || T < 1 || H < 1 || E < 1 || k < 1 || k > E ||
        (score != GEMMAR_SCORE_SOFTMAX && score != GEMMAR_SCORE_SIGMOID) || !std::isfinite(factor))
        return GEMMAR_ERR_ARG;
    if (T > GEMMAR_MOE_MAX_TOKENS || E > GEMMAR_MOE_MAX_EXPERTS || k > GEMMAR_MOE_MAX_CHOSEN || H % 8 != 0 || H > 65536)
        return GEMMAR_ERR_SHAPE;
    if ((rc = check_rows(x, x_stride, H, 2)))
        return rc;
    if (!aligned16(w) || !aligned16(bias) || !aligned16(ids) || !aligned16(weights))
        return GEMMAR_ERR_ALIGN;
    if (any_meet({span(ids, 4 * T * k), span(weights, 4 * T * k)},
                 {span_rows(x, 2 * H, 2 * x_stride, T), span(w, (int64_t)E * H * elem_bytes(w_dtype)), span(bias, 4 * (int64_t)E)}))
        return GEMMAR_ERR_ARG;
    const RouteArgs a{x, x_stride, w, w_dtype == GEMMAR_DTYPE_BF16, bias, (int)T, (int)H, E, k, score, renorm != 0, factor,
                      ids, weights};
    if (route_ws_floats(a, ctx->num_sms) > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    CUDA_OK(launch_route(a, ctx->W, ctx->counters, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

GEMMAR_API int moe_apply(gemmar_ctx *ctx, const uint8_t *xq, const float *xs, const int32_t *ids, const float *weights,
                         const int32_t *place, int64_t places, const uint8_t *w13, const float *s13, const uint8_t *w2,
                         const float *s2, int act, int64_t T, int64_t H, int64_t I, int E, int k, const uint16_t *y,
                         int64_t y_stride, uint16_t *out, int64_t out_stride, void *stream)
{
    int rc = check_ctx(ctx);
    if (rc)
        return rc;
    if (!xq || !xs || !ids || !weights || !w13 || !s13 || !w2 || !s2 || !out || !known_act(act) || T < 1 || H < 1 ||
        I < 1 || E < 1 || k < 1 || (place && (places < 1 || places > INT32_MAX)) || (y == out && y_stride != out_stride))
        return GEMMAR_ERR_ARG;
    if (T > GEMMAR_MOE_MAX_TOKENS || E > GEMMAR_MOE_MAX_EXPERTS || k > GEMMAR_MOE_MAX_CHOSEN || H % 128 != 0 ||
        I % 128 != 0 || H > 65536 || I > 32768)
        return GEMMAR_ERR_SHAPE;
    if ((y && (rc = check_rows(y, y_stride, H, 2))) || (rc = check_rows(out, out_stride, H, 2, true)))
        return rc;
    if (!aligned16(xq) || !aligned16(xs) || !aligned16(ids) || !aligned16(weights) || !aligned16(place) ||
        !aligned16(w13) || !aligned16(s13) || !aligned16(w2) || !aligned16(s2))
        return GEMMAR_ERR_ALIGN;
    const Span o = span_rows(out, 2 * H, 2 * out_stride, T);
    const int64_t w_bytes = E * H * I, s_bytes = w_bytes / (128 * 128) * 4;   // of w2; of w13 twice
    if (any_meet({o}, {span(xq, T * H), span(xs, T * H / 32), span(ids, 4 * T * k), span(weights, 4 * T * k), span(place, 4 * places),
                       span(w13, 2 * w_bytes), span(s13, 2 * s_bytes), span(w2, w_bytes), span(s2, s_bytes)}) ||
        (y != out && meet(o, span_rows(y, 2 * H, 2 * y_stride, T))))
        return GEMMAR_ERR_ARG;
    const MoeArgs a{xq, xs, ids, place, (int)(place ? places : 0), weights, w13, w2, s13, s2, (int)T, (int)H, (int)I, E, k,
                    act, y, y_stride, out, out_stride};
    const MoeLayout l = moe_layout(a, ctx->num_sms);
    if (l.floats > ctx->W_floats)
        return GEMMAR_ERR_WORKSPACE;
    if (!load_encode())
        return GEMMAR_ERR_CUDA;
    MoeParams p;
    std::memset(&p, 0, sizeof(p));
    p.a = a;
    p.pieces = ctx->W;
    p.hidden_scale = ctx->W + l.hidden_scale;
    p.parts = reinterpret_cast<uint8_t *>(ctx->W + l.parts);
    p.counters = ctx->counters + kMoeCounters;
    p.status = ctx->status;
    p.timeout_ns = ctx->timeout_ns;
    if (!make_tmap_u8(&p.tmX, xq, T, H, moe_columns((int)T)) || !make_tmap_u8(&p.tmW13, w13, (int64_t)E * 2 * I, H, 128) ||
        !make_tmap_u8(&p.tmW2, w2, (int64_t)E * H, I, 128) || !make_tmap_u8(&p.tmParts, p.parts, l.part_rows, I, 8))
        return GEMMAR_ERR_CUDA;
    CUDA_OK(launch_moe(p, ctx->num_sms, as_stream(stream)));
    return GEMMAR_OK;
}

// ---------------------------------------------------------------- create + self-test

namespace {

// Closed-form self-test: every code 0x38 (= 1.0), every scale 1 (fp32 1.0 or
// ue8m0 byte 127) -> every output equals P * K exactly.
int self_test(gemmar_ctx *ctx)
{
    const int P = std::min(2, ctx->max_P);
    const int64_t M = 128 * P, N = 256, K = 128;
    if ((int64_t)P * M * N > ctx->W_floats || ctx->N < N || ctx->K < K || ctx->max_M < M)
        return GEMMAR_OK;   // workspace too small for the test shape: nothing to run
    uint8_t *ops = nullptr;
    const size_t a_bytes = M * K, b_bytes = N * K;
    const size_t sa_bytes = M * (K / 32) * 4 + 64, sb_bytes = N * (K / 32) * 4 + 64;
    const size_t out_bytes = M * N * 2;
    const size_t total = a_bytes + b_bytes + sa_bytes + sb_bytes + out_bytes + 5 * 256;
    if (cudaMalloc(&ops, total) != cudaSuccess)
        return GEMMAR_ERR_CUDA;
    auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
    uint8_t *dA = ops, *dB = dA + al(a_bytes);
    uint8_t *dsa = dB + al(b_bytes), *dsb = dsa + al(sa_bytes);
    uint16_t *dout = reinterpret_cast<uint16_t *>(dsb + al(sb_bytes));
    int rc = GEMMAR_OK;
    cudaStream_t st;
    if (cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking) != cudaSuccess) {
        cudaFree(ops);
        return GEMMAR_ERR_CUDA;
    }
    std::vector<float> ones(std::max(sa_bytes, sb_bytes) / 4, 1.0f);
    std::vector<uint16_t> host(M * N);
    // every scale kind, on the band path and with the partials summed on chip
    for (int run = 0; run < 6 && rc == GEMMAR_OK; ++run) {
        const int kind = run % 3;
        const uint32_t flags = run < 3 ? 0u : GEMMAR_FUSE_ONCHIP;
        const uint16_t expect = (P * K == 256) ? 0x4380 : 0x4300;   // bf16 of 256 (P=2) or 128 (P=1)
        bool ok = cudaMemsetAsync(dA, 0x38, a_bytes, st) == cudaSuccess &&
                  cudaMemsetAsync(dB, 0x38, b_bytes, st) == cudaSuccess;
        if (kind == GEMMAR_SCALE_BLOCK128)
            ok = ok && cudaMemcpyAsync(dsa, ones.data(), M * (K / 128) * 4, cudaMemcpyHostToDevice, st) == cudaSuccess &&
                 cudaMemcpyAsync(dsb, ones.data(), (N / 128) * (K / 128) * 4, cudaMemcpyHostToDevice, st) == cudaSuccess;
        else if (kind == GEMMAR_SCALE_MX32)
            ok = ok && cudaMemsetAsync(dsa, 127, M * (K / 32), st) == cudaSuccess &&
                 cudaMemsetAsync(dsb, 127, N * (K / 32), st) == cudaSuccess;
        else
            ok = ok && cudaMemcpyAsync(dsa, ones.data(), M * 4, cudaMemcpyHostToDevice, st) == cudaSuccess &&
                 cudaMemcpyAsync(dsb, ones.data(), N * 4, cudaMemcpyHostToDevice, st) == cudaSuccess;
        ok = ok && cudaMemsetAsync(dout, 0, out_bytes, st) == cudaSuccess;
        if (!ok) {
            rc = GEMMAR_ERR_CUDA;
            break;
        }
        const uint8_t *As[2] = {dA, dA}, *Bs[2] = {dB, dB};
        const void *SA[2] = {dsa, dsa}, *SB[2] = {dsb, dsb};
        rc = fused_gemm_reduce(ctx, P, As, SA, Bs, SB, kind, M, N, K, P, flags, dout, st);
        if (rc == GEMMAR_OK && cudaStreamSynchronize(st) != cudaSuccess)
            rc = GEMMAR_ERR_CUDA;
        if (rc == GEMMAR_OK)
            rc = gemmar_status(ctx, nullptr);
        if (rc == GEMMAR_OK) {
            if (cudaMemcpy(host.data(), dout, out_bytes, cudaMemcpyDeviceToHost) != cudaSuccess)
                rc = GEMMAR_ERR_CUDA;
            else
                for (size_t i = 0; i < host.size(); ++i)
                    if (host[i] != expect) {
                        rc = GEMMAR_ERR_DEVICE;
                        break;
                    }
        }
    }
    cudaStreamDestroy(st);
    cudaFree(ops);
    return rc;
}

}  // namespace

GEMMAR_API int gemmar_create(gemmar_ctx **out, int device, int64_t max_M, int64_t N, int64_t K, int max_P,
                             uint32_t flags, int64_t wait_timeout_ns)
{
    if (out == nullptr)
        return GEMMAR_ERR_ARG;
    *out = nullptr;
    if (max_P < 1 || max_P > kMaxP || max_M < 1 || N < 1 || K < 1 || wait_timeout_ns < 0)
        return GEMMAR_ERR_ARG;
    if ((N % 128 != 0 && N % 224 != 0) || K % 128 != 0 || N > 65536 || K > 65536 || max_M > (int64_t(1) << 24))
        return GEMMAR_ERR_SHAPE;
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess)
        return GEMMAR_ERR_CUDA;
    if (cur != device)
        return GEMMAR_ERR_DEVICE;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, device) != cudaSuccess)
        return GEMMAR_ERR_CUDA;
    if (!(prop.major == 10 && prop.minor == 3))
        return GEMMAR_ERR_DEVICE;   // built for sm_103a only
    if (!load_encode())
        return GEMMAR_ERR_CUDA;

    gemmar_ctx *ctx = new gemmar_ctx();
    ctx->device = device;
    ctx->num_sms = prop.multiProcessorCount;
    ctx->max_M = max_M;
    ctx->N = N;
    ctx->K = K;
    ctx->max_P = max_P;
    ctx->flags = flags;
    ctx->timeout_ns = wait_timeout_ns > 0 ? (uint64_t)wait_timeout_ns : 2000000000ull;
    // fp32 partials in the tile-blocked layout: every band padded to whole
    // 128-row tiles, for up to max_P bands
    ctx->W_floats = (int64_t)max_P * (max_M + 128 * max_P) * N;
    // the adapters' gradients of max_M tokens, which pass that at N = 128 and ranks past 64
    ctx->W_floats = std::max(ctx->W_floats, lora_grad_floats(max_M, GEMMAR_LORA_MAX_RANK, 0, 0));
    // mx repack images, sized for the largest tile count any band split can give
    ctx->sfa_bytes = (int64_t)max_P * ((max_M + 127) / 128 + kMaxBands) * (K / 128) * 512;
    ctx->sfb_bytes = (int64_t)max_P * (N / 128) * (K / 128) * 1024;
    int rc = GEMMAR_OK;
    auto alloc = [&](void **p, size_t bytes) {
        if (rc == GEMMAR_OK && cudaMalloc(p, bytes) != cudaSuccess)
            rc = GEMMAR_ERR_CUDA;
        if (rc == GEMMAR_OK)
            ctx->total_bytes += (int64_t)bytes;
    };
    alloc(reinterpret_cast<void **>(&ctx->W), sizeof(float) * (size_t)ctx->W_floats);
    alloc(reinterpret_cast<void **>(&ctx->band_done), sizeof(uint32_t) * 2 * kMaxBands);   // + claim counters
    alloc(reinterpret_cast<void **>(&ctx->status), sizeof(ptx::DevStatus));
    alloc(reinterpret_cast<void **>(&ctx->sfa), (size_t)ctx->sfa_bytes);
    alloc(reinterpret_cast<void **>(&ctx->sfb), (size_t)ctx->sfb_bytes);
    alloc(reinterpret_cast<void **>(&ctx->wire_q), (size_t)(max_M * N));
    alloc(reinterpret_cast<void **>(&ctx->wire_s), sizeof(float) * (size_t)max_M);
    alloc(reinterpret_cast<void **>(&ctx->counters), sizeof(uint32_t) * kCounters);
    if (rc == GEMMAR_OK && (cudaMemset(ctx->status, 0, sizeof(ptx::DevStatus)) != cudaSuccess ||
                            cudaMemset(ctx->counters, 0, sizeof(uint32_t) * kCounters) != cudaSuccess))
        rc = GEMMAR_ERR_CUDA;
    if (rc == GEMMAR_OK && !register_split_ok(256))
        rc = GEMMAR_ERR_DEVICE;
    if (rc == GEMMAR_OK && !(flags & GEMMAR_NO_SELF_TEST))
        rc = self_test(ctx);
    if (rc != GEMMAR_OK) {
        gemmar_destroy(ctx);
        return rc;
    }
    *out = ctx;
    return GEMMAR_OK;
}

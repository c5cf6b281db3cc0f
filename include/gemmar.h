/*
 * gemmar.h -- C ABI of libgemmar: the block-scaled fp8 GEMM and row-parallel
 * reduce of a DeepSeek-style attention block's output projection (wo_b),
 * run on one GB300 GPU (sm_103a).
 *
 * What the path computes (sources are web pages, cited by title and section):
 *   - wo_b is a row-parallel linear layer: a block-scale fp8 GEMM whose
 *     [M, hidden] result is all-reduced over the ranks that each hold one
 *     K-slice of the weight (sglang pull request #40757, "What").
 *   - Quantisation "blockscale": A (activations) with one fp32 scale per 1x128
 *     group along K, B (weight) with one fp32 scale per 128x128 block
 *     ("MORI GEMM + All-Reduce Benchmark", "Running the benchmark").
 *   - Quantisation "mxfp8": e4m3 with a ue8m0 power-of-two scale per 1x32 group,
 *     the exponent taken from the IEEE bits (sglang pull request #43480,
 *     "What" and review item 7 "Duplicated ue8m0 scale rule").
 *   - The reduce accumulates in fp32 and the output is bf16; the optional
 *     "fp8 wire" sends each output row as e4m3 with one fp32 scale
 *     ("MORI GEMM + All-Reduce Benchmark", "The fp8 wire").
 *   - The fused kernel writes each destination's row band as soon as that
 *     band's tiles are done (sglang pull request #40757, "What"; MORI page,
 *     "Where the time goes").
 *
 * On one GPU the P "ranks" are P K-slices resident in this GPU's memory; the
 * exchange is the band reduce reading their fp32 partials.  No collective runs.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller, row-major,
 *     contiguous, 16-byte aligned (else GEMMAR_ERR_ALIGN).  Sizes are element
 *     counts.  e4m3 tensors are uint8 codes (OCP E4M3FN); bf16 tensors are
 *     uint16 bit patterns.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; 0 = legacy
 *     default stream) and returns a host status at once.  Any status other
 *     than GEMMAR_OK returned by a call means nothing was launched, except
 *     GEMMAR_ERR_CUDA, which reports that a launch or CUDA call failed.
 *   - Device-side failures (a bounded wait that expired) are recorded in the
 *     context's device status word; gemmar_status() reads it after the work is
 *     complete and makes the context sticky-disabled: every later call
 *     returns GEMMAR_ERR_DISABLED.  No kernel traps, hangs or faults on
 *     purpose; every device wait has a time limit.
 *   - The context owns only its workspace (fp32 partials, band counters,
 *     scale repack area, fp8-wire staging) and status word.  The workspace is
 *     overwritten by the next call that uses it; calls on one context must be
 *     stream-ordered (the same stream, or joined by events).
 *   - The current CUDA device must be the context's device.
 */
#ifndef GEMMAR_H
#define GEMMAR_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemmar_ctx gemmar_ctx;

/* Status codes. */
enum {
    GEMMAR_OK = 0,
    GEMMAR_ERR_ARG = 1,        /* NULL pointer, bad enum value, negative or zero size */
    GEMMAR_ERR_SHAPE = 2,      /* shape the kernels cannot express (see gemmar_supports) */
    GEMMAR_ERR_ALIGN = 3,      /* a pointer is not 16-byte aligned */
    GEMMAR_ERR_WORKSPACE = 4,  /* call needs more workspace than gemmar_create sized */
    GEMMAR_ERR_CUDA = 5,       /* a CUDA runtime or driver call failed */
    GEMMAR_ERR_TIMEOUT = 6,    /* a device-side bounded wait expired (read by gemmar_status) */
    GEMMAR_ERR_DISABLED = 7,   /* context disabled by an earlier device-side failure */
    GEMMAR_ERR_DEVICE = 8      /* not an sm_103 device, wrong current device, or self-test mismatch */
};

/* Element types of an output or input matrix. */
enum { GEMMAR_DTYPE_F32 = 0, GEMMAR_DTYPE_BF16 = 1 };

/* Scale kinds. BLOCK128: fp32 A scales [M, K/128], fp32 B scales [N/128, K/128].
 * MX32: ue8m0 bytes (value 2^(byte-127)), A [M, K/32], B [N, K/32].
 * PTPC: fp32 per-token A scales [M] and per-channel B scales [N] (one scale
 * per row of A and of B over the whole K). */
enum { GEMMAR_SCALE_BLOCK128 = 0, GEMMAR_SCALE_MX32 = 1, GEMMAR_SCALE_PTPC = 2 };

/* Flags of gemmar_create and fused_gemm_reduce. */
#define GEMMAR_FP8_WIRE        (1u << 0)  /* fused: per-row e4m3 quantise + dequantise of the output */
#define GEMMAR_DEBUG_CANARY    (1u << 1)  /* fused: pre-fill partials and output with NaN */
#define GEMMAR_FAULT_SKIP_BAND (1u << 2)  /* fused, testing only: band 0 is never signalled, so the
                                             reducer's bounded wait expires (GEMMAR_ERR_TIMEOUT) */
#define GEMMAR_NO_SELF_TEST    (1u << 3)  /* create: skip the closed-form self-test */
#define GEMMAR_CTA_PAIR        (1u << 5)  /* create: run blockscale GEMMs with N % 256 == 0 on the CTA-pair
                                             kernel (256 x 256 tiles over two SMs; band partials parked in
                                             shared memory and copied out by two store warps) instead of
                                             the one-CTA kernel; the same bits (tests); on the wo_b band
                                             path its GEMM runs ~1810 us against ~1680 for the one-CTA
                                             kernel (both with the band reduce after the GEMM) */
#define GEMMAR_FUSE_SLICES     (1u << 4)  /* fused: each output tile accumulates all P slices itself (no
                                             partials, no band reduce); see fused_gemm_reduce */
#define GEMMAR_FUSE_ONCHIP     (1u << 6)  /* fused: the P slice partials of a tile stay on chip and are
                                             summed in the band reducer's order; bit-equal to the band
                                             path; see fused_gemm_reduce */
#define GEMMAR_SERIAL_REDUCE   (1u << 7)  /* fused band path: the GEMM kernel reduces no band while it
                                             runs; band_reduce sums every block after it (same bits) */
#define GEMMAR_FUSE_QUANTIZE   (1u << 8)  /* fused band path with GEMMAR_FP8_WIRE, N <= 12288: the band
                                             reduce quantises each row itself, without writing and
                                             re-reading the bf16 rows (same bits); ignored otherwise */

/* Largest number of K-slices ("ranks") one call takes. */
#define GEMMAR_MAX_P 8

/*
 * gemmar_supports -- can the kernels express this shape?  (The pages' op has
 * the same question answered by its supports(); sglang pull request #40757,
 * "Worth a reviewer's attention", last item.)  Rules:
 *   M >= 1; 1 <= P <= GEMMAR_MAX_P; 1 <= bands <= min(M, 1024) and M % bands == 0;
 *   BLOCK128: N % 128 == 0 (the B scale block); MX32: N % 128 == 0 or N % 224 == 0;
 *   PTPC: N % 128 == 0;
 *   K % 128 == 0 (every scale kind: one MMA stage is 128 of K);
 *   N <= 65536, K <= 65536, M <= 2^24.
 * Returns GEMMAR_OK or GEMMAR_ERR_SHAPE / GEMMAR_ERR_ARG.  Needs no GPU.
 */
int gemmar_supports(int P, int64_t M, int64_t N, int64_t K, int bands, int scale_kind);

/*
 * gemmar_create -- make a context on `device` (which must be current) whose
 * workspace serves fused_gemm_reduce calls with P <= max_P, M <= max_M and the
 * given N and K: fp32 partials of max_P*(max_M + 128*max_P)*N floats (a tile-
 * blocked layout; each band's rows are rounded up to whole 128-row tiles; at
 * least 256*max_M, the scratch of max_M tokens' adapters), band counters, the
 * mxfp8 scale repack area and the fp8-wire staging.  Like the pages' window
 * it is sized once and never grows (sglang pull request #40757, "Worth a
 * reviewer's attention": the window is sized from the chunked-prefill
 * ceiling, not from the first request).  wait_timeout_ns bounds every
 * device-side wait (0 = 2 s).  Unless GEMMAR_NO_SELF_TEST is set, runs the
 * fused path on a closed-form case (unit codes and scales: every output
 * equals P*K) for every scale kind, on the band path and with the partials
 * summed on chip, under that deadline, and fails with GEMMAR_ERR_DEVICE on a
 * mismatch (the pages' self_test(), sglang pull request #40757).
 * On success *out owns device memory until gemmar_destroy.
 */
int gemmar_create(gemmar_ctx **out, int device, int64_t max_M, int64_t N, int64_t K, int max_P,
                  uint32_t flags, int64_t wait_timeout_ns);

/* gemmar_destroy -- synchronise the context's device and free its workspace. */
int gemmar_destroy(gemmar_ctx *ctx);

/*
 * gemmar_status -- read (blocking) the device status word; call after the
 * work is complete.  Returns GEMMAR_OK or the first device-side error
 * (GEMMAR_ERR_TIMEOUT); *detail (if not NULL) receives where it happened
 * (see the kernels' wait-site codes).  A device error disables the context.
 */
int gemmar_status(gemmar_ctx *ctx, int *detail);

/* gemmar_workspace_bytes -- device bytes the context holds. */
int64_t gemmar_workspace_bytes(const gemmar_ctx *ctx);

/*
 * Phase timing of fused_gemm_reduce, the per-layer breakdown of the MORI
 * page's "Where the time goes" table.  gemmar_set_phase_timing(ctx, 1) makes
 * every later fused call record CUDA events on its stream between its kernel
 * launches (nothing is skipped or reordered).  gemmar_phase_times waits for
 * those events, writes the summed milliseconds of each phase over the
 * recorded calls into ms[GEMMAR_NUM_PHASES] and the number of calls into
 * *calls, and clears the record.  Phases: GEMMAR_PHASE_GEMM (scale repack,
 * GEMM with band-ordered partial stores), GEMMAR_PHASE_REDUCE (band_reduce),
 * GEMMAR_PHASE_QUANTIZE and GEMMAR_PHASE_DEQUANTIZE (the fp8 wire; 0 when off;
 * with GEMMAR_FUSE_QUANTIZE the quantiser runs inside GEMMAR_PHASE_REDUCE).  On
 * the band path with the in-kernel reduce, GEMMAR_PHASE_GEMM includes the blocks
 * the GEMM kernel summed (gemmar_overlap_stats) and GEMMAR_PHASE_REDUCE the rest.
 * At most 65536 calls are recorded between reads (later ones are not timed).
 */
enum { GEMMAR_PHASE_GEMM = 0, GEMMAR_PHASE_REDUCE = 1, GEMMAR_PHASE_QUANTIZE = 2,
       GEMMAR_PHASE_DEQUANTIZE = 3, GEMMAR_NUM_PHASES = 4 };
int gemmar_set_phase_timing(gemmar_ctx *ctx, int enable);
int gemmar_phase_times(gemmar_ctx *ctx, float *ms, int *calls);

/*
 * gemmar_overlap_stats -- of the last fused_gemm_reduce band-path call on this
 * context, *total = its 32-row x 32-column output blocks and *overlapped = how
 * many of them the GEMM kernel's reducer warps summed while the GEMM was still
 * running (the rest were summed by band_reduce after it).  Both 0 when the last
 * fused call did not take the band path, or took it without the in-kernel
 * reduce (GEMMAR_SERIAL_REDUCE, or the CTA-pair kernel).  Reads device
 * memory with a synchronous copy: call after that call's work has completed.
 */
int gemmar_overlap_stats(gemmar_ctx *ctx, int64_t *overlapped, int64_t *total);

/*
 * gemm_blockscale_fp8 -- C[M,N] = A[M,K] * B[N,K]^T for one K-slice, with
 *   C[m,n] = sum_kb (sa[m,kb]*sb[n/128,kb]) * sum_{k in kb} a[m,k]*b[n,k]
 * accumulated in fp32 (tcgen05 MMA per 128-K block into TMEM, the scales
 * applied while draining TMEM).  Blockscale quantisation as on the MORI page
 * ("Running the benchmark": A 1x128, B 128x128, fp32 scales).
 *   A: e4m3 [M,K]; sa: fp32 [M, K/128]; B: e4m3 [N,K]; sb: fp32 [N/128, K/128];
 *   C: [M,N] of c_dtype (GEMMAR_DTYPE_F32 or GEMMAR_DTYPE_BF16, RNE).
 * Shape rules as gemmar_supports with P = bands = 1.
 */
int gemm_blockscale_fp8(gemmar_ctx *ctx, const uint8_t *A, const float *sa, const uint8_t *B,
                        const float *sb, void *C, int c_dtype, int64_t M, int64_t N, int64_t K,
                        void *stream);

/*
 * gemm_ptpc_fp8 -- C[M,N] = (sa[m]*sb[n]) * sum_k a[m,k]*b[n,k] for one K-slice:
 * the "ptpc" quantisation the MORI benchmark runs by default ("Negative
 * results", the paragraph on pinning `--quant`), read as per-token A scales and
 * per-output-channel B scales.  The MMA accumulates the whole K in TMEM (no
 * promotion); the epilogue multiplies by the fp32 product sa[m]*sb[n].
 *   A: e4m3 [M,K]; sa: fp32 [M]; B: e4m3 [N,K]; sb: fp32 [N];
 *   C: [M,N] of c_dtype.  Shape rules as gemmar_supports with P = bands = 1.
 */
int gemm_ptpc_fp8(gemmar_ctx *ctx, const uint8_t *A, const float *sa, const uint8_t *B,
                  const float *sb, void *C, int c_dtype, int64_t M, int64_t N, int64_t K,
                  void *stream);

/*
 * gemm_mxfp8 -- C[M,N] = sum_g 2^(ea[m,g]+eb[n,g]-254) * sum_{k in g} a[m,k]*b[n,k]
 * for one K-slice, on the native block-scaled MMA (tcgen05 kind::mxf8f6f4,
 * one ue8m0 scale per 32 of K); the mxfp8 wo_b of sglang pull request #43480.
 *   A: e4m3 [M,K]; ea: ue8m0 bytes [M, K/32]; B: e4m3 [N,K]; eb: [N, K/32];
 *   C: [M,N] of c_dtype.  Uses the context's repack area (needs M <= max_M,
 *   N and K <= those of gemmar_create, else GEMMAR_ERR_WORKSPACE).
 */
int gemm_mxfp8(gemmar_ctx *ctx, const uint8_t *A, const uint8_t *ea, const uint8_t *B,
               const uint8_t *eb, void *C, int c_dtype, int64_t M, int64_t N, int64_t K,
               void *stream);

/*
 * band_reduce -- the fixed-order reduce of the row-parallel layer: for band
 * b (rows b*M/bands .. (b+1)*M/bands-1),
 *   out[m,n] = bf16_rn( ((W[b][0][r][n] + W[b][1][r][n]) + ...) + W[b][P-1][r][n] )
 * in fp32, p ascending ("MORI GEMM + All-Reduce Benchmark", "The fp8 wire":
 * the reduce accumulates in fp32; "Negative results": the reduce streams
 * through all source slices at once).  Bit-exact and deterministic.
 *   W: fp32 [bands][P][M/bands][N] (caller-owned); out: bf16 [M,N].
 */
int band_reduce(gemmar_ctx *ctx, const float *W, int P, int64_t M, int64_t N, int bands,
                uint16_t *out, void *stream);

/*
 * rowquant_e4m3 -- the fp8 wire's narrowing: per row m of x [M,N],
 *   s[m] = fp32(amax_n |x[m,n]| / 448),  q[m,n] = e4m3_rn_sat(fp32(x[m,n] / s[m]))
 * (IEEE division; a zero row gives s = 0 and +0 codes).  One fp32 scale per
 * row ("MORI GEMM + All-Reduce Benchmark", "The fp8 wire"; sglang pull
 * request #40757, "The optional fp8 gather").  Non-finite inputs: the amax
 * skips NaN (a row of NaN alone is a zero row; a NaN value codes to NaN); an
 * infinite value makes s infinite, so finite values code to +-0 and
 * infinities to NaN.
 *   x: [M,N] of x_dtype (GEMMAR_DTYPE_BF16 or GEMMAR_DTYPE_F32); q: uint8 [M,N];
 *   row_scale: fp32 [M].  N % 16 == 0.  Bit-exact against the definition.
 */
int rowquant_e4m3(gemmar_ctx *ctx, const void *x, int x_dtype, int64_t M, int64_t N,
                  uint8_t *q, float *row_scale, void *stream);

/*
 * rowdequant_e4m3 -- the fp8 wire's widening: y[m,n] = bf16_rn(fp32(decode(q[m,n]) * s[m]))
 * ("MORI GEMM + All-Reduce Benchmark", "Who moves the gather": the second
 * kernel that widens the landed fp8).
 *   q: uint8 [M,N]; row_scale: fp32 [M]; y: bf16 [M,N].  N % 16 == 0.
 */
int rowdequant_e4m3(gemmar_ctx *ctx, const uint8_t *q, const float *row_scale, int64_t M,
                    int64_t N, uint16_t *y, void *stream);

/*
 * quant_blockscale_e4m3 -- device quantiser for blockscale operands: groups
 * of group_rows x 128 (group_rows 1 for activations, 128 for weights) of an
 * [R,C] matrix x of x_dtype (GEMMAR_DTYPE_BF16 or GEMMAR_DTYPE_F32; bf16 is
 * widened to fp32 exactly); s = fp32(amax/448), q = e4m3_rn_sat(fp32(x/s));
 * a zero group gives s = 0 and +0 codes; non-finite values as in
 * rowquant_e4m3, per group.  The real call site quantises wo_b's
 * bf16 input itself (sglang pull request #43480, "Numerics, measured where
 * the path engages"), so bf16 is the input the layer sees.
 * q: uint8 [R,C]; scales: fp32 [ceil(R/group_rows), C/128].
 * C % 128 == 0.  Bit-exact against the definition.
 */
int quant_blockscale_e4m3(gemmar_ctx *ctx, const void *x, int x_dtype, int64_t R, int64_t C, int group_rows,
                          uint8_t *q, float *scales, void *stream);

/*
 * quant_mx_e4m3 -- device mxfp8 quantiser: per 1x32 group of an [R,C] matrix x
 * of x_dtype (GEMMAR_DTYPE_BF16 or GEMMAR_DTYPE_F32), byte =
 * ceil(log2(fp32(amax/448))) + 127 from the IEEE bits (exact at powers of two;
 * sglang pull request #43480, review item 7), clamped to [0,254], 0 for a
 * zero group; q = e4m3_rn_sat(fp32(x * 2^(127-byte))).  The amax skips NaN; an
 * infinite value gives byte 254, finite values then code to +-0 and
 * infinities saturate to +-448.
 * q: uint8 [R,C]; e8m0: uint8 [R, C/32].  C % 32 == 0.  Bit-exact.
 */
int quant_mx_e4m3(gemmar_ctx *ctx, const void *x, int x_dtype, int64_t R, int64_t C, uint8_t *q,
                  uint8_t *e8m0, void *stream);

/*
 * fused_gemm_reduce -- the whole wo_b path for P K-slices resident on this
 * GPU: one persistent GEMM launch over every (band, slice, tile) in band
 * order that stores each tile's fp32 partial into the context's workspace
 * W[band][p] and signals that band's counter as soon as the tile retires
 * (sglang pull request #40757, "What": the fused kernel hands each row band
 * over as soon as that band's tiles are done).  Two reducer warps of
 * every GEMM CTA take 32 x 32 output blocks of the bands already complete and
 * sum them while the GEMM still runs (the hand-over overlapped with the
 * compute, as the pages overlap their scatter with it; not on the CTA-pair
 * kernel, whose shared memory holds no room for it); band_reduce then waits
 * (bounded) for each band's counter and sums the P partials of the remaining
 * blocks in the same fixed order to bf16 out [M,N].  With GEMMAR_FP8_WIRE the
 * reduced rows then go through rowquant_e4m3 + rowdequant_e4m3 ("The fp8
 * wire"); with GEMMAR_FUSE_QUANTIZE as well (N <= 12288), the band reduce
 * parks each group of 8 summed bf16 rows in shared memory, takes their amax
 * and writes their codes and scales itself (MORI page, "Negative results":
 * folding the narrowing into the reduce), so the rows it sums are neither
 * written as bf16 nor read back before rowdequant_e4m3; the output is
 * bit-equal to the unfolded wire.
 *   A[p], B[p], sa[p], sb[p]: HOST arrays of P device pointers; per slice as in
 *   gemm_blockscale_fp8 (scale_kind GEMMAR_SCALE_BLOCK128) or gemm_mxfp8
 *   (GEMMAR_SCALE_MX32).  bands: row bands (0 = P).  out: bf16 [M,N].
 * Deterministic: equal, bit for bit, to P x gemm_*(F32) into W followed by
 * band_reduce, and to itself on a rerun.
 *
 * With GEMMAR_FUSE_SLICES the slices are instead summed inside each output
 * tile: one fp32 accumulation chain per output element over (p, K-block) in
 * the fixed order p = 0..P-1, K ascending, rounded once to bf16.  Nothing is
 * stored between the slices, so the partial write and the band reduce
 * (2 x P*M*N*4 bytes) disappear; the result is deterministic and within the
 * same tolerance of the definition, but its fp32 rounding order differs from
 * the band path's, so the two are not bit-equal.  bands is then ignored
 * (it must still satisfy the shape rules).
 *
 * With GEMMAR_FUSE_ONCHIP each output tile computes the P slice partials one
 * after another, each exactly as the band path computes it (fp32, its own
 * K-blocks from zero), and sums them in the band reducer's order, ((W_0 +
 * W_1) + W_2) + ..., in fp32 before the single bf16 rounding, without the
 * 2 x P*M*N*4 bytes of partial traffic.  Blockscale (N % 256 == 0, a GPU that
 * runs CTA pairs) runs on the CTA-pair kernel, the running sum in shared
 * memory: bit-equal to the band path, of the default one-CTA kernel as of a
 * GEMMAR_CTA_PAIR context (the two kernels give the same bits).  mx and
 * ptpc run on the whole-K kernel, each slice accumulating in a TMEM buffer of
 * its own (ptpc: then scaled) and the running sum in registers: bit-equal to
 * their band path.  Other blockscale shapes take the band path.  Takes
 * precedence over GEMMAR_FUSE_SLICES, which for ptpc means the same as
 * GEMMAR_FUSE_ONCHIP (its scales apply after a slice's whole K, so no single
 * chain over the slices exists).
 */
int fused_gemm_reduce(gemmar_ctx *ctx, int P, const uint8_t *const *A, const void *const *sa,
                      const uint8_t *const *B, const void *const *sb, int scale_kind,
                      int64_t M, int64_t N, int64_t K, int bands, uint32_t flags,
                      uint16_t *out, void *stream);

/*
 * fused_gemm_reduce_noalloc -- the blockscale fused_gemm_reduce for callers
 * that cannot allocate device memory.  The pages have no counterpart; it is
 * an addition of this library.
 *
 * Who needs it: an inference engine that takes all of the GPU's memory for
 * its own pool at start-up and allows no cudaMalloc afterwards (a late
 * allocation would fail or split its arena), or a host application that
 * loads this library as a plugin and wants every device byte to come from its
 * own allocator.  Neither can call gemmar_create, which allocates.  This call
 * takes no context and allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library routine): its scratch -- fp32 partials for up to
 * GEMMAR_NOALLOC_MAX_PARTIALS elements (P*M*N, each band's rows rounded up to
 * whole 128-row tiles), 1024 band counters, 1024 claim counters for the
 * GEMM's in-kernel band reduce and a status word -- lives in fixed-size arrays
 * in the library's device code, which the CUDA driver reserves on every GPU
 * that loads the library (32 MiB plus a few KiB per GPU) and keeps until the
 * process exits.
 *
 * Arguments as fused_gemm_reduce with scale_kind GEMMAR_SCALE_BLOCK128 and no
 * flags: A, sa, B, sb are HOST arrays of P device pointers, out is bf16 [M,N]
 * on the current device, bands 0 means P.  Returns GEMMAR_ERR_WORKSPACE when
 * that padded P*M*N exceeds GEMMAR_NOALLOC_MAX_PARTIALS (use fused_gemm_reduce
 * then), and
 * the other codes as fused_gemm_reduce.  The result equals fused_gemm_reduce's
 * bit for bit (same kernels, same fixed-order reduce).
 *
 * The first call on a device looks up the scratch's device addresses (and the
 * driver loads the device code there); make that first call before any
 * stream capture.  Every call on a device shares the one scratch, which keeps
 * the last call's contents; the call clears its counters and status word
 * itself.  Calls whose work overlaps on the GPU (different streams without an
 * ordering between them, or several host threads) race on the scratch and
 * give wrong results: keep them stream-ordered.
 *
 * Device-side failures: every wait inside the kernels is bounded (2 s).  If
 * one expires -- for instance a GEMM CTA whose operand loads or tensor-core
 * work stall that long on a GPU shared with other work -- the kernels stop
 * early, the call has still returned GEMMAR_OK (it returns before the work
 * runs), and `out` is left incomplete.  The failure is recorded in the
 * scratch's status word: read it with fused_gemm_reduce_noalloc_status after
 * the call's work has completed, before the next call on that device clears
 * it.
 */
#define GEMMAR_NOALLOC_MAX_PARTIALS (8 * 1024 * 1024)
int fused_gemm_reduce_noalloc(int P, const uint8_t *const *A, const float *const *sa,
                              const uint8_t *const *B, const float *const *sb,
                              int64_t M, int64_t N, int64_t K, int bands, uint16_t *out, void *stream);

/*
 * fused_gemm_reduce_noalloc_status -- the device status of the last
 * fused_gemm_reduce_noalloc call on the current device: GEMMAR_OK, or
 * GEMMAR_ERR_TIMEOUT when a bounded wait of its kernels expired (then its
 * `out` is incomplete), with *detail (if not NULL) set to the wait site.
 * Reads the 8-byte status word with a synchronous device-to-host copy (no
 * allocation): call it after that call's work has completed (for example
 * after synchronising its stream).  GEMMAR_ERR_DEVICE if the current device
 * has made no such call yet.  The pages have no counterpart.
 */
int fused_gemm_reduce_noalloc_status(int *detail);

/*
 * ---- The residual stream after wo_b -----------------------------------------
 *
 * The pages end at wo_b's bf16 rows; the operators from here on are additions
 * of this library: what a transformer block does to those rows next (norms,
 * gate and residual, codes for the next block-scaled GEMM), and the low-rank
 * adapters that requests bring beside the shared projection.
 *
 * Their matrices may be views: a row stride (in elements) follows each pointer
 * that has one, stride * element size a multiple of 16 bytes (else
 * GEMMAR_ERR_ALIGN), 0 for one row read for all rows.  Everything else is
 * contiguous.  They use the context's partial-sum workspace as scratch
 * (GEMMAR_ERR_WORKSPACE when it is too small), so the rule on stream order above
 * holds.  Calls of at most max_M rows or tokens always fit (norms: rows of at most
 * N columns).  For more, in floats: norm_gate_residual none, its gradients at most
 * (M + 1) N; lora_apply T r', or none where it takes one launch; lora_apply_bwd
 * 2 T r', r' being r rounded up to 16, 32, 64 or 128.  lora_apply_bwd shares out the
 * tokens of a large adapter as finely as what is left allows: a context of few
 * columns makes it slower.
 */

/* Widest row and smallest column granule of norm_gate_residual. */
#define GEMMAR_NORM_MAX_N 16384

/*
 * norm_gate_residual -- a block's output y joins the residual stream h, and the
 * next block's input is formed from the sum; per row, with w1 = w_post,
 * w2 = w_pre and the gate g,
 *   r1 = 1 / sqrt(mean(y^2) + eps),  z = y * r1 * w1     (w_post NULL: z = y, r1 = 1)
 *   t  = alpha * h + beta * g * z                        (gate NULL: g = 1)
 *   r2 = 1 / sqrt(mean(t^2) + eps),  x = t * r2 * w2     (w_pre NULL: t only)
 * t goes out in h's type, x as bf16 rows u and/or as the A operand of
 * gemm_blockscale_fp8: e4m3 codes q [M,N] with fp32 scales [M, N/128], by the rule
 * of quant_blockscale_e4m3 applied to the fp32 x (not to its bf16 rounding).
 * All arithmetic is fp32 and every output is rounded once; x is formed from the
 * fp32 t, not from its rounding to h's type.  Rows are independent: a row with a
 * NaN or an infinity leaves the others alone.  Where a row's sum of squares passes
 * fp32's range (a root mean square above 1.8e19 / sqrt(N)) its r is 0; squares below
 * 1e-38 lose digits and vanish.
 *   y [M,N] of y_dtype, h [M,N] of h_dtype (GEMMAR_DTYPE_F32 or _BF16), row
 *   strides y_stride, h_stride; w_post, w_pre fp32 [N] or NULL; gate bf16:
 *   gate_stride 0 is one row [N] for every row, else [M,N].
 *   t [M,N] of h_dtype (may be h itself when h is contiguous); u bf16 [M,N], q,
 *   scales, rstd fp32 [M,2] (r1, r2; r2 is 1 without w_pre): NULL to leave out.
 *   u may be y itself when y is contiguous bf16.
 * N % 8 == 0, N <= GEMMAR_NORM_MAX_N; with q N % 128 == 0 (else
 * GEMMAR_ERR_SHAPE).  eps >= 0, alpha, beta and eps finite.
 */
int norm_gate_residual(gemmar_ctx *ctx, const void *y, int y_dtype, int64_t y_stride,
                       const void *h, int h_dtype, int64_t h_stride,
                       const float *w_post, const float *w_pre, const uint16_t *gate, int64_t gate_stride,
                       float alpha, float beta, float eps, int64_t M, int64_t N,
                       void *t, uint16_t *u, uint8_t *q, float *scales, float *rstd, void *stream);

/*
 * norm_gate_residual_bwd -- its gradients, from dt (of t, type h_dtype; NULL: 0) and
 * du (of x, bf16; required with w_pre, else ignored), given the forward pass's y,
 * h and rstd; t is recomputed in fp32.  With n = y r1 and that = t r2:
 *   d    = dt + r2 (du w2 - that mean(du w2 that))      (w_pre NULL: d = dt)
 *   dh   = alpha d,   e = beta g d w1
 *   dy   = r1 (e - n mean(e n))                         (w_post NULL: dy = beta g d)
 *   dw_pre = sum_rows du that,   dw_post = sum_rows beta g d n
 *   dgate  = beta n w1 d per token (bf16 [M,N]), or its sum over the rows when
 *            the gate is one row (fp32 [N])
 * dy [M,N] has y_dtype, dh [M,N] h_dtype (may be dt itself when dt is contiguous);
 * dw_post, dw_pre fp32 [N] are overwritten and NULL leaves one out; dgate NULL
 * likewise.  The sums over rows run in fp32 in an order fixed by M, N and the GPU:
 * two calls give the same bits.
 */
int norm_gate_residual_bwd(gemmar_ctx *ctx, const void *y, int y_dtype, int64_t y_stride,
                           const void *h, int h_dtype, int64_t h_stride, const float *rstd,
                           const float *w_post, const float *w_pre, const uint16_t *gate, int64_t gate_stride,
                           float alpha, float beta, int64_t M, int64_t N,
                           const void *dt, int64_t dt_stride, const uint16_t *du, int64_t du_stride,
                           void *dy, void *dh, float *dw_post, float *dw_pre, void *dgate, void *stream);

/* Limits of the adapters: how many one call takes, and their largest rank. */
#define GEMMAR_LORA_MAX_ADAPTERS 1024
#define GEMMAR_LORA_MAX_RANK 128

/*
 * lora_plan -- the tokens of a batch in the order of their adapters: order[T] holds
 * the tokens of adapter 0 in ascending order, then those of adapter 1, ..., then
 * those without one (an id outside [0, R)); adapter a's are
 * order[offsets[a] .. offsets[a+1]).  One batch's plan serves every layer.
 *   adapter_ids int32 [T]; order int32 [T]; offsets int32 [R+1].
 * 1 <= R <= GEMMAR_LORA_MAX_ADAPTERS, T <= 2^24.
 */
int lora_plan(gemmar_ctx *ctx, const int32_t *adapter_ids, int64_t T, int R, int32_t *order, int32_t *offsets,
              void *stream);

/*
 * lora_apply -- low-rank adapters of many requests beside a shared projection: for
 * token t with adapter a,
 *   v[t,j]   = sum_k x[t,k] A[a,j,k]
 *   out[t,n] = y[t,n] + scales[a] sum_{j < ranks[a]} v[t,j] B[a,j,n]
 * and out[t] = y[t] for a token without one.  Both factors are stored rank-major
 * (B is the transpose of an [N, r] up-projection), so a rank of any size keeps its
 * rows on 16 bytes.  v is fp32 and enters the second product as two bf16 parts
 * (its rounding error is below 2^-16; an infinite v keeps its sign); out is rounded
 * once.  An infinite element of B makes its column of out NaN or infinite: its
 * products with the two parts may cancel.
 *   x bf16 [T,K], y bf16 [T,N] (NULL: 0) and out bf16 [T,N] with row strides; y may
 *   be out itself, at the same stride.  order, offsets: lora_plan's form (entries outside [0,T) are
 *   skipped).  A bf16 [R,r,K], B bf16 [R,r,N], scales fp32 [R], ranks int32 [R] (NULL:
 *   r for all; rows beyond ranks[a] are not used).  v: NULL, or fp32 [T,r] for the
 *   backward pass: row i belongs to token order[i]; rows past offsets[R] are left
 *   alone, columns past ranks[a] are 0.
 * K % 8 == 0, N % 8 == 0 (else GEMMAR_ERR_SHAPE), K, N <= 65536, T <= 2^24,
 * 1 <= r <= GEMMAR_LORA_MAX_RANK.
 */
int lora_apply(gemmar_ctx *ctx, const uint16_t *x, int64_t x_stride, const int32_t *order, const int32_t *offsets,
               const uint16_t *A, const uint16_t *B, const float *scales, const int32_t *ranks,
               int64_t T, int64_t K, int64_t N, int R, int r, const uint16_t *y, int64_t y_stride,
               uint16_t *out, int64_t out_stride, float *v, void *stream);

/*
 * lora_apply_bwd -- its gradients, from dy (of out) and the forward pass's x and v:
 *   w[t,j]    = scales[a] sum_n dy[t,n] B[a,j,n]
 *   dx[t,k]   = dx0[t,k] + sum_{j < ranks[a]} w[t,j] A[a,j,k]   (dx0[t] for a token without one)
 *   dA[a,j,k] = sum_{t of a} w[t,j] x[t,k],   dB[a,j,n] = scales[a] sum_{t of a} v[t,j] dy[t,n]
 * (the gradient of y is dy itself).  dx0 bf16 [T,K] (NULL: 0; may be dx itself) and
 * dx bf16 [T,K] with row strides; dA, dB bf16, of A's and B's shapes, overwritten:
 * 0 for an adapter without tokens and for rows past ranks[a].  Sums are fp32 in a
 * fixed order, rounded once.  w and v enter the second products as v does in
 * lora_apply.  dx lies apart from x, dy, A and B, and dA and dB apart from
 * each other and from A and B: one is written while others are read.  GEMMAR_ERR_ARG where
 * dA or dB does not, or dx starts where x or dy does or, at the same stride, shares elements.
 * Other arguments and limits as lora_apply.
 */
int lora_apply_bwd(gemmar_ctx *ctx, const uint16_t *x, int64_t x_stride, const uint16_t *dy, int64_t dy_stride,
                   const int32_t *order, const int32_t *offsets, const uint16_t *A, const uint16_t *B,
                   const float *scales, const int32_t *ranks, const float *v,
                   int64_t T, int64_t K, int64_t N, int R, int r, const uint16_t *dx0, int64_t dx0_stride,
                   uint16_t *dx, int64_t dx_stride, uint16_t *dA, uint16_t *dB, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMMAR_H */

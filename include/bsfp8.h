/*
 * bsfp8.h -- block-scaled FP8 / MXFP4 quantisation and GEMM on AMD MI355X (gfx950).
 *
 * A small C ABI over hand-written HIP kernels.  Every pointer argument is a
 * DEVICE pointer owned by the caller; the library never allocates or frees
 * device memory and never synchronises (adamw_step takes host memory during the
 * call to check more than about 64 tensors).  Every call is asynchronous on `stream` (0 = the null stream).
 * All argument checks run on the host before anything is launched: a call
 * that returns a status other than BSFP8_OK has launched nothing.  After a
 * launch the HIP launch error, if any, is returned as BSFP8_ERR_HIP.  No
 * global state: calls are thread-safe; calls that write the same output
 * buffer concurrently race.
 *
 * Pages cited (by title and section):
 *   [CDNA4-FP8] "Why grind FP8 GEMM on CDNA4" (dpshk.com article)
 *   [RUBIN-FP4] "Rubin FP4 GEMM deep dive: from Blackwell to the next GPU"
 *   [HOPPER-MMA] "FP8 MMA internals on Hopper"
 *
 * Layout conventions ([CDNA4-FP8] section 3.1, [RUBIN-FP4] section 3.1):
 * A is M x K row-major (K contiguous); B is K x N column-major, i.e. stored as
 * N rows of K contiguous elements; D is M x N row-major with leading
 * dimension ldd (elements).  A "K block" is 32 consecutive K indices.
 */
#ifndef BSFP8_H
#define BSFP8_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same typedef as the HIP runtime's; repeating it is harmless. */
typedef struct ihipStream_t* hipStream_t;

typedef enum {
    BSFP8_OK = 0,
    BSFP8_ERR_INVALID_ARG = 1,  /* null pointer, negative size, K not a multiple of 32, ld < k, ... */
    BSFP8_ERR_UNSUPPORTED = 2,  /* undefined enum value or format mix, tile_rows != 128 */
    BSFP8_ERR_HIP = 3,          /* the HIP runtime reported a launch error */
    BSFP8_ERR_NO_MEMORY = 4     /* no host memory for a call's check (adamw_step) */
} bsfp8_status;

typedef enum {
    BSFP8_E4M3 = 0,   /* OCP E4M3 ("FN"): max 448, no infinity */
    BSFP8_E5M2 = 1,   /* OCP E5M2: max 57344 */
    BSFP8_MXFP4 = 2   /* E2M1 elements, two per byte, E8M0 scale per 32-element K block */
} bsfp8_format;

typedef enum {
    BSFP8_OUT_F32 = 0,
    BSFP8_OUT_BF16 = 1,
    BSFP8_OUT_F16 = 2   /* IEEE binary16, round to nearest even, overflow to +-inf */
} bsfp8_out;

/*
 * fp8_quantize -- per-tile FP8 quantisation ([CDNA4-FP8] sections 3.3 and 4.2).
 *
 * x:      rows x k FP32, row-major, leading dimension ld (elements).
 *         16-byte aligned, ld a multiple of 4, ld >= k.
 * rows:   >= 0, any value; the last tile may have fewer than tile_rows rows.
 * k:      >= 0, a multiple of 32.
 * tile_rows: rows per scale tile; must be 128 (tiles are 128 x 32).
 * fmt:    BSFP8_E4M3 (F = 448) or BSFP8_E5M2 (F = 57344).
 * codes:  out, rows x k bytes, row stride k, 16-byte aligned.
 * scales: out, FP32 [ceil(rows / 128)][k / 32], K-block index fastest.
 *
 * Per tile: amax = max |x|, s = amax / F rounded to FP32 (s = 1 when that is
 * zero), code = saturating round-to-nearest-even of (x / s rounded to FP32).
 * Output is bit-exact: the same bytes on every call and every launch shape.
 * Finite inputs only.  A B operand (K x N column-major) is quantised by
 * passing its N x K storage: rows = N, k = K, giving the 32 x 128 (K x N)
 * tiles of the pages.
 */
bsfp8_status fp8_quantize(const float* x, int64_t rows, int64_t k, int64_t ld, int tile_rows,
                          bsfp8_format fmt, uint8_t* codes, float* scales, hipStream_t stream);

/*
 * fp8_quantize_pair -- fp8_quantize of the two operands of one GEMM, A
 * (a_rows x k) and B (b_rows x k, N x K storage), in a single launch
 * ([CDNA4-FP8] sections 3.3 and 4.2; 128 x 32 tiles as fp8_quantize).
 *
 * Each operand takes the arguments, layout, alignment and ownership rules of
 * fp8_quantize for its side (x, ld, fmt, codes, scales), with one shared k.
 * The outputs are byte-for-byte those of two fp8_quantize calls.  Either side
 * may have 0 rows (its pointers are then ignored).  Errors as fp8_quantize;
 * nothing is launched unless both sides pass the checks.  The two sides'
 * buffers must not overlap.
 */
bsfp8_status fp8_quantize_pair(const float* a, int64_t a_rows, int64_t a_ld, bsfp8_format a_fmt,
                               uint8_t* a_codes, float* a_scales, const float* b, int64_t b_rows,
                               int64_t b_ld, bsfp8_format b_fmt, uint8_t* b_codes, float* b_scales,
                               int64_t k, hipStream_t stream);

/*
 * fp8_quantize_transposed -- per-tile FP8 quantisation of x^T, for operands
 * stored the other way round, such as the gradient G and activation X of a
 * weight-gradient product dW = G^T X ([CDNA4-FP8] section 3.3's per-tile
 * scales; section 2.2 of the same page puts gradients in E5M2).
 *
 * x:      k x rows FP32, row-major, leading dimension ld (elements):
 *         16-byte aligned, ld a multiple of 4, ld >= rows.
 * k:      >= 0, a multiple of 32 (the K dimension of the GEMM operand).
 * rows:   >= 0, any value (M for an A operand, N for a B operand).
 * tile_rows, fmt: as for fp8_quantize.
 * codes:  out, rows x k bytes, row stride k, 16-byte aligned.
 * scales: out, FP32 [ceil(rows / 128)][k / 32].
 *
 * The result is byte-for-byte that of fp8_quantize applied to an explicitly
 * transposed copy of x (rows x k, row-major); no transposed copy is made.
 */
bsfp8_status fp8_quantize_transposed(const float* x, int64_t k, int64_t rows, int64_t ld,
                                     int tile_rows, bsfp8_format fmt, uint8_t* codes,
                                     float* scales, hipStream_t stream);

/*
 * mxfp4_quantize -- MXFP4 block quantisation ([RUBIN-FP4] sections 2.1, 2.2, 3.1, 4.2).
 *
 * x:      rows x k FP32, row-major, leading dimension ld; 16-byte aligned,
 *         ld a multiple of 4, ld >= k.  rows >= 0; k >= 0, a multiple of 32.
 * packed: out, rows x (k / 2) bytes, row stride k / 2.  Element 2i sits in the
 *         low nibble of byte i, element 2i+1 in the high nibble.
 * scales: out, E8M0 bytes [rows][k / 32].
 *
 * Per 32-element block of a row: e = the smallest integer with 6 * 2^e >= amax
 * (e = 0 when amax is 0), clamped to [-127, 127]; scale byte = e + 127;
 * element code = round-to-nearest-even E2M1 of x * 2^-e (exact scaling).
 * Bit-exact.  Finite inputs only.
 */
bsfp8_status mxfp4_quantize(const float* x, int64_t rows, int64_t k, int64_t ld,
                            uint8_t* packed, uint8_t* scales, hipStream_t stream);

/*
 * scaled_gemm -- D = deq(A) * deq(B) with FP32 accumulation
 * ([CDNA4-FP8] sections 2.3, 3.2-3.4, 4.3, 4.4; [RUBIN-FP4] sections 2.2, 3.1-3.3).
 *
 * M, N >= 0 (any value; edge tiles are masked), K >= 0 a multiple of 32.
 * FP8 operands (a_fmt, b_fmt each BSFP8_E4M3 or BSFP8_E5M2, any mix):
 *   a: M x K codes (row stride K); a_scales: FP32 [ceil(M/128)][K/32]
 *   b: N x K codes (row stride K); b_scales: FP32 [ceil(N/128)][K/32]
 *   exactly the outputs of fp8_quantize with tile_rows = 128.
 *   Each 32-wide K block's partial product is scaled by
 *   a_scale(tile, block) * b_scale(tile, block) before it is accumulated.
 * MXFP4 operands (a_fmt = b_fmt = BSFP8_MXFP4):
 *   a: M x K/2 packed bytes; a_scales: E8M0 [M][K/32]
 *   b: N x K/2 packed bytes; b_scales: E8M0 [N][K/32]
 *   (the outputs of mxfp4_quantize).
 * out:  BSFP8_OUT_F32, BSFP8_OUT_BF16 or BSFP8_OUT_F16 (the last two round
 *       to nearest even; [CDNA4-FP8] section 4.4 writes 16-bit results to halve
 *       the output traffic).
 * d:    M x N row-major, leading dimension ldd >= N (elements), aligned to
 *       its element size.
 * a, b must be 16-byte aligned.  K = 0 writes zeros.  FP8 operands need
 * K < 2^24 (the kernel addresses a 128-row band of an operand with 32-bit
 * offsets) and MXFP4 operands K < 2^26 (a 32-row band); larger K returns
 * BSFP8_ERR_UNSUPPORTED.  M and N are limited only
 * by the 2^31 - 1 bound on each dimension and on the number of 128 x 128 tiles.
 *
 * Accuracy: with S = sum_k |a_k b_k| (dequantised operands), every output
 * satisfies |D - exact| <= 2^-19 S for FP32 output and <= 2^-7 S for bf16 and
 * FP16 output on the synthetic workloads the library is tested on.  The FP8
 * matrix instructions used for 16-bit outputs align each group of 8 products
 * to 13 fraction bits below the group's largest exponent and cut the rest
 * (the truncation studied for Hopper in [HOPPER-MMA] is present on gfx950
 * too): at most 7 * 2^-13 S per 32-element block.  FP32 output widens the
 * codes to bf16 and uses instructions that keep 24 fraction bits: about
 * 2^-20.4 S per block, plus one FP32 rounding per block of the accumulation.
 */
bsfp8_status scaled_gemm(int64_t M, int64_t N, int64_t K,
                         bsfp8_format a_fmt, const void* a, const void* a_scales,
                         bsfp8_format b_fmt, const void* b, const void* b_scales,
                         bsfp8_out out, void* d, int64_t ldd, hipStream_t stream);

/*
 * scaled_gemm_ex -- D = alpha * deq(A) deq(B) + beta * C (the alpha/beta
 * epilogue of the CUTLASS argument list in [RUBIN-FP4] section 3.4).
 *
 * All arguments as for scaled_gemm, plus:
 * alpha: scales the FP32 accumulator (alpha * acc is rounded to FP32).
 * c:     M x N row-major, the same element type as d, leading dimension
 *        ldc >= N, aligned to its element size.  Read only when beta != 0
 *        (then it must not be null); it may be d itself (with ldc == ldd) to
 *        accumulate in place.  Any other overlap of c and d is undefined.
 * beta:  beta * C is added to alpha * acc with one FP32 fused multiply-add,
 *        then the sum is converted to the output type.
 * K = 0 writes beta * C (zeros when beta == 0).
 * scaled_gemm(...) is scaled_gemm_ex(..., 1.0f, NULL, 0, 0.0f, ...).
 *
 * Accuracy: |D - (alpha exact + beta C)| <= tau (|alpha| S + |beta C|), with
 * tau as for scaled_gemm (plus one FP32 rounding for FP32 output).
 */
bsfp8_status scaled_gemm_ex(int64_t M, int64_t N, int64_t K,
                            bsfp8_format a_fmt, const void* a, const void* a_scales,
                            bsfp8_format b_fmt, const void* b, const void* b_scales,
                            float alpha, const void* c, int64_t ldc, float beta,
                            bsfp8_out out, void* d, int64_t ldd, hipStream_t stream);

/*
 * Scale granularity of an operand ([CDNA4-FP8] section 3.3 weighs per-row,
 * per-column and per-tensor scales against per-tile ones and keeps per tile;
 * its closing section keeps a per-matrix scale for evenly distributed data).
 * The rows are those of the operand's rows x K storage: per-row scales of A
 * are per output row, per-row scales of B (stored N x K) are per output column.
 */
typedef enum {
    BSFP8_GRAN_TILE = 0,    /* FP8: FP32 [ceil(rows / 128)][K / 32], one per 128 x 32 tile */
    BSFP8_GRAN_ROW = 1,     /* FP8: FP32 [rows], one per row, constant along K */
    BSFP8_GRAN_TENSOR = 2,  /* FP8: FP32 [1], one for the whole operand */
    BSFP8_GRAN_MX32 = 3     /* MXFP4: E8M0 [rows][K / 32], one per 32-element K block */
} bsfp8_granularity;

/*
 * fp8_quantize_granular -- FP8 quantisation with the scale granularity g.
 *
 * x, rows, k, ld, fmt, codes: as for fp8_quantize.
 * g: BSFP8_GRAN_TILE (exactly fp8_quantize with tile_rows = 128),
 *    BSFP8_GRAN_ROW or BSFP8_GRAN_TENSOR; BSFP8_GRAN_MX32 is UNSUPPORTED.
 * scales: out, FP32, the shape g names (4-byte aligned).
 *
 * Per scale group (tile, row or whole operand): amax = max |x|, s = amax / F
 * rounded to FP32 (s = 1 when that is zero), code = saturating round-to-
 * nearest-even of (x / s rounded to FP32).  Bit-exact.  rows == 0 or k == 0
 * writes nothing.  BSFP8_GRAN_TENSOR runs three launches and keeps partial
 * maxima in the codes buffer between them, so reads of codes or scales[0]
 * that overlap the call race with it.
 */
bsfp8_status fp8_quantize_granular(const float* x, int64_t rows, int64_t k, int64_t ld,
                                   bsfp8_granularity g, bsfp8_format fmt, uint8_t* codes,
                                   float* scales, hipStream_t stream);

/*
 * scaled_gemm_granular -- scaled_gemm_ex with a scale granularity per operand:
 * D = alpha * deq(A) deq(B) + beta * C, deq(X)[r][k] = code * scale(r, k).
 *
 * All arguments as for scaled_gemm_ex, plus a_g and b_g, the granularities of
 * a_scales and b_scales.  Supported combinations:
 *   FP8, both scales constant along K (ROW or TENSOR on each side): the scale
 *     product multiplies the FP32 sum over all of K once, at write-back.
 *   FP8, TILE with TILE or TENSOR: the product of the two K block scales
 *     multiplies each 32-wide K block's partial sum, as in scaled_gemm.
 *   FP8, TILE with ROW (either side): the TILE side's K block scale
 *     multiplies each K block's partial sum, and the ROW side's scale (of the
 *     output row for A, of the output column for B) multiplies the FP32 sum
 *     over K at write-back.
 *   MXFP4: MX32 on both sides (as scaled_gemm).
 * Other combinations return BSFP8_ERR_UNSUPPORTED, and so does K >= 2^23
 * with both FP8 scales constant along K.
 * Accuracy as for scaled_gemm_ex.
 */
bsfp8_status scaled_gemm_granular(int64_t M, int64_t N, int64_t K,
                                  bsfp8_format a_fmt, const void* a, const void* a_scales,
                                  bsfp8_granularity a_g,
                                  bsfp8_format b_fmt, const void* b, const void* b_scales,
                                  bsfp8_granularity b_g,
                                  float alpha, const void* c, int64_t ldc, float beta,
                                  bsfp8_out out, void* d, int64_t ldd, hipStream_t stream);

/*
 * MX variants ([RUBIN-FP4] section 5.3 offers blocks of 16 or 8 elements where
 * 32 is too coarse; section 3.2 offers FP16 or BF16 block scales where a power
 * of two is too coarse, at twice the scale storage).
 */
typedef enum {
    BSFP8_MX_E8M0 = 0,  /* one byte, 2^(code - 127) */
    BSFP8_MX_F16 = 1,   /* IEEE binary16 bit pattern */
    BSFP8_MX_BF16 = 2   /* bfloat16 bit pattern (upper half of a binary32) */
} bsfp8_mx_scale;
/*
 * mx_quantize -- E2M1 quantisation with blocks of `block` consecutive K
 * elements (32, 16 or 8) and block scales of format sfmt.
 *
 * x:      rows x k FP32, row-major, leading dimension ld; 16-byte aligned,
 *         ld a multiple of 4, ld >= k.  rows >= 0; k >= 0, a multiple of 32.
 * packed: out, rows x (k / 2) bytes, row stride k / 2, low nibble first.
 * scales: out, [rows][k / block]: bytes (E8M0) or 16-bit patterns (FP16,
 *         BF16, 2-byte aligned).
 *
 * Per block, amax = max |x|:
 *   E8M0: as mxfp4_quantize (block = 32 with E8M0 is exactly mxfp4_quantize);
 *   FP16 / BF16: s = the format's value nearest to amax / 6 (ties to even),
 *         the largest finite value when beyond it, 1 when it is zero (or
 *         amax is 0); code = saturating round-to-nearest-even E2M1 of
 *         (x / s rounded to FP32).
 * Bit-exact.  Finite inputs only.
 */
bsfp8_status mx_quantize(const float* x, int64_t rows, int64_t k, int64_t ld, int block,
                         bsfp8_mx_scale sfmt, uint8_t* packed, void* scales, hipStream_t stream);

/*
 * scaled_gemm_mx -- D = alpha * deq(A) deq(B) + beta * C for E2M1 operands
 * with blocks of `block` (32, 16, 8) K values and sfmt block scales, as
 * mx_quantize writes them.
 *
 * a: M x K/2 packed bytes, a_scales [M][K/block]; b: N x K/2 packed bytes
 * (the K x N column-major operand), b_scales [N][K/block]; a and b 16-byte
 * aligned, the scale arrays 8-byte aligned.  M, N >= 0; K >= 0 a multiple of
 * 32, below 2^23 unless block == 32 with E8M0 scales (BSFP8_ERR_UNSUPPORTED).
 * alpha, c, ldc, beta, out, d, ldd: as for scaled_gemm_ex.
 * block = 32 with E8M0 scales runs the block-scaled MXFP4 GEMM of
 * scaled_gemm.  block = 16 or 8 with E8M0 scales runs on the same
 * block-scaled instruction (block = 8 except on shapes with at least 128
 * tiles of 256 x 256 that the large MXFP4 tiling does not take):
 * each 32-value K block of an operand lane is multiplied in 32 / block
 * passes, one per block with the other values zeroed, each under its own
 * block's scale, so every block keeps its exact scale.  Every other combination is beyond
 * the matrix instructions' block scaling (one E8M0 scale per 32 K values): its
 * operands are dequantised exactly to bf16 (a wide scale as an exact bf16
 * pair hi + lo) and multiplied with FP32 accumulation; 16-bit outputs leave
 * out the lo * lo products (below 2^-16 of hi * hi).  Accuracy as for
 * scaled_gemm_ex.
 */
bsfp8_status scaled_gemm_mx(int64_t M, int64_t N, int64_t K, int block, bsfp8_mx_scale sfmt,
                            const void* a, const void* a_scales, const void* b,
                            const void* b_scales, float alpha, const void* c, int64_t ldc,
                            float beta, bsfp8_out out, void* d, int64_t ldd, hipStream_t stream);

/*
 * scaled_gemm_quantize_a -- D = alpha * deq(Q(x)) deq(B) + beta * C, where
 * Q(x) is the per-tile FP8 quantisation of the FP32 matrix x, carried out
 * inside the GEMM while x is loaded (activations quantised online:
 * [CDNA4-FP8] section 4.2 converts and scales on load, section 3.3 computes
 * each tile's scale from its maximum; [RUBIN-FP4] section 4.2, step 4).
 *
 * x:       M x K FP32, row-major, leading dimension ldx (elements): 16-byte
 *          aligned, ldx a multiple of 4, K <= ldx < 2^22.
 * a_fmt:   the FP8 format of A's codes (E4M3 or E5M2).
 * b_fmt, b, b_scales: as for scaled_gemm; b_g is BSFP8_GRAN_TILE (b_scales
 *          FP32 [ceil(N/128)][K/32]) or BSFP8_GRAN_TENSOR (b_scales FP32 [1]).
 * alpha, c, ldc, beta, out, d, ldd: as for scaled_gemm_ex.
 * a_codes, a_scales: both NULL, or both non-NULL and 4-byte aligned: then
 *          they receive A's codes (M x K bytes, row stride K) and scales
 *          (FP32 [ceil(M/128)][K/32]), byte-for-byte what fp8_quantize with
 *          tile_rows = 128 writes for x (for instance to keep the quantised
 *          activations for a backward pass).  With them and N > 384 the call
 *          runs fp8_quantize into them and then the GEMM (two launches, the
 *          same result): quantising every A tile once beats re-quantising it
 *          for every column of output tiles.
 *
 * The codes the GEMM multiplies are exactly those of fp8_quantize, so D is
 * that of fp8_quantize followed by scaled_gemm_ex, with the same accuracy.
 * M, N >= 0 (any value), K >= 0 a multiple of 32.  K = 0 writes beta * C.
 * N = 0 writes only a_codes / a_scales (when given).  x must not overlap d,
 * a_codes or a_scales.  Every output tile that reads the same rows of x
 * quantises them again, so the single-launch form pays off on narrow outputs
 * (a few hundred columns) and small, launch-bound products.
 */
bsfp8_status scaled_gemm_quantize_a(int64_t M, int64_t N, int64_t K, const float* x, int64_t ldx,
                                    bsfp8_format a_fmt, bsfp8_format b_fmt, const void* b,
                                    const void* b_scales, bsfp8_granularity b_g, float alpha,
                                    const void* c, int64_t ldc, float beta, bsfp8_out out,
                                    void* d, int64_t ldd, uint8_t* a_codes, float* a_scales,
                                    hipStream_t stream);

/*
 * Blocks of 128: FP8 codes with one power-of-two scale (an E8M0 byte, as for
 * MXFP4) per 1 x 128 block of a row, or per 128 x 128 block.  Activations and
 * gradients usually take 1 x 128 blocks, weights 128 x 128 blocks, whose
 * transpose has the same scales.
 *
 * Code matrices are rows x kp bytes with row stride kp = k rounded up to a
 * multiple of 32; columns k .. kp-1 hold zero codes (NaN codes where their block
 * holds an infinity or a NaN), so any k is accepted and kp is the K of the GEMM.
 * Scale bytes lie in words of four K blocks,
 * [ceil(k / 512)][R][4] with R = rows (1 x 128) or ceil(rows / 128)
 * (128 x 128): byte (g, r, j) is the scale of K block 4 g + j of scale row r.
 * The words are 4-byte aligned.
 */

/*
 * fp8_quantize_block128 -- block-of-128 FP8 quantisation of x, of its
 * transpose, or of both from one read.
 *
 * x:      rows x k elements of type x_type (BSFP8_OUT_F32, BSFP8_OUT_BF16 or
 *         BSFP8_OUT_F16), row-major, leading dimension ld >= k, aligned to its
 *         element size.  16-byte aligned x with a row stride of a multiple of
 *         16 bytes is read with 16-byte loads; anything else element by element.
 * rows, k: >= 0, any value, at most 2^31 - 1 and 2^23 tiles of 128 x 128.
 * block_rows: 1 (1 x 128 blocks) or 128 (128 x 128 blocks); for the transpose
 *         the blocks are those of x^T.
 * codes, scales:     out, the codes and scales of x; both NULL: not wanted.
 * codes_t, scales_t: out, those of x^T (k rows, K = rows); both NULL: not wanted.
 *         Code buffers are 16-byte aligned.  At least one pair must be given.
 *
 * Per block: e = the smallest integer with F * 2^e >= max |x| (0 when that is
 * 0), clamped to [-127, 127]; scale byte e + 127; code = round-to-nearest-even
 * of x * 2^-e (exact scaling).  A block with an infinity or a NaN gets the
 * scale byte 255 (NaN) and NaN codes (0x7F).  Unused bytes of the last scale
 * word are 127.  Bit-exact.  rows == 0 or k == 0 writes nothing.  The outputs
 * must not overlap x or each other.
 */
bsfp8_status fp8_quantize_block128(const void* x, bsfp8_out x_type, int64_t rows, int64_t k, int64_t ld,
                                   int block_rows, bsfp8_format fmt, uint8_t* codes, uint8_t* scales,
                                   uint8_t* codes_t, uint8_t* scales_t, hipStream_t stream);

/*
 * scaled_gemm_block128 -- D = alpha * deq(A) deq(B) + beta * C for operands
 * written by fp8_quantize_block128.
 *
 * a: M x K codes, a_scales E8M0 words [ceil(K / 512)][M or ceil(M / 128)][4]
 * for a_block_rows 1 or 128; b: N x K codes (the K x N column-major operand)
 * likewise.  a and b 16-byte aligned, the scales 4-byte aligned.  M and N at
 * most 2^31 - 257.  All formats (E4M3, E5M2) and block shapes mix.  K a
 * multiple of 32, below 2^23 (the kernels address a 256-row band of an operand
 * with 32-bit offsets; larger K returns BSFP8_ERR_UNSUPPORTED).  alpha, c, ldc, beta, out, d, ldd: as for
 * scaled_gemm_ex.  A NaN scale makes every output that uses its block NaN.
 *
 * 16-bit outputs run on the block-scaled FP8 matrix instruction, which takes
 * the E8M0 bytes itself; FP32 output widens the codes, times their scale, to
 * bf16 and uses the bf16 instruction (exact for dequantised magnitudes from
 * 2^-126 to below 2^128; smaller ones lose bits, those below 2^-133 count as
 * zero; 2^128 and more, beyond FP32 too, count as infinite where 16-bit outputs
 * multiply them out: fp8_quantize_block128 writes such codes for |x| above
 * 0.93 2^128).
 * Accuracy as for scaled_gemm_ex.  For 16-bit outputs the instruction keeps 13
 * fraction bits of each group of 8 products: before it is rounded to the output
 * type, D is within 7 2^-13 of sum |a b| besides the FP32 accumulator's
 * roundings.  That worst case is above half a step of FP16 (2^-11): results that
 * need FP16's last bit take FP32 output.
 * The kernel form is chosen by the sizes and the output type alone, and no sum
 * depends on timing: equal calls give equal
 * bits.
 */
bsfp8_status scaled_gemm_block128(int64_t M, int64_t N, int64_t K, bsfp8_format a_fmt, const void* a,
                                  const void* a_scales, int a_block_rows, bsfp8_format b_fmt, const void* b,
                                  const void* b_scales, int b_block_rows, float alpha, const void* c,
                                  int64_t ldc, float beta, bsfp8_out out, void* d, int64_t ldd,
                                  hipStream_t stream);

/*
 * rmsnorm_quantize_block128 -- the residual's addition and root-mean-square norm ahead of a
 * projection, to FP8 codes with one E8M0 scale per 1 x 128 block, from one read.
 *
 *   h = x + residual, rounded to h_type (without a residual h = x)
 *   rstd = 1 / sqrt(mean over k of h^2 + eps)          y = (h * rstd) * weight
 *
 * x:        rows x k elements of x_type, row-major, leading dimension ldx >= k.
 * residual: NULL, or rows x k of h_type (ldr); then h receives the sum (rows x k of
 *           h_type, ldh).  h may be residual itself, or x itself where the types agree.
 * weight:   NULL (ones), or k elements of w_type.
 * eps:      finite, >= 0.
 * codes, scales: out, as fp8_quantize_block128 with block_rows 1 writes them for the
 *           FP32 matrix y; both NULL: not wanted.
 * y:        out, rows x k of y_type (ldy), rounded once from FP32; NULL: not wanted.
 *           codes or y must be given.  y may be x itself where the types agree.
 * rstd:     out, FP32 [rows], what rmsnorm_backward takes; NULL: not wanted.
 * rows >= 0; k at most 32768 (BSFP8_ERR_UNSUPPORTED beyond).  Every array is aligned to
 * its element size, codes to 16 bytes, scales to 4; any other overlap is undefined.
 *
 * FP32 arithmetic, each operation (the reciprocal root is one) rounded once; the sum of squares in an order that depends on k
 * alone, so a row gives the same bits in every call.  The norm is that of the rounded h, which a backward
 * pass reads.  Infinities and NaN spread as the formulas have it: a NaN to its row,
 * an infinity (rstd = 0) to itself as NaN, its row otherwise zeros (a row whose squares add
 * up past FP32's range is zeros likewise).  Blocks of y with a
 * non-finite value get the scale byte 255 and NaN codes.  rows == 0 or k == 0 writes nothing.
 */
bsfp8_status rmsnorm_quantize_block128(const void* x, bsfp8_out x_type, int64_t rows, int64_t k, int64_t ldx,
                                       const void* residual, bsfp8_out h_type, int64_t ldr, const void* weight,
                                       bsfp8_out w_type, float eps, bsfp8_format fmt, uint8_t* codes, uint8_t* scales,
                                       void* y, bsfp8_out y_type, int64_t ldy, void* h, int64_t ldh, float* rstd,
                                       hipStream_t stream);

/*
 * rmsnorm_backward -- the gradients of y = (h * rstd(h)) * weight.
 *
 *   g = dy * weight, xh = h * rstd
 *   dx = rstd (g - xh mean(g xh)) (+ dh)               dweight = sum over rows of dy xh
 *
 * dy: rows x k of dy_type (ldy); h: rows x k of h_type (ldh) and rstd as the forward call
 * left them; weight as there.  dh: NULL, or the gradient that reaches h along the
 * residual, rows x k of dh_type (lddh).  dx: out, rows x k of h_type (ldx), the
 * gradient of x and of the residual; it may be dy, h or dh itself where type and leading
 * dimension agree.  dweight: out, FP32 [k], added to what is there with accumulate = 1
 * (0 otherwise); NULL: not wanted.  workspace: rmsnorm_backward_workspace(rows, k) bytes,
 * 16-byte aligned (needed with dweight only); calls that may run at once need one each.
 * FP32 arithmetic, sums in a fixed order (dx's, as the norm's, in one that depends on k alone).  rows == 0 writes only dweight (zeros, or
 * nothing with accumulate); k as in the forward call.
 */
int64_t rmsnorm_backward_workspace(int64_t rows, int64_t k);
bsfp8_status rmsnorm_backward(const void* dy, bsfp8_out dy_type, int64_t ldy, const void* h, bsfp8_out h_type,
                              int64_t ldh, const float* rstd, const void* weight, bsfp8_out w_type, const void* dh,
                              bsfp8_out dh_type, int64_t lddh, int64_t rows, int64_t k, void* dx, int64_t ldx,
                              float* dweight, int accumulate, void* workspace, int64_t workspace_bytes,
                              hipStream_t stream);

/*
 * Grouped operators: rows sorted by group (by the expert a token is sent to), group e
 * being rows offsets[e] .. offsets[e + 1] - 1.  offsets is a DEVICE array of
 * groups + 1 int32 that does not decrease, from >= 0 to <= rows; it is read when the kernels run,
 * so that no size has to reach the host and a captured call follows it.  Groups may be
 * empty; rows of no group are left as they were.  An array that breaks these rules gives
 * undefined results within the outputs, never an access outside the arrays.  At most
 * 1024 groups and 2^30 rows (BSFP8_ERR_UNSUPPORTED beyond).
 */

/*
 * fp8_quantize_grouped_block128 -- fp8_quantize_block128 (1 x 128 blocks) of rows in
 * groups, optionally taken by index, and of their transpose group by group.
 *
 * x:      source_rows x k of x_type, leading dimension ld, as fp8_quantize_block128.
 * index:  NULL (then source_rows >= rows), or a device array of `rows` int32: sorted row i
 *         is row index[i] of x; a number outside 0 .. source_rows - 1 stands for a row of zeros.
 * codes, scales: out, those of the sorted rows (rows x kp, [ceil(k / 512)][rows][4]);
 *         both NULL: not wanted.
 * codes_t, scales_t: out, those of the transpose; both NULL: not wanted.  codes_t is k rows of
 *         `columns` bytes: group e's rows are the columns from c(e) on, c(e) the sum of
 *         the sizes before it, each rounded up to a multiple of 128; zero codes fill
 *         its last block (NaN codes where the block holds an infinity or a NaN).
 *         scales_t is [words][k][4]: group e's words start at w(e), the sum over the
 *         groups before it of ceil(size / 512); byte (w(e) + j / 4, r, j % 4) is the scale of its
 *         block j of row r, unused bytes of its last word 127.  What lies past the last
 *         group is left as it was.
 * columns, words: a multiple of 128 and a count, at least what
 *         block128_grouped_columns(rows, groups) and block128_grouped_words(rows, groups) return
 *         (enough for any sizes of so many groups).
 * At most 2^23 tiles of 128 x 128 (columns / 128 * ceil(k / 128)) with the transpose, 2^27 pieces of 512
 * (rows * ceil(k / 512)) without.
 */
int64_t block128_grouped_columns(int64_t rows, int64_t groups);
int64_t block128_grouped_words(int64_t rows, int64_t groups);
bsfp8_status fp8_quantize_grouped_block128(const void* x, bsfp8_out x_type, int64_t source_rows, int64_t k, int64_t ld,
                                           const int32_t* index, int64_t rows, const int32_t* offsets, int64_t groups,
                                           bsfp8_format fmt, uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                                           int64_t columns, uint8_t* scales_t, int64_t words, hipStream_t stream);

/*
 * scaled_gemm_grouped_block128 -- D[i] = alpha deq(A)[i] deq(B[e])^T + beta C[i] for the rows i of
 * each group e: the forward product of experts and, with transposed weights, the gradient
 * of their input.
 *
 * a: M x K codes, a_scales E8M0 words [ceil(K / 512)][M][4] (1 x 128 blocks); b: `groups`
 * matrices of N x K codes, one after another, b_scales likewise [groups][ceil(K / 512)][R][4], R = N or
 * ceil(N / 128) for b_block_rows 1 or 128.  alpha, c, ldc, beta, out, d, ldd, the
 * limits on N and K and the accuracy: as for scaled_gemm_block128.  At most 2^24 - 16 tiles of
 * 64 x 128 ((M / 64 + groups) ceil(N / 128)).  The kernel form is chosen by the sizes, the
 * number of groups, the output type, ldd, ldc and whether beta is 0: equal calls give equal bits.
 */
bsfp8_status scaled_gemm_grouped_block128(int64_t M, int64_t N, int64_t K, int64_t groups, const int32_t* offsets,
                                          bsfp8_format a_fmt, const void* a, const void* a_scales, bsfp8_format b_fmt,
                                          const void* b, const void* b_scales, int b_block_rows, float alpha,
                                          const void* c, int64_t ldc, float beta, bsfp8_out out, void* d, int64_t ldd,
                                          hipStream_t stream);

/*
 * scaled_gemm_grouped_wgrad_block128 -- D[e] = alpha sum over the rows i of group e of
 * deq(A)[:, i] deq(B)[:, i]^T + beta C[e]: the weight gradients of experts.
 *
 * a: M x columns, b: N x columns codes, a_scales [words][M][4], b_scales [words][N][4]:
 * transposes that fp8_quantize_grouped_block128 wrote with the same offsets.  columns below 2^23
 * (BSFP8_ERR_UNSUPPORTED).  d: `groups` matrices of M x N, d_group elements apart (at least
 * (M - 1) ldd + N with more than one group), c likewise (c_group).  A group without
 * rows gives beta C (zeros for beta == 0).  At most 2^23 tiles of 128 x 128 in all, each
 * group's padded to 8.  Otherwise as scaled_gemm_block128.
 */
bsfp8_status scaled_gemm_grouped_wgrad_block128(int64_t M, int64_t N, int64_t columns, int64_t words, int64_t groups,
                                                const int32_t* offsets, bsfp8_format a_fmt, const void* a,
                                                const void* a_scales, bsfp8_format b_fmt, const void* b,
                                                const void* b_scales, float alpha, const void* c, int64_t ldc,
                                                int64_t c_group, float beta, bsfp8_out out, void* d, int64_t ldd,
                                                int64_t d_group, hipStream_t stream);

/*
 * The states of an AdamW step: FP32, or FP8 (E4M3 codes with one E8M0 scale
 * per 128 consecutive elements).
 */
typedef enum {
    BSFP8_STATE_F32 = 0,
    BSFP8_STATE_FP8 = 1
} bsfp8_state;

/* One tensor of an AdamW step: n contiguous elements, every pointer a device
 * pointer aligned to its element size. */
typedef struct {
    void* p;             /* parameters, in and out */
    const void* g;       /* gradients */
    void* m;             /* first moment, in and out: FP32 values, or E4M3 codes */
    void* v;             /* FP32: the second moment; FP8: E4M3 codes of its square root */
    uint8_t* m_scales;   /* FP8: E8M0 [ceil(n / 128)], in and out; FP32: NULL */
    uint8_t* v_scales;
    int64_t n;           /* >= 0 */
} bsfp8_adamw_tensor;

/* What the tensors of a step share.  Pointers are device pointers, read when
 * the kernel runs, so that a captured step follows them; NULL: not used. */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;               /* the number of this step, >= 1 */
    uint32_t seed;              /* of the stochastic rounding */
    const float* lr_dev;        /* replaces lr */
    const int64_t* step_dev;    /* replaces step, >= 1 when the kernel runs */
    const float* grad_scale;    /* multiplies every gradient */
    const float* found_inf;     /* not zero: the step changes nothing */
} bsfp8_adamw_args;

/*
 * adamw_step -- one step of AdamW (decoupled weight decay) over `count`
 * tensors in one launch per 48 tensors.  `tensors` and `args` are host arrays,
 * read during the call.
 *
 * Per element, in FP32 with each operation rounded once (the constants in
 * parentheses are formed in 64 bits, each operation rounded once, and rounded to
 * FP32; with lr_dev or step_dev on the device, whose pow may differ from the
 * host's in the last of the 64 bits):
 *   g  = gradient * grad_scale
 *   m' = (beta1) m + (1 - beta1) g          v' = (beta2) v + ((1 - beta2) g) g
 *   p' = (1 - lr weight_decay) p - ((lr / (1 - beta1^t)) m') / ((1 / sqrt(1 - beta2^t)) sqrt(v') + (eps))
 *
 * p_type:  FP32 or bf16 parameters; g_type: FP32, bf16 or FP16 gradients.
 * state:   FP32 keeps m' and v'.  FP8 keeps E4M3 codes of m' and of
 *          r' = sqrt(v') (v = r * r when read back), scaled per 128 elements
 *          as fp8_quantize_block128 does and rounded stochastically: with y the
 *          scaled magnitude cut to 2^-20 of its code step, the code above is
 *          taken when y's distance from the code below, in steps, plus b / 2^16
 *          reaches 1.  A nonzero r' keeps a nonzero code.  bf16 parameters are
 *          rounded likewise: the 16 bits cut off carry when their sum with b
 *          reaches 2^16.  The random bits b depend on (seed, step, position of
 *          the tensor in `tensors`, element) only, so a step is reproducible.
 * Zeroed codes and scale bytes are valid initial states, as zeroed FP32 ones.
 *
 * beta1, beta2 in [0, 1); eps >= 0; all finite.  The p, m, v and scale arrays
 * of a call must not overlap each other, the gradients or the scalars that args
 * points to (BSFP8_ERR_INVALID_ARG; BSFP8_ERR_NO_MEMORY where the check of many
 * tensors finds no host memory).  Infinities and NaN in gradients spread to p, m and
 * v; with FP8 states to the whole block of 128 (scale byte 255): use found_inf.
 */
bsfp8_status adamw_step(const bsfp8_adamw_tensor* tensors, int64_t count, bsfp8_out p_type, bsfp8_out g_type,
                        bsfp8_state state, const bsfp8_adamw_args* args, hipStream_t stream);

/*
 * bsfp8_status_string -- the name of a status code ("BSFP8_OK", ...;
 * "BSFP8_ERR_UNKNOWN" for a value that is not a bsfp8_status), in static
 * storage owned by the library; never NULL.  The status values follow the
 * check-then-run flow of the CUTLASS GEMM interface in [RUBIN-FP4] section
 * 3.4 (can_implement, then initialize and run): every argument check happens
 * before anything runs, and a rejected call reports why instead of running.
 */
const char* bsfp8_status_string(bsfp8_status s);

/* Library version, (major << 16) | minor. */
int bsfp8_version(void);

#ifdef __cplusplus
}
#endif
#endif /* BSFP8_H */

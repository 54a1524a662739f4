/*
 * fp8fg.h -- fine-grained FP8 quantization and block-scaled FP8 GEMM on
 * AMD Instinct MI355X (gfx950).  C ABI of libfp8fg.so.
 *
 * What is computed follows the DeepSeek-V3 FP8 training text as it appears
 * on these pages (no section numbers; passages are named by subject):
 *   [why-be]   why-be.why-be.co.kr (untitled): online max-abs per 1x128
 *              activation tile / 128x128 weight block; E4M3 on all tensors;
 *              1x128 -> 128x1 tiles in the backward pass; integral
 *              power-of-two scaling factors.
 *   [thedaegu] thedaegu.com, "OMG! The most effective Deepseek Ever!":
 *              max-abs mapped onto the largest FP8 value; promotion of
 *              partial sums to FP32 with per-group scaling along K
 *              (Figure 7(b) passage); Fprop / Dgrad / Wgrad in FP8
 *              (Figure 6 passage).
 *   [hearaon]  hearaon.co.kr (untitled): limited accumulation width of
 *              FP8 MMA; activations quantized before the MoE up-projection.
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library never allocates, frees, copies to the host or synchronizes:
 *     it validates the host-visible arguments, enqueues its kernels on
 *     `stream` (a hipStream_t passed as void*; NULL = the default stream)
 *     on the current HIP device, and returns.
 *   - Sizes and strides are in ELEMENTS of the pointed-to type.
 *   - FP8 is OCP E4M3 (bias 7, largest finite 448, no infinity); bytes are
 *     produced with round-to-nearest-even and saturation.
 *   - Scratch memory is the caller's too: an entry point that needs some has a
 *     ..._workspace function that gives its size in bytes (0 for arguments
 *     that it would refuse).
 *   - Return value: FP8FG_OK (0) or an error code.  On any error other than
 *     FP8FG_ELAUNCH nothing was enqueued.  FP8FG_ELAUNCH reports a HIP
 *     launch failure after enqueue (the stream state is then undefined).
 *   - Inputs must be finite, except where an entry point says what it does
 *     with others; results for NaN/Inf inputs are unspecified.
 *   - Outputs must not alias inputs.
 *   - Calls are thread-safe; the only global state is a per-device cache of
 *     the compute-unit count, filled once.
 */
#ifndef FP8FG_H
#define FP8FG_H

#include <stdint.h>

#if defined(FP8FG_BUILDING_LIBRARY)
#define FP8FG_API __attribute__((visibility("default")))
#else
#define FP8FG_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

enum fp8fg_status {
  FP8FG_OK = 0,
  FP8FG_EINVAL = 1,       /* null pointer, negative size, bad enum value     */
  FP8FG_ESHAPE = 2,       /* size not a required multiple; stride or workspace
                             too small                                      */
  FP8FG_EALIGN = 3,       /* pointer or row pitch misaligned                  */
  FP8FG_EUNSUPPORTED = 4, /* valid combination that is not implemented        */
  FP8FG_ELAUNCH = 5       /* HIP reported an error at launch                  */
};

/* element types */
enum { FP8FG_BF16 = 0, FP8FG_F32 = 1, FP8FG_E4M3 = 2 };
/* tile orientation of fp8_quantize_rowtile */
enum { FP8FG_TILE_1x128 = 0, FP8FG_TILE_128x1 = 1 };
/* scale rules */
enum { FP8FG_SCALE_AMAX = 0, FP8FG_SCALE_POW2 = 1 };
/* how the B operand of the GEMM is scaled along N */
enum { FP8FG_BSCALE_BLOCK128 = 0, FP8FG_BSCALE_COL = 1 };
/* score of the router */
enum { FP8FG_SCORE_SOFTMAX = 0, FP8FG_SCORE_SIGMOID = 1 };
/* GEMM flags (bit set) */
enum {
  FP8FG_GEMM_DEFAULT = 0,
  /* sum the whole K inside the FP8 matrix-core datapath and scale once at the
     end (the naive per-tensor baseline; implies FP8FG_GEMM_FP8_MFMA) */
  FP8FG_GEMM_NO_PROMOTION = 1,
  /* form each 128-wide K group's partial sum with the FP8 MFMA instead of the
     default exact path (faster, but gfx950's FP8 MFMA keeps only ~14 bits
     below the largest of every 8 consecutive products) */
  FP8FG_GEMM_FP8_MFMA = 2,
  /* the FP8 matrix instruction dequantizes, with the scales' powers of two
     as its E8M0 operand scales (the microscaling form; implies
     FP8FG_GEMM_FP8_MFMA and its precision; fastest with power-of-two
     scales) */
  FP8FG_GEMM_E8M0_SCALES = 4,
  /* default path with BLOCK128 scales only: fix the tile shape instead of
     choosing it from the sizes -- WIDE the 256-row tiles, NARROW the 64x128
     weight-streaming tiles.  Every choice gives the same result bit for bit
     (for N >= 256); for tests and tuning.  Setting both, or either together
     with an FP8 flag or COL scales, is FP8FG_EINVAL. */
  FP8FG_GEMM_TILES_WIDE = 8,
  FP8FG_GEMM_TILES_NARROW = 16
};

/*
 * fp8_quantize_rowtile -- online max-abs per tile, scale, E4M3 quantization.
 * [why-be] fine-grained quantization and backward-pass paragraphs;
 * [thedaegu] dynamic-range paragraph.
 *
 *   x      : input [rows][cols], row pitch ldx (elements of x_type).
 *            x_type BF16 or F32: the values themselves.
 *            x_type E4M3 (requantization, tile == 128x1 only): bytes of a
 *            1x128-quantized tensor whose scales are
 *            x_scale[r * xs_rs + (c / 128) * xs_ts]; the source value is
 *            RN32(dec(x[r][c]) * scale).  x_scale is ignored otherwise.
 *   tile == FP8FG_TILE_1x128: a tile is 128 consecutive columns of one row.
 *            Requires cols % 128 == 0.  Output q[r * ldq + c] (u8, same
 *            orientation), scale s[r * s_rs + (c / 128) * s_ts].
 *   tile == FP8FG_TILE_128x1: a tile is 128 consecutive rows of one column.
 *            Requires rows % 128 == 0 and cols % 128 == 0.  Output is
 *            TRANSPOSED: q[c * ldq + r], scale s[c * s_rs + (r / 128) * s_ts]
 *            (i.e. the 1x128 tiling of the transpose).
 *   scale_rule AMAX: s = max(RN32(amax / 448), 2^-126);
 *              POW2: s = max(2^ceil(log2(amax / 448)), 2^-126).
 *   q = E4M3_RNE(RN32(x / s)) with correctly rounded fp32 division.
 *
 *   Alignment: x, q 16-byte aligned; ldx * sizeof(x_type) and ldq multiples
 *   of 16 bytes; s and x_scale 4-byte aligned.  rows == 0 or cols == 0 is a
 *   valid no-op.
 *   Limits (FP8FG_EUNSUPPORTED beyond them): 1x128, at most 2^31 tiles
 *   (rows * cols / 128); 128x1, rows / 128 <= 65535 and
 *   cols / 128 <= (2^32 - 1) / 256.
 */
FP8FG_API int fp8_quantize_rowtile(const void* x, int x_type, int64_t rows, int64_t cols,
                         int64_t ldx, const float* x_scale, int64_t xs_rs,
                         int64_t xs_ts, int tile, int scale_rule, uint8_t* q,
                         int64_t ldq, float* s, int64_t s_rs, int64_t s_ts,
                         void* stream);

/*
 * fp8_quantize_block -- 128x128 weight blocks.  [why-be] / [thedaegu]
 * paragraphs on computing the max-abs online per 128x128 weight block.
 *
 *   w      : input [rows][cols] (BF16 or F32), row pitch ldw; rows and cols
 *            multiples of 128.  One scale per block:
 *            s[(r / 128) * s_rs + (c / 128) * s_cs], same rules as above.
 *   transpose_out == 0: q[r * ldq + c];  == 1: q[c * ldq + r] (cols x rows,
 *            rows contiguous -- the K-contiguous operand layout the GEMM
 *            reads when w is a K x N weight).
 *   Alignment as for fp8_quantize_rowtile.
 *   Limits: rows / 128 <= 65535, cols / 128 <= (2^32 - 1) / 256
 *   (FP8FG_EUNSUPPORTED beyond).
 */
FP8FG_API int fp8_quantize_block(const void* w, int w_type, int64_t rows, int64_t cols,
                       int64_t ldw, int scale_rule, int transpose_out,
                       uint8_t* q, int64_t ldq, float* s, int64_t s_rs,
                       int64_t s_cs, void* stream);

/*
 * fp8_gemm_blockscaled -- C = A . B^T with per-group dequantization scales
 * and FP32 accumulation promoted every 128 elements of K.  [thedaegu]
 * Figure 7(b) passage (promotion; per-group scaling along K) and Figure 6
 * passage (Fprop / Dgrad / Wgrad in FP8); [hearaon] accumulation-precision
 * paragraph.
 *
 *   C[m][n] = sum_kb  sa(m, kb) * sb(kb, n) * P_kb[m][n],
 *   P_kb[m][n] = sum_{k = 128 kb}^{128 kb + 127} dec(a[m * lda + k]) * dec(b[n * ldb + k])
 *
 *   Default path: the products of each P_kb are exact (the FP8 operands are
 *   converted exactly to BF16 in registers and multiplied on the BF16 matrix
 *   cores) and added in FP32; the group's two scales are applied to the FP32
 *   accumulator once per output element and K group (with 128x128 B block
 *   scales the accumulator is kept in units of the current group's scale and
 *   rescaled at each group; a group whose scale lies more than 2^64 below
 *   the largest taken so far for that element is added in units of 2^-64 of
 *   it).  Kernels, tiles and launch counts are chosen from the arguments;
 *   with block scales and N >= 256 every choice gives the same result bit
 *   for bit (so a row's result does not depend on M or on the expert
 *   counts); N = 128 and per-column scales use a kernel that promotes
 *   separate group sums, whose rounding differs within the same accuracy.
 *   Small grids (few 256x256 tiles for the compute units, as with a small
 *   M x N and a long K) run on 64x128 tiles; the flags
 *   FP8FG_GEMM_TILES_WIDE / FP8FG_GEMM_TILES_NARROW fix that choice.  The
 *   library reads no environment variables.
 *
 *   a : E4M3 [M][K] (K contiguous), sa(m, kb) = sa[m * sa_ms + kb * sa_ks].
 *   b : E4M3 [N][K] (K contiguous -- the transposed weight),
 *       b_scale_mode BLOCK128: sb(kb, n) = sb[(n / 128) * sb_ns + kb * sb_ks]
 *       b_scale_mode COL     : sb(kb, n) = sb[n * sb_ns + kb * sb_ks]
 *   c : [M][N] of c_type BF16 (round-to-nearest-even of the FP32 result)
 *       or F32, row pitch ldc.
 *   Requires K % 128 == 0 and N % 128 == 0; any M >= 0.  Scale strides may
 *   be 0 (broadcast).
 *   flags: a bit set of FP8FG_GEMM_NO_PROMOTION, FP8FG_GEMM_FP8_MFMA,
 *       FP8FG_GEMM_E8M0_SCALES and one of FP8FG_GEMM_TILES_WIDE /
 *       FP8FG_GEMM_TILES_NARROW.
 *       NO_PROMOTION: the whole K is summed in the FP8 matrix-core
 *       accumulator and scaled once by sa(m, 0) * sb(0, n); only meaningful
 *       for per-tensor scales, so sa_ks and sb_ks must then be 0.
 *       FP8_MFMA: P_kb comes from the FP8 MFMA (limited internal precision,
 *       see above); promotion and scaling as in the default path.
 *       E8M0_SCALES ([why-be] power-of-two scaling factors; [thedaegu]
 *       passage on exponents shared within small groups): the FP8 MFMA
 *       dequantizes: each scale's power of two 2^(E - 127), E its exponent
 *       field, is the instruction's E8M0 operand scale, and the rest
 *       f = s * 2^(127 - E) -- exactly 1 when s is a power of two, as
 *       FP8FG_SCALE_POW2 produces -- is applied in FP32.  With block scales
 *       and N a multiple of 256 the kernel runs on 256x256 tiles and adds
 *       the products into the accumulator inside the instruction; the
 *       accumulator is kept in units of the current group's f per row and
 *       rescaled by one multiply where f changes (never for power-of-two
 *       scales), as the default path does with whole scales.  Its rounding
 *       then differs from FP8_MFMA's within the same bound.  Otherwise (N
 *       not a multiple of 256, per-column scales) each group's partial sum
 *       is multiplied by f as it is added, and power-of-two scales give
 *       FP8_MFMA's result bit for bit.  Scales must be finite and positive
 *       (an E8M0 scale has no zero; the quantizers' scales are at least
 *       2^-126).  Not combinable with NO_PROMOTION (FP8FG_EINVAL).
 *   Alignment: a, b 16-byte aligned, lda and ldb multiples of 16; c aligned
 *   to its element; scales 4-byte aligned.  (c 16-byte aligned with ldc a
 *   multiple of 4 lets the kernel store 4 outputs per instruction.)
 *   Limits (FP8FG_EUNSUPPORTED beyond them; the kernels address a tile with
 *   32-bit offsets): lda < 2^23, ldb < 2^24, K < 2^31; when promoting,
 *   sa_ms < 2^21 (and sb_ns < 2^21 in the COL mode) and
 *   sa_ks * K/128, sb_ks * K/128 < 2^29; every launch of the chosen kernel
 *   within HIP's 2^32 - 1 work-items per grid dimension (the workgroup
 *   count is computed for the tile shape that will run).
 */
FP8FG_API int fp8_gemm_blockscaled(int64_t M, int64_t N, int64_t K, const uint8_t* a,
                         int64_t lda, const float* sa, int64_t sa_ms,
                         int64_t sa_ks, const uint8_t* b, int64_t ldb,
                         const float* sb, int64_t sb_ns, int64_t sb_ks,
                         int b_scale_mode, void* c, int c_type, int64_t ldc,
                         int flags, void* stream);

/*
 * fp8_grouped_gemm_blockscaled -- the same GEMM for G experts sharing one
 * activation matrix sorted by expert (MoE up/down projections on FP8
 * activations quantized before dispatch: [hearaon] and [thedaegu]
 * paragraphs on FP8 Fprop in MoE up-projections).
 *
 *   offsets : DEVICE int32 [G + 1]; expert e owns rows [offsets[e],
 *             offsets[e+1]) of a and c.  Caller contract (not checked --
 *             that would need a synchronization): offsets[0] == 0,
 *             nondecreasing, offsets[G] <= M_total.  Empty experts are
 *             legal.  Rows of c from offsets[G] on (fp8_dispatch puts its
 *             dropped entries there) are not written.
 *   b_e  = b + e * b_gs   ([N][K], K contiguous, pitch ldb)
 *   sb_e = sb + e * sb_gs (128x128 block scales, indexed as BLOCK128 above)
 *   Other arguments as for fp8_gemm_blockscaled (B scaling is BLOCK128).
 *   Requires G >= 1 (G == 0 with M_total == 0 is a no-op), K % 128 == 0,
 *   N % 128 == 0; b_gs a multiple of 16.  M_total and G at most 2^31 - 1
 *   (the offsets are int32), plus the limits of fp8_gemm_blockscaled
 *   (FP8FG_EUNSUPPORTED beyond them).
 */
FP8FG_API int fp8_grouped_gemm_blockscaled(int64_t G, const int32_t* offsets,
                                 int64_t M_total, int64_t N, int64_t K,
                                 const uint8_t* a, int64_t lda,
                                 const float* sa, int64_t sa_ms, int64_t sa_ks,
                                 const uint8_t* b, int64_t ldb, int64_t b_gs,
                                 const float* sb, int64_t sb_ns, int64_t sb_ks,
                                 int64_t sb_gs, void* c, int c_type,
                                 int64_t ldc, int flags, void* stream);

/*
 * fp8_rmsnorm_quantize -- root-mean-square norm with the residual's addition
 * and an E4M3 output in 1x128 tiles: the producer of the activations that
 * the GEMMs read ([why-be], [thedaegu]: every GEMM input is quantized per
 * 1x128 tile), without the bf16 tensor in between.
 *
 *   h[m][c]  = RN(x[m][c] + r[m][c]) in x_type (h = x where r is null)
 *   rstd[m]  = 1 / sqrt(sum_c h^2 / cols + eps), at most FLT_MAX; 0 for a row
 *              of zeros with eps 0 (y is then 0, and the gradient below has
 *              no part of the norm)
 *   y[m][c]  = (h * rstd) * gamma[c], in fp32
 *   s, q     = the 1x128 scale and E4M3 bytes of the fp32 y, by the rules of
 *              fp8_quantize_rowtile
 *
 *   x, r, h, y : x_type BF16 or F32 with row pitches ldx, ldr, ldh, ldy.
 *            r may be null (nothing is added).  h may be null (not stored);
 *            so may y (the norm rounded to x_type), q with s (no quantized
 *            output) and rstd.
 *   gamma    : [cols], g_type BF16 or F32.  eps >= 0, finite.
 *   A row's results do not depend on the other rows or their number.
 *   Any finite h, also one whose squares leave fp32's range: the statistics
 *   of such a row are formed in fp64.
 *   Requires cols % 128 == 0.  rows == 0 or cols == 0 is a valid no-op.
 *   Alignment: x, r, h, y, gamma, q 16-byte aligned, their pitches multiples
 *   of 16 bytes; s and rstd 4-byte aligned.
 *   Limits (FP8FG_EUNSUPPORTED): cols <= 32768 (a row stays in one
 *   workgroup's registers); here and below rows <= 2^31 - 1, row pitches and
 *   s_rs <= 2^29 elements, s_ts <= 2^31 - 1 (64-bit offsets hold their
 *   products).
 */
FP8FG_API int fp8_rmsnorm_quantize(const void* x, int x_type, int64_t rows, int64_t cols,
                         int64_t ldx, const void* r, int64_t ldr, const void* gamma,
                         int g_type, float eps, int scale_rule, void* h, int64_t ldh,
                         void* y, int64_t ldy, uint8_t* q, int64_t ldq, float* s,
                         int64_t s_rs, int64_t s_ts, float* rstd, void* stream);

/*
 * fp8_rmsnorm_backward -- gradient of the norm above, passed straight
 * through the quantizer.
 *
 *   xh = h * rstd,  a = dy * gamma,  dx = rstd * (a - xh * mean_c(a * xh)) + dh
 *   dgamma[c] = sum_m dy * xh
 *
 *   dy, dh, h, dx : x_type, as above.  dh (the gradient reaching h along the
 *            residual stream) may be null.  dx is the gradient of both x and
 *            r.
 *   rstd     : as the forward stored it.
 *   dgamma   : fp32 [cols], overwritten (zeros for rows == 0).
 *   workspace: at least fp8_rmsnorm_backward_workspace(rows, cols) bytes,
 *            16-byte aligned: partial sums of dgamma, added in a fixed
 *            order.  FP8FG_ESHAPE if workspace_bytes is less.
 *   Requires cols % 8 == 0.  Alignment and limits as above.
 */
FP8FG_API int64_t fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols);
FP8FG_API int fp8_rmsnorm_backward(const void* dy, int x_type, int64_t rows, int64_t cols,
                         int64_t lddy, const void* dh, int64_t lddh, const void* h,
                         int64_t ldh, const void* gamma, int g_type,
                         const float* rstd, void* dx, int64_t lddx, float* dgamma,
                         void* workspace, int64_t workspace_bytes, void* stream);

/*
 * fp8_route -- the experts of each token and their weights, with choices
 * restricted to groups of experts and a bias that balances their load
 * without an auxiliary loss.
 *
 *   logits : [rows][experts], l_type BF16 or F32, row pitch ldl.  A logit of
 *            -inf or NaN masks its expert.
 *   score  : s = softmax or sigmoid of the logits, to fp32.
 *   bias   : fp32 [experts] or null, added to s for the choice alone:
 *            c = s + bias (a NaN masks the expert).
 *   groups : the experts form `groups` equal runs.  If top_groups < groups,
 *            only the experts of the top_groups groups with the largest sums
 *            of their group_top (1 or 2) best c are candidates.
 *   k      : idx[m][0..k) are the candidates with the largest c, in
 *            descending order.  On equal values the lower index comes first,
 *            of groups as of experts.
 *   w      : scale * s, divided by the sum of the chosen s if renorm is 1
 *            (sigmoid: 0 where that sum is 0 in fp32; softmax: formed as the
 *            softmax over the chosen logits, which the bias may have chosen
 *            far below the largest, where s itself underflows).
 *   A token's results do not depend on the other tokens or their number.
 *   A masked expert is never chosen: with fewer candidates than k the last
 *   slots are idx = -1, w = 0.
 *   Requires 1 <= k <= experts, groups dividing experts, 1 <= top_groups <=
 *   groups, scale finite.  No alignment beyond the element's.
 *   Limits (FP8FG_EUNSUPPORTED): experts <= 1024, k <= 64; rows and pitches as
 *   above.
 */
FP8FG_API int fp8_route(const void* logits, int l_type, int64_t rows, int64_t experts,
              int64_t ldl, const float* bias, int score, int64_t groups,
              int64_t top_groups, int group_top, int64_t k, int renorm, float scale,
              int32_t* idx, int64_t ld_idx, float* w, int64_t ldw, void* stream);

/*
 * fp8_route_backward -- gradient of fp8_route's weights with respect to the
 * logits (the choice itself is constant, and the bias has no gradient).
 *
 *   idx    : the forward's indexes; entries outside [0, experts) have no
 *            part.  A row's other entries must be distinct.
 *   dw     : [rows][k] fp32, row pitch lddw.
 *   dlogits: [rows][experts] of l_type, row pitch lddl, overwritten.
 *   Other arguments and limits as for fp8_route.
 */
FP8FG_API int fp8_route_backward(const void* logits, int l_type, int64_t rows, int64_t experts,
                       int64_t ldl, int score, int64_t k, int renorm, float scale,
                       const int32_t* idx, int64_t ld_idx, const float* dw,
                       int64_t lddw, void* dlogits, int64_t lddl, void* stream);

/*
 * fp8_dispatch -- rows into expert order: the sorted activations and the
 * offsets that fp8_grouped_gemm_blockscaled takes ([hearaon]: activations
 * are quantized before they are dispatched to the experts).
 *
 *   idx    : DEVICE int32 [tokens][k], row pitch ld_idx: entry (t, j) goes to
 *            expert idx[t][j]; an index outside [0, experts) drops it.
 *   The entries are ordered by expert, within an expert by (t, j), dropped
 *   ones last.  Entry (t, j) being the r-th:
 *   offsets: int32 [experts + 1], entries of the experts below e; the last
 *            one counts the entries that are not dropped.
 *   pos    : int32 [tokens][k], contiguous: r, or -2 - r for a dropped entry.
 *   token  : int32 [tokens * k]: token[r] = t, or -1 for a dropped entry.
 *   x      : [tokens][cols] of x_type E4M3 (with 1x128 scales xs), BF16 or
 *            F32 (xs, os ignored), or null: the places alone.
 *   out, os: [tokens * k][cols] and its scales: out[r] = x[t]; zero bytes and
 *            the scale 2^-126 for a dropped entry.
 *   workspace: at least fp8_dispatch_workspace(tokens, k, experts) bytes,
 *            16-byte aligned; FP8FG_ESHAPE if workspace_bytes is less.
 *   Requires k >= 1, experts >= 1; with x, cols a multiple of 128 (E4M3) or
 *   8.  tokens == 0 writes zero offsets.
 *   Alignment: x, out 16-byte aligned, pitches multiples of 16 bytes; idx,
 *   offsets, pos, token, xs, os 4-byte aligned.
 *   Limits (FP8FG_EUNSUPPORTED): tokens * k <= 2^31 - 3 (the rows are int32),
 *   experts <= 1024, cols <= 2^28; pitches and scale strides as above.
 */
FP8FG_API int64_t fp8_dispatch_workspace(int64_t tokens, int64_t k, int64_t experts);
FP8FG_API int fp8_dispatch(const int32_t* idx, int64_t ld_idx, int64_t tokens, int64_t k,
                 int64_t experts, const void* x, int x_type, int64_t cols, int64_t ldx,
                 const float* xs, int64_t xs_rs, int64_t xs_ts, int32_t* offsets,
                 int32_t* pos, int32_t* token, void* out, int64_t ldo, float* os,
                 int64_t os_rs, int64_t os_ts, void* workspace, int64_t workspace_bytes,
                 void* stream);

/*
 * fp8_combine -- the experts' rows back in token order.
 *
 *   out[t][c] = base[t][c] + sum_j w[t][j] * z[pos[t][j]][c], in fp32 in the
 *   order of j, base last, rounded once to `type`; places outside [0, z_rows)
 *   have no part (their rows are not read).
 *   z, base, out: type BF16 or F32; base may be null (nothing is added), w
 *            too (ones: the gradient of fp8_dispatch).
 *   pos    : int32 [tokens][k], contiguous.
 *   Requires k >= 1, cols % 8 == 0.  Alignment: z, base, out 16-byte aligned,
 *   pitches multiples of 16 bytes; pos and w 4-byte aligned.
 *   Limits (FP8FG_EUNSUPPORTED): z_rows, tokens <= 2^31 - 1, k <= 2^31 - 16,
 *   cols <= 2^28; pitches as above.
 */
FP8FG_API int fp8_combine(const void* z, int type, int64_t z_rows, int64_t tokens, int64_t k,
                int64_t cols, int64_t ldz, const int32_t* pos, const float* w,
                int64_t ldw, const void* base, int64_t ldb, void* out, int64_t ldo,
                void* stream);

/*
 * fp8_combine_backward -- gradients of fp8_combine's z and w (base's is dy).
 *
 *   dz[pos[t][j]] = w[t][j] * dy[t],  dw[t][j] = sum_c dy[t][c] * z[pos[t][j]][c]
 *   for places in [0, z_rows); otherwise dw = 0, and if -2 - pos[t][j] is in
 *   [0, z_rows) (an entry that fp8_dispatch dropped) that row of dz is zeroed.
 *   With the places of one fp8_dispatch and z_rows = tokens * k every row of
 *   dz is written; rows that no place names are left as they are.  The
 *   places must be distinct.
 *   dw may be null (then z may be too); w may be null (ones).
 *   Other arguments, alignment and limits as for fp8_combine.
 */
FP8FG_API int fp8_combine_backward(const void* dy, int type, int64_t z_rows, int64_t tokens,
                         int64_t k, int64_t cols, int64_t lddy, const void* z,
                         int64_t ldz, const int32_t* pos, const float* w, int64_t ldw,
                         void* dz, int64_t lddz, float* dw, int64_t lddw, void* stream);

/*
 * fp8_swiglu_quantize -- the silu gate between the two products of an expert:
 * its result as the E4M3 operand of the second product, and its input kept
 * in E4M3 for the backward pass ([why-be]: E4M3 on all tensors, 1x128 tiles;
 * the gate's output is formed again from its input instead of being kept).
 *
 *   u      : [rows][2 inner] of u_type BF16 or F32, row pitch ldu: the gate g in
 *            the first inner columns, the linear half l in the others.
 *   a      = (g * sigmoid(g)) * l in fp32.  The sigmoid takes g below -87 for
 *            -87, so that |g * sigmoid(g)| stays at 1.5e-36 there; above 87 it is
 *            1.  Where a (or, in the functions below, a gradient) overflows,
 *            the amax rule's scale of the tile is infinite and its bytes mean
 *            nothing; the power-of-two rule's scale is 2^120, and the tile's
 *            infinite values saturate.  A quiet NaN in u or da (arithmetic makes
 *            no others) shows in every value that it enters (bytes 0x7F or 0xFF)
 *            and has no part in the scales.
 *   q, s   : E4M3 bytes [rows][inner] and 1x128 scales of the fp32 a, by the
 *            rules of fp8_quantize_rowtile
 *   uq, us : E4M3 bytes [rows][2 inner] and 1x128 scales of u; uq may be null
 *            (nothing is kept: serving), us is then ignored.
 *   used   : DEVICE int32, or null.  Rows from *used on are neither read nor
 *            written (offsets + G of the grouped GEMM, which leaves them alone
 *            too); held within [0, rows].
 *   A row's results do not depend on the other rows or their number.
 *   Requires inner % 128 == 0.  rows == 0 or inner == 0 is a valid no-op.
 *   Alignment: u, q, uq 16-byte aligned, their pitches multiples of 16 bytes;
 *   s, us, used 4-byte aligned.
 *   Limits (FP8FG_EUNSUPPORTED), here and in the two functions below: rows *
 *   inner / 128 <= 2^31, rows <= 2^31 - 1, inner <= 2^27; pitches and scale
 *   strides as above.
 */
FP8FG_API int fp8_swiglu_quantize(const void* u, int u_type, int64_t rows, int64_t inner,
                        int64_t ldu, const int32_t* used, int scale_rule, uint8_t* q,
                        int64_t ldq, float* s, int64_t s_rs, int64_t s_ts, uint8_t* uq,
                        int64_t lduq, float* us, int64_t us_rs, int64_t us_ts, void* stream);

/*
 * fp8_swiglu_backward -- gradient of the gate above from its 8-bit checkpoint,
 * passed straight through both quantizers.
 *
 *   g, l   = RN32(dec(uq) * us)
 *   dg     = da * l * sg * (1 + g * (1 - sg)),  dl = da * g * sg,
 *   a      = g * sg * l,  sg = sigmoid(g), in fp32
 *   da     : [rows][inner] of type BF16 or F32.
 *   dq, ds : E4M3 bytes [rows][2 inner] and 1x128 scales of [dg | dl] (the
 *            operand of the first product's data gradient); may be null.
 *   du     : [dg | dl] in da's type; may be null.
 *   a      : [rows][inner] in da's type, for the second product's weight
 *            gradient; may be null.  One of dq, du and a is needed.
 *   used, alignment and limits as above.
 */
FP8FG_API int fp8_swiglu_backward(const void* da, int type, int64_t rows, int64_t inner,
                        int64_t ldda, const uint8_t* uq, int64_t lduq, const float* us,
                        int64_t us_rs, int64_t us_ts, const int32_t* used, int scale_rule,
                        uint8_t* dq, int64_t lddq, float* ds, int64_t ds_rs, int64_t ds_ts,
                        void* du, int64_t lddu, void* a, int64_t lda, void* stream);

/*
 * fp8_swiglu_backward_128x1 -- the same gradient with the operands of both
 * weight gradients ([why-be] backward-pass paragraph: 1x128 -> 128x1 tiles),
 * formed from the fp32 values in the same pass.
 *
 *   dq, ds   : as above.
 *   dqt, dst : 128x1 tiles of [dg | dl], transposed: bytes [2 inner][rows],
 *              scales dst[c * dst_rs + (r / 128) * dst_ts]
 *   aqt, ast : 128x1 tiles of a, transposed: bytes [inner][rows]
 *   All are written.  Requires rows % 128 == 0 and inner % 128 == 0.  The rows
 *   are one expert's (a dense or shared one): there are no bounds, and a tile of
 *   128 rows that holds two experts' has one scale for both.
 *   Limits also: rows / 128 <= 65535.
 */
FP8FG_API int fp8_swiglu_backward_128x1(const void* da, int type, int64_t rows, int64_t inner,
                        int64_t ldda, const uint8_t* uq, int64_t lduq, const float* us,
                        int64_t us_rs, int64_t us_ts, int scale_rule, uint8_t* dq,
                        int64_t lddq, float* ds, int64_t ds_rs, int64_t ds_ts, uint8_t* dqt,
                        int64_t lddqt, float* dst, int64_t dst_rs, int64_t dst_ts,
                        uint8_t* aqt, int64_t ldaqt, float* ast, int64_t ast_rs,
                        int64_t ast_ts, void* stream);

/*
 * fp8_balance_loss -- the loss that keeps a router's experts evenly loaded over
 * each sequence of tokens, and the experts' counts.
 *
 *   logits : [rows][experts] of l_type, row pitch ldl, as fp8_route takes them;
 *            score is its score.  share[t][i] = s_i / sum_j s_j (softmax: s
 *            itself).  A logit of -inf or NaN masks its expert, whose share is
 *            0 (in a sigmoid's sums below 2^-124, as of any logit below -87);
 *            a token whose experts are all masked (padding) is not counted.
 *   idx    : int32 [rows][k], row pitch ld_idx, as fp8_route gives them;
 *            entries outside [0, experts) are not counted.
 *   offsets: DEVICE int32 [seqs + 1], nondecreasing (not checked; held within
 *            the rows): sequence s has the tokens [offsets[s], offsets[s + 1]);
 *            the others belong to none.  Null: all rows are one sequence, seqs 1.
 *   Over the n counted tokens of sequence s:
 *   counts : int32 [seqs][experts], contiguous: entries of idx that name i
 *   slope  : fp32 [seqs][experts], contiguous: scale * experts / (k n^2) *
 *            counts, which is d loss / d share; 0 for n == 0
 *   loss   : fp32 [seqs]: sum_i slope[s][i] * sum_t share[t][i]
 *   Sums are in a fixed order (fp32 within at most 4096 tokens, fp64 beyond).
 *   workspace: at least fp8_balance_loss_workspace(rows, experts, seqs) bytes,
 *            16-byte aligned; FP8FG_ESHAPE if workspace_bytes is less.
 *   Requires 1 <= k <= experts, scale finite; seqs == 0 is a no-op, rows == 0
 *   writes zeros.  No alignment beyond the element's.
 *   Limits (FP8FG_EUNSUPPORTED): experts <= 1024, k <= 64, seqs <= 2^31 - 1,
 *   rows * k <= 2^31 - 1 (the counts); rows and pitches as above.
 */
FP8FG_API int64_t fp8_balance_loss_workspace(int64_t rows, int64_t experts, int64_t seqs);
FP8FG_API int fp8_balance_loss(const void* logits, int l_type, int64_t rows, int64_t experts,
                     int64_t ldl, const int32_t* idx, int64_t ld_idx, int64_t k,
                     const int32_t* offsets, int64_t seqs, int score, float scale, float* loss,
                     int32_t* counts, float* slope, void* workspace, int64_t workspace_bytes,
                     void* stream);

/*
 * fp8_balance_loss_backward -- gradient of the loss with respect to the logits
 * (the counts are constant).
 *
 *   dloss  : fp32 [seqs], or null (ones).
 *   slope  : as the forward stored it.
 *   base   : [rows][experts] of l_type, added (the gradient of fp8_route's
 *            weights); may be null.
 *   dlogits: [rows][experts] of l_type, row pitch lddl, overwritten; base's row
 *            or zeros for a token in no sequence or with all experts masked.
 *   Other arguments and limits as above.
 */
FP8FG_API int fp8_balance_loss_backward(const float* dloss, const void* logits, int l_type,
                     int64_t rows, int64_t experts, int64_t ldl, const float* slope,
                     const int32_t* offsets, int64_t seqs, int score, const void* base,
                     int64_t ldb, void* dlogits, int64_t lddl, void* stream);

/*
 * fp8_rmsnorm_block_quantize -- from a block's output to the next block's input:
 * the norm after the block, its gate, the scaled residual addition and the next
 * norm with an E4M3 output.
 *
 *   rstd_post[m] = 1 / sqrt(sum_c z^2 / cols + eps)
 *   t[m][c]  = ((z * rstd_post) * gamma_post[c]) * gate, in fp32
 *   h[m][c]  = RN(residual_scale * r + block_scale * t) in x_type
 *   rstd, y, q, s: the norm of h with gamma, defined as fp8_rmsnorm_quantize's
 *            (its sums are in another order: last bits may differ)
 *
 *   z, r, h, y : x_type BF16 or F32 with row pitches ldz, ldr, ldh, ldy.  h is
 *            needed; y, q with s, rstd_post and rstd may be null.
 *   gamma_post, gamma : [cols], g_type BF16 or F32.
 *   gate     : null (1), one value per column (ldg == 0: [cols] of g_type) or
 *            rows (ldg >= cols: [rows][cols] of x_type).
 *   residual_scale, block_scale : finite.  eps, and rows beyond fp32's range,
 *            as for fp8_rmsnorm_quantize.
 *   A row's results do not depend on the other rows or their number.
 *   Requires cols % 128 == 0.  rows == 0 or cols == 0 is a valid no-op.
 *   Alignment: all but the scales, rstd_post and rstd (4 bytes) 16-byte
 *   aligned, pitches multiples of 16 bytes.
 *   Limits (FP8FG_EUNSUPPORTED): cols <= 16384; the others as for
 *   fp8_rmsnorm_quantize.
 */
FP8FG_API int fp8_rmsnorm_block_quantize(const void* z, int x_type, int64_t rows, int64_t cols,
                     int64_t ldz, const void* r, int64_t ldr, const void* gamma_post,
                     const void* gamma, int g_type, const void* gate, int64_t ldg,
                     float residual_scale, float block_scale, float eps, int scale_rule,
                     void* h, int64_t ldh, void* y, int64_t ldy, uint8_t* q, int64_t ldq,
                     float* s, int64_t s_rs, int64_t s_ts, float* rstd_post, float* rstd,
                     void* stream);

/*
 * fp8_rmsnorm_block_backward -- its gradient, passed straight through the
 * quantizer.
 *
 *   xh = h * rstd,  a = dy * gamma,  dH = rstd * (a - xh * mean_c(a * xh)) + dh
 *   zh = z * rstd_post,  b = block_scale * dH * gate
 *   dr = residual_scale * dH
 *   dz = rstd_post * (b * gamma_post - zh * mean_c(b * gamma_post * zh))
 *   dgamma[c] = sum_m dy * xh,  dgamma_post[c] = sum_m b * zh
 *   dgate = block_scale * dH * zh * gamma_post, for a gate per column summed over m
 *
 *   dy, dh, z, h, dz, dr : x_type.  dh (the gradient reaching h along the
 *            residual stream) may be null.
 *   rstd_post, rstd : as the forward stored them.
 *   dgamma_post, dgamma : fp32 [cols], overwritten (zeros for rows == 0).
 *   dgate    : needed with a gate: fp32 [cols] (ldg == 0; zeros for rows ==
 *            0) or [rows][cols] of x_type, row pitch lddg.
 *   workspace: at least fp8_rmsnorm_block_backward_workspace(rows, cols) bytes,
 *            16-byte aligned: partial sums over the rows, added in a fixed
 *            order.  FP8FG_ESHAPE if workspace_bytes is less.
 *   Requires cols % 8 == 0.  Alignment and limits as above.
 */
FP8FG_API int64_t fp8_rmsnorm_block_backward_workspace(int64_t rows, int64_t cols);
FP8FG_API int fp8_rmsnorm_block_backward(const void* dy, int x_type, int64_t rows, int64_t cols,
                     int64_t lddy, const void* dh, int64_t lddh, const void* z, int64_t ldz,
                     const void* h, int64_t ldh, const void* gamma_post, const void* gamma,
                     int g_type, const void* gate, int64_t ldg, const float* rstd_post,
                     const float* rstd, float residual_scale, float block_scale, void* dz,
                     int64_t lddz, void* dr, int64_t lddr, float* dgamma_post, float* dgamma,
                     void* dgate, int64_t lddg, void* workspace, int64_t workspace_bytes,
                     void* stream);

/* Static, thread-safe description of a status code. */
FP8FG_API const char* fp8fg_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FP8FG_H */

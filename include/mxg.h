/*
 * mxg.h -- C ABI of the GB300 (sm_103a) grouped block-scaled quantize +
 * grouped GEMM library (libmxg.so).
 *
 * The operations follow three public pages:
 *   [TE-gemm]  TransformerEngine transformer_engine/jax/cpp_extensions/gemm.py
 *              (commit 070b5b7): swizzled_scale, grouped_gemm,
 *              _jax_scaled_matmul, _get_nvfp4_tensor_scale_inv.
 *   [PR2763]   TransformerEngine PR #2763 "[JAX] MXFP8 Grouped Quant+GEMM".
 *   [PR3661]   TransformerEngine PR #3661 "Add row-scaled NVFP4 support to
 *              grouped-tensor GEMM".
 *
 * Conventions for every entry point
 *   - All buffers are caller-owned DEVICE memory unless stated otherwise.
 *     The library never allocates, frees or synchronises on these calls, so
 *     each of them may be captured in a CUDA graph.
 *   - Work is enqueued on `stream` (NULL = the legacy default stream).
 *   - Host-detectable errors (null pointers, sizes, alignment, unsupported
 *     combinations, a device that is not sm_103) are returned synchronously
 *     and nothing is launched.  MXG_ERR_LAUNCH reports a failed launch.
 *   - Data-dependent errors cannot be known on the host without a sync; the
 *     kernels record them in a caller-owned sticky device word `dev_status`
 *     (int32, atomicOr of the MXG_DEV_* bits) and clamp so that no access
 *     leaves the buffers.  Read it after the stream or graph has completed.
 *     `dev_status` may be NULL (then nothing is recorded).
 *   - Rows are dense (a [rows, cols] matrix has leading dimension cols),
 *     except the GEMM operands' data, whose leading dimension the operand
 *     descriptor gives.
 *   - bf16 is IEEE bfloat16 stored as uint16; E4M3 is the "fn" variant.
 *   - The grouped matrices are 128-row aligned: every group size, K, N and
 *     rows_capacity is a multiple of 128 (the alignment [PR2763] states for
 *     the grouped quantize and GEMM setup kernels).
 */
#ifndef MXG_H_
#define MXG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* CUDA stream handle (same type as cudaStream_t / CUstream). */
struct CUstream_st;
typedef struct CUstream_st* mxg_stream_t;

typedef enum {
  MXG_OK = 0,
  MXG_ERR_INVALID_ARG = 1,         /* null pointer, bad size or enum value      */
  MXG_ERR_ALIGNMENT = 2,           /* size not a multiple of 128, pointer not   */
                                   /* 16-byte aligned                           */
  MXG_ERR_UNSUPPORTED_ARCH = 3,    /* current device is not sm_103 (GB300)      */
  MXG_ERR_LAUNCH = 4,              /* the CUDA launch failed                    */
  MXG_ERR_WORKSPACE_TOO_SMALL = 5, /* workspace smaller than the size query     */
  MXG_ERR_UNSUPPORTED = 6          /* valid but not implemented combination     */
} mxg_status_t;

/* Sticky device status bits (atomicOr into dev_status). */
#define MXG_DEV_NEG_SIZE 1          /* a group size was negative: used as 0       */
#define MXG_DEV_MISALIGNED 2        /* a group size was not a multiple of 128:    */
                                    /* rounded down                               */
#define MXG_DEV_SUM_OVER_CAPACITY 4 /* the sizes summed past rows_capacity: the   */
                                    /* rows beyond it were dropped                */
#define MXG_DEV_BOUNDS 8            /* an index check failed (debug builds)       */
#define MXG_DEV_TIMEOUT 16          /* a pipeline wait ran out; the kernel gave   */
                                    /* up on its tile and returned                */

typedef enum {
  MXG_MXFP8_E4M3 = 1,     /* E4M3 data, one E8M0 scale per 1x32 block          */
  MXG_NVFP4_ROWSCALED = 2 /* E2M1 data, one E4M3 scale per 1x16 block, plus an  */
                          /* FP32 outer scale per row                           */
} mxg_format_t;

typedef enum { MXG_ROWWISE = 1, MXG_COLWISE = 2, MXG_BOTH = 3 } mxg_qlayout_t;

typedef enum {
  MXG_FPROP_TN = 0, /* ragged output rows:  C[M_cap, N] = X[M_cap, K] . W[g]^T  */
  MXG_WGRAD_NT = 1, /* ragged contraction:  dW[G, N, K] = dY_g^T . X_g          */
  MXG_DGRAD_NN = 2  /* ragged output rows:  dX[M_cap, K] = dY[M_cap, N] . W[g]  */
} mxg_gemm_mode_t;

typedef enum { MXG_OUT_F32 = 0, MXG_OUT_BF16 = 1 } mxg_out_t;

/* One quantized GEMM operand: rowwise-quantized rows of the contraction dim
 * ([PR2763] GEMM-setup review thread: per-group operand pointers come from
 * the offsets and the leading dimensions).
 *   data  : E4M3 bytes [rows, cols] (MXFP8) or packed E2M1 [rows, cols/2]
 *           (NVFP4, element 2i in the low nibble of byte i), consecutive rows
 *           ld elements apart.
 *   scale : block scales in the swizzled layout of [TE-gemm] swizzled_scale
 *           for the [rows, cols/32] (MXFP8) or [rows, cols/16] (NVFP4) scale
 *           matrix: 128x4 tiles of 512 contiguous bytes, byte
 *           ((r/128 * C/4 + c/4) * 32 + r%32) * 16 + (r%128)/32 * 4 + c%4.
 *           Always dense (the swizzle fixes its layout).
 *   outer : NVFP4 only: FP32 outer scale per row [rows]; NULL for MXFP8.
 *   rows, cols : the operand's rows and contraction length in elements, as
 *           the GEMM mode implies them (listed at mxg_grouped_gemm); 0 means
 *           "as implied" (no check), any other value must match.
 *   ld    : elements from one row of data to the next; 0 means cols (dense).
 *           Otherwise ld >= cols and ld bytes (ld for MXFP8, ld/2 for NVFP4,
 *           ld even) a multiple of 16, so that an operand can be a view of
 *           rows inside a wider buffer.
 * data and scale must be 16-byte aligned. */
typedef struct {
  const void* data;
  const uint8_t* scale;
  const float* outer;
  int64_t rows;
  int64_t cols;
  int64_t ld;
} mxg_operand_t;

/* ------------------------------------------------------------------------- */
/* Group sizes -> int64 sizes + element offsets ([PR2763] description: int32 */
/* sizes widened to int64 with a multiplier; offsets-kernel review thread:   */
/* exclusive prefix sum of size * last_dim, G+1 values; workspace review     */
/* thread: layout [G int64 sizes | G+1 int64 offsets]).                      */
/* ------------------------------------------------------------------------- */

/* Bytes of the offsets workspace: (2G + 1) * 8.  Returns 0 if G < 1. */
size_t mxg_offsets_workspace_bytes(int G);

/* sizes          : device int32[G] (sizes_is_int64 = 0) or int64[G] (= 1).
 * multiplier     : rows per size unit (1 when sizes are row counts).
 * last_dim       : elements per row, used for the element offsets.
 * rows_capacity  : rows of the buffers the groups live in.
 * ws             : device int64[2G+1]; written as
 *                  ws[g] = s_g (sanitised rows of group g),
 *                  ws[G] = 0, ws[G+1+g] = ws[G+g] + s_g * last_dim.
 * Sanitisation (recorded in dev_status): a negative size counts as 0
 * (NEG_SIZE); a size not a multiple of 128 is rounded down (MISALIGNED);
 * rows past rows_capacity are dropped (SUM_OVER_CAPACITY).
 * A size times the multiplier is formed exactly (no 64-bit overflow): a
 * product past rows_capacity is clamped to it.
 * Errors: MXG_ERR_INVALID_ARG for null sizes/ws, G < 1 or G > 65536,
 * multiplier < 1 or > 2^31, last_dim < 1, rows_capacity < 0 or > 2^62, or
 * rows_capacity * last_dim beyond int64. */
mxg_status_t mxg_group_offsets(const void* sizes, int sizes_is_int64, int G, int64_t multiplier,
                               int64_t last_dim, int64_t rows_capacity, int64_t* ws,
                               int32_t* dev_status, mxg_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Grouped quantize with the swizzled scale layout written directly         */
/* ([PR2763] description: swizzle fused into the grouped quantize;          */
/* [PR3661] description: row-scaled NVFP4 cast writes swizzled scales).     */
/* ------------------------------------------------------------------------- */
/* x             : bf16 [rows_capacity, cols], 16-byte aligned.
 * group_ws      : offsets workspace from mxg_group_offsets (its first G
 *                 entries are the rows of each group); the live rows are
 *                 their sum, clamped to rows_capacity.  NULL: all
 *                 rows_capacity rows are live (weights, [TE-gemm]
 *                 grouped_gemm quantizes the kernel with no group sizes).
 * Rows at or beyond the live count are neither read nor written.
 *
 * MXG_MXFP8_E4M3, rowwise (layout ROWWISE or BOTH):
 *   q_row  : E4M3 [rows_capacity, cols]
 *   sf_row : E8M0 swizzled [rows_capacity, cols/32]; group g's scales start
 *            at byte row_off_g * cols / 32 ([PR2763]: scale offset = data
 *            offset / 32).
 *   Per 1x32 block: amax -> e = ceil(log2(amax / 448)) clamped to
 *   [-127, 127] (all-zero block: e = -127), byte e + 127, data
 *   E4M3_RNE(x * 2^-e).
 * MXG_MXFP8_E4M3, colwise (layout COLWISE or BOTH), written transposed:
 *   q_col  : E4M3 [cols, rows_capacity], q_col[k, m] = Q(x[m, k]) over
 *            32x1 blocks along rows
 *   sf_col : E8M0 swizzled [cols, rows_capacity/32] ([TE-gemm]
 *            swizzled_scale, colwise: the scale matrix is transposed first).
 * MXG_NVFP4_ROWSCALED, rowwise (layout ROWWISE or BOTH):
 *   q_row     : packed E2M1 [rows_capacity, cols/2]
 *   sf_row    : E4M3 swizzled [rows_capacity, cols/16]
 *   outer_row : FP32 [rows_capacity], s_r = amax_r / 2688
 *               ([TE-gemm] _get_nvfp4_tensor_scale_inv: amax / (6 * 448)).
 *   Per 1x16 block, fp32 round-to-nearest steps: S = 2688 / amax_r,
 *   sb = E4M3_RNE_satfinite((amax_b / 6) * S), code =
 *   E2M1_RNE_satfinite(x * (S / sb)) (signed zeros when sb or amax_r is 0).
 * MXG_NVFP4_ROWSCALED, colwise (layout COLWISE or BOTH), written transposed
 * for wgrad ([PR3661]: columnwise amax per column, split per expert):
 *   q_col     : packed E2M1 [cols, rows_capacity/2]; byte q_col[k, m/2] holds
 *               rows m (low nibble) and m+1 of column k
 *   sf_col    : E4M3 swizzled [cols, rows_capacity/16] (16-row blocks)
 *   outer_col : FP32 [G, cols] (G = 1 when group_ws is NULL):
 *               A[g, k] / 2688 with A the amax of column k over group g's
 *               rows; the same block rule as rowwise runs down the column.
 *               Groups with no rows get 0.  Requires G <= 1024.
 * Unused output pointers may be NULL.
 * Errors: INVALID_ARG (null required pointer, bad enum, NVFP4 colwise with
 * G > 1024), ALIGNMENT (rows_capacity or cols not a multiple of 128, pointer
 * not 16-byte aligned), UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_group_quantize(mxg_format_t fmt, mxg_qlayout_t layout, const void* x,
                                int64_t rows_capacity, int64_t cols, const int64_t* group_ws,
                                int G, void* q_row, uint8_t* sf_row, void* q_col, uint8_t* sf_col,
                                float* outer_row, float* outer_col, int32_t* dev_status,
                                mxg_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Grouped block-scaled GEMM ([TE-gemm] grouped_gemm; [PR2763] V2 grouped    */
/* GEMM consuming pre-swizzled scales; [PR3661] row-scaled NVFP4: neutral    */
/* outer scales, FP32 accumulation, outer scales applied afterwards).       */
/* ------------------------------------------------------------------------- */
/* MXG_FPROP_TN (ragged rows):
 *   A = activations, rowwise: data [M_cap, K]; B = weights, rowwise:
 *   data [G*N, K] (expert g owns rows g*N .. g*N+N-1).
 *   C[off_g + i, n] = alpha_g * sum_k A[off_g+i, k] * B[g*N+n, k]
 *                     + beta_g * C[off_g + i, n];   C is [M_cap, N].
 *   Rows of C at or beyond the live count are not written.
 *   NVFP4: A.outer [M_cap] and B.outer [G*N] are required, and the result is
 *   multiplied by A.outer[row] * B.outer[g*N + n].
 * MXG_WGRAD_NT (ragged contraction; MXFP8, or row-scaled NVFP4 whose
 * operands are the colwise copies with A.outer = dY's outer_col [G, N] and
 * B.outer = X's outer_col [G, K], applied as
 * dW[g, n, k] *= A.outer[g, n] * B.outer[g, k]):
 *   A = colwise copy of dY: data [N, M_cap], scale [N, M_cap/32];
 *   B = colwise copy of X:  data [K, M_cap], scale [K, M_cap/32].
 *   dW[g, n, k] = alpha_g * sum_{m in group g} A[n, m] * B[k, m]
 *                 + beta_g * dW[g, n, k];   C = dW is [G, N, K].
 *   An empty group writes beta_g * dW[g] (zeros when beta is NULL or
 *   beta_g is 0).  With M_cap = 0 every group is empty and A and B are not
 *   read (their pointers must still be non-NULL).
 * MXG_DGRAD_NN (ragged rows, weights not transposed, MXFP8; [TE-gemm]
 * _quantize_gemm_operands: an RHS whose contraction dim is not last is
 * quantized colwise):
 *   A = rowwise dY: data [M_cap, N], scale [M_cap, N/32];
 *   B = colwise copy of W viewed as [G*N, K]: data [K, G*N], scale
 *       [K, G*N/32] (mxg_group_quantize(MXFP8, COLWISE, W, G*N, K, NULL, ...)).
 *   dX[off_g + i, k] = alpha_g * sum_n A[off_g+i, n] * B[k, g*N + n]
 *                      + beta_g * dX[off_g + i, k];   C = dX is [M_cap, K].
 * M_cap = 0: fprop and dgrad have no output rows and launch nothing.
 * group_ws : offsets workspace of mxg_group_offsets (first G entries used).
 * alpha, beta : device float[G] or NULL (alpha = 1, beta = 0).
 * bias  : device float [G, N] (fprop) or [G, K] (dgrad), or NULL: per-group
 *         bias ([TE-gemm] grouped_gemm: bias of shape (G, N)); the output is
 *         alpha_g * acc + bias[g, col] + beta_g * C.  Rejected for wgrad.
 * workspace : not needed by this implementation (size query returns 0);
 *             may be NULL.
 * Accumulation is FP32 in tensor memory; the FP32 output is the parity
 * output, bf16 is rounded to nearest even from it.
 * Operand shapes (rows x cols of mxg_operand_t, checked when nonzero):
 *   FPROP_TN: A M_cap x K, B G*N x K;  WGRAD_NT: A N x M_cap, B K x M_cap;
 *   DGRAD_NN: A M_cap x N, B K x G*N.
 * Errors: INVALID_ARG (nulls, G < 1 or G > 1024, NVFP4 dgrad, beta with
 * NVFP4 -- rejected as on [PR3661] --, an operand's rows or cols not the
 * mode's, ld < cols), ALIGNMENT (M_cap, N, K not multiples of 128;
 * data/scale/C not 16-byte aligned; ld bytes not a multiple of 16),
 * UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_grouped_gemm(mxg_format_t fmt, mxg_gemm_mode_t mode, const mxg_operand_t* A,
                              const mxg_operand_t* B, const int64_t* group_ws, int G,
                              int64_t M_cap, int64_t N, int64_t K, const float* alpha,
                              const float* beta, const float* bias, void* C, mxg_out_t out_type,
                              void* workspace, size_t workspace_bytes, int32_t* dev_status,
                              mxg_stream_t stream);

/* Test entry point (no counterpart on the pages): mxg_grouped_gemm with the
 * kernel choices that the parity tests need to reach every variant, and a
 * hook for the failure path of the bounded pipeline waits.  Same arguments
 * and checks as mxg_grouped_gemm, plus:
 *   tile_n          : 0 -- the default kernel choice (the CTA-pair kernel
 *                     with 256 x 256 units when B has at least 256 rows);
 *                     256 or 128 -- the single-CTA kernel with 128 x 256 or
 *                     128 x 128 tiles (256 only where the output width is a
 *                     multiple of 256, else 128).
 *   stage_bytes     : 0 -- default; 128 -- 128 bytes of K per pipeline stage
 *                     where the default takes 256 (MXFP8 fprop, K % 256 == 0).
 *   inject_flags    : bit 0 -- CTA 0 withholds the arrival that tells its
 *                     epilogue that its first accumulator is ready, so the
 *                     epilogue's wait runs out; 0 -- a normal run.
 *   wait_timeout_ns : bound on every pipeline wait, in ns (0 = 1 s default).
 * With bit 0 set the launch ends with MXG_DEV_TIMEOUT in dev_status, the
 * affected CTA drains its copies and MMAs, frees its tensor memory and
 * returns; the output is undefined and the device stays usable.
 * Errors: as mxg_grouped_gemm, plus INVALID_ARG for another tile_n or
 * stage_bytes value or unknown inject bits. */
mxg_status_t mxg_grouped_gemm_debug(mxg_format_t fmt, mxg_gemm_mode_t mode, const mxg_operand_t* A,
                                    const mxg_operand_t* B, const int64_t* group_ws, int G,
                                    int64_t M_cap, int64_t N, int64_t K, const float* alpha,
                                    const float* beta, const float* bias, void* C,
                                    mxg_out_t out_type, int32_t* dev_status, int tile_n,
                                    int stage_bytes, int inject_flags, int64_t wait_timeout_ns,
                                    mxg_stream_t stream);

/* Workspace bytes mxg_grouped_gemm needs (0 for every combination here). */
size_t mxg_grouped_gemm_workspace_bytes(mxg_format_t fmt, mxg_gemm_mode_t mode, int G,
                                        int64_t M_cap, int64_t N);

/* ------------------------------------------------------------------------- */
/* Group sizes that are not multiples of 128 (MXFP8).  [PR2763] review       */
/* thread on the V2 alignment rule: the 128-row requirement comes from how   */
/* the grouped quantize and the GEMM setup compute per-group scale offsets,  */
/* not from the GEMM; [TE-gemm] grouped_gemm: padding belongs to the group   */
/* and is zero-filled so that it does not change the result; [TE-gemm]      */
/* apply_padding_to_scale_inv pads scale matrices of non-128 dims.  Here     */
/* each group's scales, and its slab of a colwise copy, are padded to a      */
/* multiple of 128 rows with zeros; rowwise data stays dense.                */
/* ------------------------------------------------------------------------- */

/* Rows of the padded layouts: rows_capacity + 128 * G (an upper bound on
 * the sum over groups of each group's rows rounded up to 128).  Returns 0
 * if rows_capacity < 0 or G < 1. */
int64_t mxg_unaligned_rows_capacity(int64_t rows_capacity, int G);

/* As mxg_group_offsets, but sizes are kept as given: no rounding and no
 * MISALIGNED bit (negative sizes and rows past rows_capacity are sanitised
 * as there).  Same workspace layout. */
mxg_status_t mxg_group_offsets_unaligned(const void* sizes, int sizes_is_int64, int G,
                                         int64_t multiplier, int64_t last_dim,
                                         int64_t rows_capacity, int64_t* ws, int32_t* dev_status,
                                         mxg_stream_t stream);

/* MXFP8 grouped quantize for groups of any size.  group_ws (required) is a
 * workspace of mxg_group_offsets_unaligned; group g owns data rows
 * [row_off_g, row_off_g + M_g) and padded rows [prow_off_g, prow_off_g +
 * P_g) with P_g = M_g rounded up to 128 and prow_off the prefix sum of P.
 * With R_pad = mxg_unaligned_rows_capacity(rows_capacity, G):
 *   q_row  : E4M3 [rows_capacity, cols], dense (row r of group g at row_off_g + r);
 *   sf_row : E8M0 swizzled [R_pad, cols/32]; group g's scale rows start at
 *            prow_off_g; its padding rows get byte 0;
 *   q_col  : E4M3 [cols, R_pad], transposed; group g's slab is columns
 *            [prow_off_g, prow_off_g + P_g), its padding columns 0x00;
 *   sf_col : E8M0 swizzled [cols, R_pad/32]; 32-row blocks start at each
 *            group's first row (a block never spans two groups).
 * Each group is quantized as if it were its own tensor, zero-padded to P_g
 * rows, with the block rules of mxg_group_quantize.  Rows and columns past
 * the padded groups are not written.  Unused output pointers may be NULL.
 * Errors: INVALID_ARG (null x or group_ws, G < 1 or G > 1024, bad layout,
 * null required output, rows_capacity + 128 * G above 2^31 - 128),
 * ALIGNMENT (rows_capacity or cols not multiples of 128, pointers not
 * 16-byte aligned), UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_group_quantize_unaligned(mxg_qlayout_t layout, const void* x,
                                          int64_t rows_capacity, int64_t cols,
                                          const int64_t* group_ws, int G, uint8_t* q_row,
                                          uint8_t* sf_row, uint8_t* q_col, uint8_t* sf_col,
                                          int32_t* dev_status, mxg_stream_t stream);

/* MXFP8 grouped GEMM for groups of any size (operands from
 * mxg_group_quantize_unaligned, weights from mxg_group_quantize).  Same
 * formulas, arguments and epilogue as mxg_grouped_gemm, with group_ws from
 * mxg_group_offsets_unaligned and these operand shapes (R_pad as above):
 *   FPROP_TN : A data [M_cap, K] dense, A scale [R_pad, K/32] padded;
 *   WGRAD_NT : A = dY colwise [N, R_pad] + [N, R_pad/32], B = X colwise
 *              [K, R_pad] + [K, R_pad/32]; each group contracts over its
 *              padded slab (the zero padding adds nothing);
 *   DGRAD_NN : A data [M_cap, N] dense, A scale [R_pad, N/32] padded
 *              (WGRAD_NT operands are R_pad columns long).
 * Output rows are the dense data rows; rows past a group are not written.
 * Errors: as mxg_grouped_gemm, plus INVALID_ARG when B has fewer than 256
 * rows (G * N for fprop, K otherwise) or M_cap + 128 * G exceeds 2^31 - 128. */
mxg_status_t mxg_grouped_gemm_unaligned(mxg_gemm_mode_t mode, const mxg_operand_t* A,
                                        const mxg_operand_t* B, const int64_t* group_ws, int G,
                                        int64_t M_cap, int64_t N, int64_t K, const float* alpha,
                                        const float* beta, const float* bias, void* C,
                                        mxg_out_t out_type, int32_t* dev_status,
                                        mxg_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Dequantize ([PR2763] dequantizer: inverse swizzle of the scales, then    */
/* data * scale).  Test helper; not on the timed path.                      */
/* ------------------------------------------------------------------------- */
/* ROWWISE: q [rows, cols] (NVFP4: [rows, cols/2]), sf swizzled [rows,
 *          cols/32 or cols/16], outer [rows] (NVFP4) -> out [rows, cols].
 * COLWISE: (MXFP8 only) q is the transposed copy [cols, rows], sf swizzled
 *          [cols, rows/32] -> out [rows, cols] (transposed back).
 * out is FP32 or bf16 (round to nearest even).
 * Errors: INVALID_ARG, ALIGNMENT (rows or cols not multiples of 128),
 * UNSUPPORTED (NVFP4 colwise), UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_dequantize(mxg_format_t fmt, mxg_qlayout_t layout, const void* q,
                            const uint8_t* sf, const float* outer, int64_t rows, int64_t cols,
                            void* out, mxg_out_t out_type, mxg_stream_t stream);

/* ------------------------------------------------------------------------- */
/* 16-bit operators of an expert block: the grouped products on bf16 or fp16 */
/* tensors, the norms around the block with its gate and residual, and the   */
/* clipping of the gradients.                                                */
/* ------------------------------------------------------------------------- */

typedef enum { MXG_F32 = 0, MXG_BF16 = 1, MXG_F16 = 2 } mxg_dtype_t;

/* Grouped products on 16-bit operands as they are: no quantization, no
 * transposed copies.  in_type is MXG_BF16 or MXG_F16 (A and B alike).  Group g
 * owns rows off_g .. off_g + M_g - 1 of the ragged matrices; sizes of any
 * value >= 0 (a workspace of either offsets entry point).
 *   MXG_FPROP_TN : A = X [M_cap, K], B = W [G, N, K], C [M_cap, N]:
 *     C[off_g+i, n] = alpha_g sum_k A[off_g+i, k] B[g, n, k] + beta_g C[off_g+i, n]
 *   MXG_DGRAD_NN : A = dY [M_cap, N], B = W [G, N, K], C = dX [M_cap, K]:
 *     C[off_g+i, k] = alpha_g sum_n A[off_g+i, n] B[g, n, k] + beta_g C[off_g+i, k]
 *   MXG_WGRAD_NT : A = dY [M_cap, N], B = X [M_cap, K], C = dW [G, N, K]:
 *     C[g, n, k] = alpha_g sum_{i in g} A[off_g+i, n] B[off_g+i, k] + beta_g C[g, n, k]
 *     (an empty group writes beta_g C[g], or zeros).
 * Sums are FP32; the result is rounded once, to out_type: MXG_F32 or in_type.
 * The tensor cores add by truncation: an FP32 result takes over their sums every
 * 512 products and adds those rounding to nearest, a 16-bit one (whose own
 * rounding is larger) is the whole contraction's truncated sum.
 * G, N, K >= 1 of any value; G <= 1024; M_cap >= 0 (with 0 the pointers of
 * the ragged matrices may be NULL).
 * lda, ldb, ldc : elements from one row to the next, 0 for dense rows; W and
 *             dW hold N rows per expert without a gap (expert stride N * ld).
 * A, B      : 16-byte aligned, lda and ldb multiples of 8 (so dense operands
 *             need N and K that are).  C: aligned to its element, any ldc.
 * alpha, beta : device float[G] or NULL (1 and 0).  C is read only where
 *             beta_g is not 0.
 * Rows of the ragged operands at or beyond the live count take no part, and
 * rows of a ragged C there are not written; a NaN or infinity in one group's
 * rows reaches no other group.  Negative sizes count as 0 and rows past M_cap
 * are dropped, each recorded in dev_status (as is TIMEOUT, a pipeline wait that
 * ran out).
 * Errors: INVALID_ARG (nulls, sizes, types, a leading dimension below its row),
 * ALIGNMENT, UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_grouped_gemm_16bit(mxg_dtype_t in_type, mxg_gemm_mode_t mode, const void* A,
                                    int64_t lda, const void* B, int64_t ldb,
                                    const int64_t* group_ws, int G, int64_t M_cap, int64_t N,
                                    int64_t K, const float* alpha, const float* beta, void* C,
                                    int64_t ldc, mxg_dtype_t out_type, int32_t* dev_status,
                                    mxg_stream_t stream);

/* How a block's gate is laid out. */
typedef enum {
  MXG_GATE_NONE = 0, /* no gate                                                */
  MXG_GATE_ROW = 1,  /* float [rows]: one per token (a router's weight)        */
  MXG_GATE_COL = 2,  /* dtype [cols]: one per channel                          */
  MXG_GATE_FULL = 3  /* dtype [rows, cols]                                     */
} mxg_gate_t;

/* The norms after and before a residual block in one pass:
 *   after  : x' = x + res_scale * gate . (y * ry . w_post)
 *   before : n  = x' * rx . w_pre
 * with ry = 1 / sqrt(mean(y^2) + eps) over the row's cols, and rx likewise of
 * x'.  Without y there is no "after" part (x' = x); without n_out no "before".
 *   dtype     : type of y, n_out, the weights and the COL / FULL gate
 *   res_dtype : type of the residual stream x, x_out: dtype or MXG_F32
 *   ld*       : elements between rows, 0 for cols
 *   w_post, w_pre : [cols], or NULL for ones
 *   x_out     : required with y; may be x itself (with the same ld)
 * n is formed from x' before x' is rounded.  1 <= cols <= 16384, rows >= 0
 * (0 launches nothing; the [rows, cols] pointers may then be NULL), eps > 0.  Sums
 * are FP32.  Any element alignment; rows that start on 16 bytes with cols a
 * multiple of 8 take 16-byte accesses. */
typedef struct {
  mxg_dtype_t dtype, res_dtype;
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  const void* y;
  int64_t ldy;
  const void* w_post;
  const void* gate;
  int64_t ldg;
  mxg_gate_t gate_mode;
  float res_scale;
  void* x_out;
  int64_t ldxo;
  const void* w_pre;
  void* n_out;
  int64_t ldn;
  float eps;
} mxg_block_norm_t;

/* Errors: INVALID_ARG (nulls, sizes, types, eps, a leading dimension below
 * cols, neither y nor n_out), ALIGNMENT (a pointer not aligned to its
 * element), UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_block_norm(const mxg_block_norm_t* desc, mxg_stream_t stream);

/* The gradients of mxg_block_norm.  x is the block's output x' as
 * mxg_block_norm stored it (x itself without y); dx_out is the gradient with
 * respect to x' (NULL: zero), dn the one with respect to n (NULL: no "before"
 * part); at least one of them is given.
 *   dx [rows, cols] of res_dtype : gradient of x; may be dx_out itself
 *   dy [rows, cols] of dtype     : gradient of y, required with y; may be y or dn
 *   dw_post, dw_pre : float [cols] or NULL
 *   dgate : float [rows] (ROW), float [cols] (COL), dtype [rows, cols] (FULL,
 *           ld lddg), or NULL.  The sums over rows have a fixed order.
 * x may be NULL without dn.  rows = 0 writes zeros to dw_post, dw_pre and a COL
 * dgate. */
typedef struct {
  mxg_dtype_t dtype, res_dtype;
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  const void* y;
  int64_t ldy;
  const void* w_post;
  const void* gate;
  int64_t ldg;
  mxg_gate_t gate_mode;
  float res_scale;
  const void* w_pre;
  float eps;
  const void* dx_out;
  int64_t lddxo;
  const void* dn;
  int64_t lddn;
  void* dx;
  int64_t lddx;
  void* dy;
  int64_t lddy;
  float* dw_post;
  float* dw_pre;
  void* dgate;
  int64_t lddg;
} mxg_block_norm_grad_t;

/* Bytes of the backward workspace (0 for sizes that the call refuses: rows < 0,
 * cols < 1 or > 16384); 16-byte aligned device memory whose contents mean nothing
 * before or after the call. */
size_t mxg_block_norm_workspace_bytes(int64_t rows, int64_t cols);

/* Errors: as mxg_block_norm, plus WORKSPACE_TOO_SMALL. */
mxg_status_t mxg_block_norm_backward(const mxg_block_norm_grad_t* desc, void* workspace,
                                     size_t workspace_bytes, mxg_stream_t stream);

/* One gradient of a list: numel elements of src_type at src and, for clipping,
 * of dst_type at dst (src itself is allowed with the same type; dst otherwise
 * overlaps no src of the list). */
typedef struct {
  const void* src;
  void* dst;
  int64_t numel;
  mxg_dtype_t src_type, dst_type;
} mxg_grad_t;

/* Bytes of the workspace of the two calls below (16-byte aligned device
 * memory, contents meaningless before and after). */
size_t mxg_grad_workspace_bytes(void);

/* norm[0] = sqrt(sum over the list of g^2): the L2 norm of all gradients as
 * one vector.  `grads` is a HOST array, read before the call returns; n = 0 or
 * empty tensors give 0.  Squares are summed in FP32 over short runs and in
 * FP64 from there on, in a fixed order; magnitudes anywhere in FP32's range
 * neither overflow nor vanish on the way (the norm itself can pass FP32's).
 * Errors: INVALID_ARG (nulls, n < 0, numel < 0 or > 2^40, types), ALIGNMENT
 * (a tensor not aligned to its element, workspace), WORKSPACE_TOO_SMALL,
 * UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_grad_norm(const mxg_grad_t* grads, int n, float* norm, void* workspace,
                           size_t workspace_bytes, mxg_stream_t stream);

/* The same norm, and dst = src * min(1, max_norm / (norm + 1e-6)) for every
 * tensor, also where the norm or the factor leaves FP32's range.  max_norm >= 0;
 * with an infinite one the factor is 1, whatever the norm.  With a finite one an
 * infinite gradient gives factor 0 (and NaN where 0 meets the infinity).  A NaN makes
 * every output NaN.  Errors: as mxg_grad_norm. */
mxg_status_t mxg_grad_clip(const mxg_grad_t* grads, int n, float max_norm, float* norm,
                           void* workspace, size_t workspace_bytes, mxg_stream_t stream);

/* ------------------------------------------------------------------------- */
/* Around the products of an expert block: the routing of tokens to experts  */
/* with its balance loss, the rows moved there and back, and the gated       */
/* activation between the products with its inputs kept in 8 bits.           */
/* ------------------------------------------------------------------------- */

/* What a router's logit l becomes: MXG_SCORE_SOFTMAX: s_e = exp(l_e) / sum_i
 * exp(l_i); MXG_SCORE_SIGMOID: s_e = 1 / (1 + exp(-l_e)). */
typedef enum { MXG_SCORE_SOFTMAX = 0, MXG_SCORE_SIGMOID = 1 } mxg_score_t;

/* Routing of `tokens` tokens to k of `experts` experts each, with the counts,
 * the balance loss and, where wanted, the rows that the tokens take.
 *   logits : [tokens, experts] of dtype, ld elements between rows (0: dense)
 *   mask   : uint8 [tokens], 0 for a token that takes no part (padding), or NULL
 * For each token the k experts of the largest logits, in falling order; the
 * lower expert first where logits are equal (-0 equals 0), NaN above infinity.
 * A logit of -infinity is never chosen.  The logits alone decide: a router that
 * chooses by them and a bias per expert, and weighs without it, chooses elsewhere
 * and takes mxg_route_rows.
 *   expert : int32 [tokens, k]; -1 where there is none: a masked token, a
 *            token whose logits are all -infinity (it counts as masked), or
 *            less than k logits above -infinity
 *   weight : float [tokens, k] = scale * s_e, or with `normalize` scale * s_e /
 *            (the sum of the token's chosen s); 0 where there is no expert
 *   counts : int32 [experts], tokens of each expert
 * The balance loss, with p = s / (sum of the token's s), n the tokens that take
 * part and P_e = (sum over them of p_e) / n:
 *   slope  : float [experts], balance * experts / n * counts_e / (sum of counts)
 *            -- the loss's derivative with respect to each p_e, for
 *            mxg_route_backward -- or NULL
 *   loss   : float [1], n * sum_e slope_e P_e, or NULL
 * (0 without any such token; the counts have no gradient).  A NaN
 * among a token's logits -- with MXG_SCORE_SOFTMAX +infinity too -- is chosen first
 * and makes the weights and shares that depend on it, and the loss, NaN.
 * Rows, where row_of and group_ws are given (both or neither): sorted by
 * expert, an expert's in the order of the tokens, each expert's group padded at
 * its end to a multiple of `align` rows (1 <= align <= 1024):
 *   row_of   : int32 [tokens, k], -1 where there is no expert
 *   group_ws : int64 [2 experts + 1], the padded sizes and the offsets times
 *              last_dim as the offsets entry points write them
 * Rows at or beyond rows_capacity, rounded down to a multiple of align, are
 * dropped: row_of -1, MXG_DEV_SUM_OVER_CAPACITY in dev_status.  tokens * k +
 * experts * (align - 1) rows always suffice.
 * 1 <= experts <= 1024, 1 <= k <= min(experts, 32), tokens >= 0 and tokens * k
 * and rows_capacity up to 2^31 - 128; scale and balance finite.  Sums are FP32
 * and of a fixed order; the loss's adds no more than tokens / 1216 + 256 terms
 * one after the other.  Exponentials, of the differences of logits (sigmoid: of
 * logits), are off by at most 2 + 1.7 |difference| units of 2^-23, a score by
 * about twice that; a score, weight or share below 2^-126 may be 0.  Any element
 * alignment; logits whose rows start on 16 bytes with experts a multiple of 8
 * take 16-byte accesses. */
typedef struct {
  mxg_dtype_t dtype;
  int64_t tokens;
  int32_t experts, k;
  const void* logits;
  int64_t ld;
  const uint8_t* mask;
  mxg_score_t score;
  int32_t normalize;
  float scale, balance;
  int32_t* expert;
  float* weight;
  int32_t* counts;
  float* loss;
  float* slope;
  int32_t* row_of;
  int64_t* group_ws;
  int32_t align;
  int64_t rows_capacity, last_dim;
} mxg_route_t;

/* Bytes of the workspace of mxg_route and mxg_route_rows (0 for sizes that they
 * refuse), which grow with the tokens: that of the largest batch serves smaller
 * ones.  16-byte aligned device memory whose contents mean nothing before or after
 * the call. */
size_t mxg_route_workspace_bytes(int64_t tokens, int experts, int k);

/* Errors: INVALID_ARG (nulls, sizes, types, ld < experts, last_dim < 1, or
 * rows_capacity * last_dim beyond int64), ALIGNMENT (a pointer not aligned to
 * its element, workspace, dev_status), WORKSPACE_TOO_SMALL, UNSUPPORTED_ARCH,
 * LAUNCH. */
mxg_status_t mxg_route(const mxg_route_t* desc, void* workspace, size_t workspace_bytes,
                       int32_t* dev_status, mxg_stream_t stream);

/* The counts and rows of mxg_route for experts chosen elsewhere: expert int32
 * [tokens, k], any value outside [0, experts) being no expert (an expert may be
 * named twice for a token: two rows).  row_of and group_ws as there (both or
 * neither).  Errors: as mxg_route. */
mxg_status_t mxg_route_rows(const int32_t* expert, int64_t tokens, int experts, int k, int align,
                            int64_t rows_capacity, int64_t last_dim, int32_t* counts,
                            int32_t* row_of, int64_t* group_ws, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, mxg_stream_t stream);

/* The gradient of mxg_route with respect to the logits.
 *   logits, expert : as given to and as written by mxg_route (a token's experts
 *                    are distinct, or outside [0, experts) for none)
 *   dweight : float [tokens, k], the gradient of the weights, or NULL: 0
 *   slope   : float [experts] of mxg_route, with dloss float [1], the gradient
 *             of the loss; both or neither (no loss)
 *   dlogits : [tokens, experts] of dtype, ldd elements between rows (0: dense);
 *             may be logits itself, with the same ld.  A token without any
 *             expert gets zeros; an entry of dweight beside no expert counts
 *             as 0, whatever it holds. */
typedef struct {
  mxg_dtype_t dtype;
  int64_t tokens;
  int32_t experts, k;
  const void* logits;
  int64_t ld;
  const int32_t* expert;
  mxg_score_t score;
  int32_t normalize;
  float scale;
  const float* dweight;
  const float* slope;
  const float* dloss;
  void* dlogits;
  int64_t ldd;
} mxg_route_grad_t;

/* Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_ARCH, LAUNCH, as mxg_route. */
mxg_status_t mxg_route_backward(const mxg_route_grad_t* desc, mxg_stream_t stream);

/* Rows between the tokens' order and the experts'.  `tokens` is [n, cols] (ldt
 * elements between rows, 0: dense), `rows` [rows_capacity, cols] (ldr), both of
 * dtype; row_of int32 [n, k] as mxg_route writes it: distinct values, and one
 * outside [0, rows_capacity) is no row.
 *   mxg_dispatch : rows[row_of[t, j]] = tokens[t]
 *   mxg_combine  : tokens[t] = sum_j weight[t, j] * rows[row_of[t, j]], summed in
 *                  FP32 in the order of j and rounded once; a token without rows
 *                  gets zeros.  weight float [n, k], or NULL for ones (the
 *                  gradient of mxg_dispatch).
 *   mxg_combine_backward : rows[row_of[t, j]] = weight[t, j] * tokens[t], with
 *                  tokens the gradient of the sums and rows that of the rows; and,
 *                  where dweight is given, dweight[t, j] = the sum over the
 *                  columns of tokens[t] * y_rows[row_of[t, j]] in FP32 (0 where
 *                  there is no row), y_rows [rows_capacity, cols] being what
 *                  mxg_combine summed (ldy); y_rows may be rows itself, with the
 *                  same ld.  rows may be NULL: only dweight.
 * Rows that row_of does not name are not written, but for padding: where counts
 * (int32 [experts]) and group_ws (as mxg_route writes them) are given to
 * mxg_dispatch or mxg_combine_backward, the rows between an expert's count and
 * its padded size are set to 0.  Where they are not, both are NULL and experts 0.
 * n >= 0, k from 1 to 32, n * k and rows_capacity up to 2^31 - 128, 1 <= cols <=
 * 2^20; without tokens (n = 0) or rows (rows_capacity = 0) their pointers may be
 * NULL.  Any element alignment; rows on 32 or 16 bytes take accesses of that size.
 * Apart from the one place named above, outputs do not overlap inputs. */
typedef struct {
  mxg_dtype_t dtype;
  int64_t n, cols;
  int32_t k, experts;
  int64_t rows_capacity;
  void* tokens;
  int64_t ldt;
  void* rows;
  int64_t ldr;
  const int32_t* row_of;
  const float* weight;
  const void* y_rows;
  int64_t ldy;
  float* dweight;
  const int32_t* counts;
  const int64_t* group_ws;
} mxg_expert_rows_t;

/* Errors of the three: INVALID_ARG (nulls, sizes, types, a leading dimension
 * below cols, a field that the call does not take being set), ALIGNMENT (a
 * pointer not aligned to its element), UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_dispatch(const mxg_expert_rows_t* desc, mxg_stream_t stream);
mxg_status_t mxg_combine(const mxg_expert_rows_t* desc, mxg_stream_t stream);
mxg_status_t mxg_combine_backward(const mxg_expert_rows_t* desc, mxg_stream_t stream);

/* The activations between an expert's products: x sigmoid(z(x)) with
 *   MXG_ACT_SILU      : z = x
 *   MXG_ACT_GELU_TANH : z = 2 sqrt(2 / pi) (x + 0.044715 x^3), which is
 *                       x / 2 (1 + tanh(z / 2)) */
typedef enum { MXG_ACT_SILU = 0, MXG_ACT_GELU_TANH = 1 } mxg_act_t;

/* Forward (mxg_gated_act): h = act(gate) . up, all [rows, cols] of dtype
 * (MXG_BF16 or MXG_F16), ld* elements between rows (0: dense); without up h =
 * act(gate).  FP32 inside, h rounded once; the exponential is off by at most 2 +
 * 1.2 |z| units of 2^-23, and where sigmoid(z) is below 2^-126 (z below about
 * -87.3) it counts as 0, in both directions.  Where q and sf are given, the inputs
 * are kept in 8 bits for the backward pass:
 *   q  : E4M3 [rows, cols] of gate and, beside it in the same row from column
 *        cols on, of up; ldq bytes between rows (0: cols, or 2 cols with up)
 *   sf : E8M0 [rows, B] of gate and beside it of up, B = ceil(cols / 32), dense:
 *        one byte for each 32 columns of a row (the last ones may be fewer)
 * by the rule of mxg_group_quantize's 1x32 blocks (the scale the least power of two
 * with amax <= 448 2^e; E4M3 to nearest even), the amax being taken over finite
 * values; an infinity or NaN is kept as NaN and does not touch its neighbours (a
 * bf16 value of more than 2^127 may be kept as 2^128, which is restored as
 * infinity).
 * Backward (mxg_gated_act_backward): from q, sf (gate and up being the values
 * that they stand for) and dh, the gradient of h:
 *   dgate = dh . up . act'(gate), dup = dh . act(gate), rounded once; and, where h
 *   is given, h again from those values, for the weight gradient of the second
 *   product.
 * gated : 1, or 0 where there is no up (nor dup).
 * group_ws : an offsets workspace of G groups, or NULL with G = 0.  Its first G
 *   entries sum to the live rows (negative ones count as 0); rows at or beyond
 *   them are neither read nor written.
 * rows from 0 to 2^31 - 128, 1 <= cols <= 2^20, G <= 1024.  h may be gate or up,
 * with the same ld, and dh dgate or dup.  Any element alignment; rows on 32 or 16
 * bytes (q: 16 or 8) with cols a multiple of 16 or 8 take accesses of that size. */
typedef struct {
  mxg_dtype_t dtype;
  mxg_act_t act;
  int64_t rows, cols;
  int32_t gated, G;
  const int64_t* group_ws;
  const void* gate;
  int64_t ldg;
  const void* up;
  int64_t ldu;
  void* h;
  int64_t ldh;
  uint8_t* q;
  int64_t ldq;
  uint8_t* sf;
  const void* dh;
  int64_t lddh;
  void* dgate;
  int64_t lddg;
  void* dup;
  int64_t lddu;
} mxg_gated_act_t;

/* Errors of both: INVALID_ARG (nulls, sizes, types, a leading dimension below its
 * row, only one of q and sf, a field of the other direction being set),
 * ALIGNMENT, UNSUPPORTED_ARCH, LAUNCH. */
mxg_status_t mxg_gated_act(const mxg_gated_act_t* desc, mxg_stream_t stream);
mxg_status_t mxg_gated_act_backward(const mxg_gated_act_t* desc, mxg_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* mxg_status_string(mxg_status_t status);

/* Library version: major * 10000 + minor * 100 + patch. */
int mxg_version(void);

/* Number of kernel launches this library has issued in this process
 * (all entry points, all devices).  For launch accounting in benchmarks. */
uint64_t mxg_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* MXG_H_ */

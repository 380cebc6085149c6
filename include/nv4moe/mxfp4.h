/*
 * nv4moe/mxfp4.h -- the MXFP4 calls of the expert path (included by nv4moe.h).
 *
 * MXFP4 (OCP Microscaling Formats v1.0): blocks of 32 FP4 E2M1 values under one E8M0
 * scale, a power of two.  Against NVFP4 (blocks of 16, E4M3 scale, FP32 tensor scale)
 * it has no tensor scale, so a block is quantised from its own 32 values alone, and
 * gfx950's scaled matrix instructions multiply it as it is stored: the products below
 * decode nothing.
 *
 * Numerics:
 *   block of 32 values v:  A = max|v|;
 *     NV4_MX_FLOOR  e = floor(log2 A) - 2   (the OCP rule: 2 is E2M1's largest exponent;
 *                                            values above 6 * 2^e saturate)
 *     NV4_MX_CEIL   e = the smallest with A <= 6 * 2^e   (nothing saturates)
 *     clamped to e >= -127; A == 0 gives e = -127.
 *   scale byte = e + 127; code = E2M1_rne_sat(v / 2^e), ties to the even code;
 *   element 2i sits in the low nibble of byte i; a code is sign << 3 | magnitude index
 *   (0, .5, 1, 1.5, 2, 3, 4, 6).  The value is e2m1(code) * 2^e, which BF16 holds exactly
 *   (but for 2^128 and above, which NV4_MX_CEIL makes of 1.75 * 2^127 and more: infinity).
 *   A block with a NaN or infinity gets scale byte 255 (NaN) and codes 0, and raises
 *   NV4_DS_NONFINITE; everything computed from it is NaN.
 *   Products are exact, sums are FP32.  SwiGLU is gate / (1 + exp(-gate)) * up in FP32 with a
 *   relative error of at most (1.25 |gate| + 8) 2^-24; it may be 0 for gates below -87.3, where
 *   exp(-gate) nears FP32's largest value.  Every call is deterministic.
 *
 * The conventions of nv4moe.h hold for every call here.
 */
#ifndef NV4MOE_MXFP4_H
#define NV4MOE_MXFP4_H

#include "../nv4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* scale rule */
#define NV4_MX_FLOOR 0
#define NV4_MX_CEIL 1

/* columns to which NV4_COLS pads each segment, and the tokens of mx_moe_few */
#define NV4_MX_SEGMENT 128
#define NV4_MX_FEW_TOKENS 64

/*
 * One MXFP4 tensor of logical shape [rows][K] (K % 32 == 0), memory owned by the caller:
 *   codes   [rows][K/2]  packed E2M1 codes, 16-byte aligned
 *   scales  [rows][mxfp4_scale_stride(K)]  E8M0 bytes, 4-byte aligned: K/32 of them and,
 *           behind the last block, zeros up to a multiple of 4
 */
typedef struct nv4_mx_tensor {
  uint8_t *codes;
  uint8_t *scales;
  int64_t rows;
  int64_t K;
} nv4_mx_tensor;

/* Bytes between two rows of scales: K/32 rounded up to a multiple of 4. */
int64_t mxfp4_scale_stride(int64_t K);

/*
 * mxfp4_quantize -- MXFP4 quantisation of a BF16 or FP32 matrix, one pass over it.
 *   x, xtype, x_rows, ldx  input [x_rows][ldx] (ldx >= K; at most 2^22 in the column layouts)
 *   rows, K          logical rows (after the gather) and columns, K % 32 == 0
 *   row_index        device int32 [rows] or NULL (not with NV4_COLS_BATCHED): logical row
 *                    r is row row_index[r] of x; an index outside x is clamped into it
 *   layout           NV4_ROWS: out [rows][K].
 *                    NV4_COLS: out [K][out->K], the transpose by segments as in
 *                      nvfp4_quantize, each segment padded with zeros to
 *                      NV4_MX_SEGMENT columns (seg_padded_offsets of mx_padded_offsets);
 *                      out->K >= rows + 127 * nseg, a multiple of 128; columns at and
 *                      after seg_padded_offsets[nseg] are not written.
 *                    NV4_ROWS_AND_COLS: NV4_COLS into out and NV4_ROWS into out_rows, of
 *                      which rows behind the last segment are not written.
 *                    NV4_COLS_BATCHED: nseg equal matrices of m = rows/nseg rows
 *                      (m % 32 == 0); out [nseg*K][m] holds each transposed.
 *   nseg, seg_offsets, seg_padded_offsets   device int32 [nseg+1], for NV4_COLS and
 *                    NV4_ROWS_AND_COLS (nseg alone for NV4_COLS_BATCHED).
 *   rule             NV4_MX_FLOOR or NV4_MX_CEIL
 * Errors: EINVAL, EALIGN (K % 32, ldx or x not in 16-byte steps, misaligned outputs,
 * m % 32), EUNSUPPORTED (row_index with NV4_COLS_BATCHED), EHIP.
 */
nv4_status mxfp4_quantize(const void *x, nv4_dtype xtype, int64_t x_rows, int64_t rows, int64_t K, int64_t ldx,
                          const int32_t *row_index, int layout, int nseg, const int32_t *seg_offsets,
                          const int32_t *seg_padded_offsets, int rule, nv4_mx_tensor *out, nv4_mx_tensor *out_rows,
                          int32_t *dev_status, void *stream);

/*
 * mxfp4_dequantize -- the values of an MXFP4 tensor, [q->rows][ldo], BF16 or FP32 (both
 * exact); scale byte 255 gives NaN.
 * Errors: EINVAL, EALIGN (ldo or out not in 16-byte steps, misaligned q), EHIP.
 */
nv4_status mxfp4_dequantize(const nv4_mx_tensor *q, void *out, nv4_dtype otype, int64_t ldo, void *stream);

/*
 * mx_padded_offsets -- padded[s] = sum over segments before s of their length rounded up
 * to NV4_MX_SEGMENT, from moe_permute's expert_offsets; int32 [nseg+1], nseg <= 1024.
 * Errors: EINVAL, EHIP.
 */
nv4_status mx_padded_offsets(const int32_t *offsets, int nseg, int32_t *padded, void *stream);

/*
 * mxfp4_grouped_gemm -- nvfp4_grouped_gemm's grouping on MXFP4 operands, by gfx950's
 * scaled FP4 matrix instruction.
 * NV4_GROUP_M: rows [offsets[e], offsets[e+1]) of A (or A rows a_rows[r]; an index
 *   outside A is clamped into it) times B_e^T; B [E*N][K] (EPI_NONE) or [E*2N][K]
 *   (EPI_SWIGLU: gate rows, then up rows); rows [0, min(offsets[E], M_cap)) of C are
 *   written and no others.
 *   q_out (EPI_SWIGLU, N % 32 == 0; NULL otherwise): the epilogue also quantises its FP32
 *   result into this [M_cap][N] tensor under `rule`: bit for bit what mxfp4_quantize
 *   makes of an FP32 C.  C may then be NULL.
 * NV4_GROUP_K: A [N][Kcap], B [M][Kcap] as NV4_COLS lays them out; expert e contracts
 *   over [offsets[e], offsets[e+1]) (multiples of NV4_MX_SEGMENT, from
 *   mx_padded_offsets); C [E][N][ldc] gets A_e . B_e^T, zeros for an empty range.
 *   offsets   device int32 [E+1], 1 <= E <= 1024
 * A, and an expert's part of B (GROUP_K: B), each stay below 4 GiB of codes.
 * No workspace.  Errors: EINVAL, EALIGN (K % 32, misaligned operands), EUNSUPPORTED
 * (a row index, q_out or SwiGLU with GROUP_K; q_out without SwiGLU), EHIP.
 */
nv4_status mxfp4_grouped_gemm(const nv4_mx_tensor *A, const nv4_mx_tensor *B, const int32_t *offsets, int E,
                              int64_t M_cap, int64_t N, const int32_t *a_rows, int group_mode, int epilogue,
                              void *C, nv4_dtype ctype, int64_t ldc, nv4_mx_tensor *q_out, int rule, void *stream);

/*
 * mx_moe_few -- a whole MXFP4 expert layer for at most NV4_MX_FEW_TOKENS tokens (a decode
 * step), in two to four kernels: routing and activation quantisation; gate and up products,
 * SwiGLU, re-quantisation; down product and weighted sum.
 *   out[t] = sum_j w[t][j] * W2_e . Q(silu(W13g_e . Q(x[t])) * (W13u_e . Q(x[t]))), e = id[t][j]
 * with every sum in FP32 and Q the quantisation above: the layer that moe_permute,
 * mxfp4_quantize, mxfp4_grouped_gemm (SwiGLU with q_out, then the down product) and
 * moe_combine compose, up to the order of the FP32 sums (which may take a value next to
 * a rounding border to the other code).
 *   x, xtype, ldx    [T][ldx], BF16 or FP32, H columns
 *   logits           FP32 [T][E], or NULL: topk_ids and topk_w are inputs (ids outside
 *                    [0, E) are skipped and raise NV4_DS_BAD_EXPERT; the same id twice
 *                    adds its weights)
 *   topk_ids, topk_w int32 / FP32 [T][k]: outputs when logits are given (may be NULL)
 *   w13 [E*2I][H], w2 [E*H][I]   H % 32 == 0, I % 32 == 0
 *   flags            NV4_RENORM or 0
 *   out              [T][H], BF16 or FP32
 *   dev_status       NV4_DS_NAN_LOGIT, NV4_DS_BAD_EXPERT, and NV4_DS_NONFINITE for x (a SwiGLU
 *                    value past FP32's range makes the token's results NaN without it)
 *   ws, ws_bytes     mx_moe_few_workspace() bytes, 256-byte aligned; calls that share one
 *                    must not overlap
 * Errors: EINVAL, EALIGN, EUNSUPPORTED (T > NV4_MX_FEW_TOKENS, E > 1024, k > min(E, 32)),
 * EWORKSPACE, EHIP.
 */
size_t mx_moe_few_workspace(int64_t T, int E, int k, int64_t H, int64_t I);
nv4_status mx_moe_few(const void *x, nv4_dtype xtype, int64_t ldx, const float *logits, int64_t T, int E, int k,
                      int flags, int32_t *topk_ids, float *topk_w, const nv4_mx_tensor *w13, const nv4_mx_tensor *w2,
                      int64_t H, int64_t I, int rule, void *out, nv4_dtype otype, int64_t ldo, void *ws,
                      size_t ws_bytes, int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NV4MOE_MXFP4_H */

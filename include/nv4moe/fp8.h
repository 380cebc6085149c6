/*
 * nv4moe/fp8.h -- the FP8 calls of the expert path (included by nv4moe.h).
 *
 * FP8 E4M3 (OCP OFP8, max 448) with an FP32 scale for each block of 128 values: activations
 * and gradients in blocks of 1 x 128 along their contraction dimension, weights in blocks of
 * 128 x 128.  Against the 4-bit formats it keeps three bits of significand, needs no tensor scale, and
 * a weight matrix's transpose is exact: the blocks of a data gradient's operand are the
 * forward's own, transposed.
 *
 * Numerics:
 *   block of values v:  A = max|v|;
 *     NV4_F8_FP32  S = min(fp32(448 / A), 2^126)
 *     NV4_F8_POW2  S = the largest power of two, at most 2^126, with A * S <= 448
 *     A == 0 gives S = 1.  The stored scale is G = fp32(1 / S);
 *   code = E4M3_rne(fp32(v * S)), ties to the even code; the value is e4m3(code) * G.
 *   Every FP32 step is one correctly rounded operation, so codes and scales are exactly
 *   defined.  |v * S| stays below 448 (1 + 2^-23), which rounds to 448: nothing saturates.
 *   A block with a NaN or infinity gets the scale NaN and codes 0; everything computed from it is
 *   NaN.  fp8_quantize raises NV4_DS_NONFINITE for it; fp8_grouped_gemm, which quantises into q_out as
 *   well, has no status: there the scale NaN alone shows it.
 *   Products: the sum of a block's code products, times fp32(Ga * Gb), is added in FP32, blocks in
 *   ascending order.  Where Ga * Gb falls below 2^-126 it loses bits, and above FP32's range it is
 *   infinite.  For an FP32 result (C in FP32) a block's sum is taken in FP32 from exact products.
 *   For a result that leaves as BF16 or FP8 only, the FP8 matrix instruction takes it: groups of eight
 *   products are added at the exponent of the largest with 13 bits behind it, the groups in FP32; the
 *   error is about 2^-16 of the result and at most 7 * 2^-13 of the sum of |products|.  Of a quantised
 *   result (q_out) about two codes in a thousand then are the neighbour of the one that FP32 sums give (K 2048, normal
 *   inputs): the values differ by 1.5e-3 of their norm, where quantising at all moves them by 2.3e-2, as far with
 *   either sum.  A call that also asks for C in FP32 quantises the FP32 sums' result.
 *   SwiGLU is gate / (1 + exp(-gate)) * up in FP32 with a relative error of at most
 *   (1.25 |gate| + 8) 2^-24; it may be 0 for gates below -87.3.
 *   Every call is deterministic.
 *
 * The conventions of nv4moe.h hold for every call here.
 */
#ifndef NV4MOE_FP8_H
#define NV4MOE_FP8_H

#include "../nv4moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a quantisation layout beside NV4_ROWS, NV4_COLS and NV4_ROWS_AND_COLS: 128 x 128 blocks */
#define NV4_F8_TILES 5

/* scale rule */
#define NV4_F8_FP32 0
#define NV4_F8_POW2 1

/* elements under one scale; also the columns to which NV4_COLS pads each segment */
#define NV4_F8_BLOCK 128

/*
 * One FP8 tensor of logical shape [rows][K] (K % 16 == 0), memory owned by the caller:
 *   codes   [rows][K]  E4M3 bytes, 16-byte aligned
 *   scales  FP32, 4-byte aligned, kb = ceil(K / 128):
 *           nseg == 0: [rows][kb], one for each 128 elements of a row;
 *           nseg >= 1: the rows are nseg stacked matrices of m = rows / nseg rows;
 *             [nseg][ceil(m / 128)][kb], one for each 128 x 128 block of a matrix
 *   rule    NV4_F8_POW2 says that every scale is a power of two from 2^-126 on (or NaN);
 *           NV4_F8_FP32 says nothing of them
 * fp8_quantize, fp8_transpose and fp8_grouped_gemm (q_out) set nseg and rule of what they write.
 */
typedef struct nv4_f8_tensor {
  uint8_t *codes;
  float *scales;
  int64_t rows;
  int64_t K;
  int32_t nseg;
  int32_t rule;
} nv4_f8_tensor;

/*
 * fp8_quantize -- FP8 quantisation of a BF16 or FP32 matrix, one pass over it.
 *   x, xtype, x_rows, ldx  input [x_rows][ldx] (ldx >= K; at most 2^22 but with NV4_ROWS)
 *   rows, K          logical rows (after the gather) and columns, K % 16 == 0
 *   row_index        device int32 [rows] or NULL (not with NV4_F8_TILES): logical row r is
 *                    row row_index[r] of x; an index outside x is clamped into it
 *   layout           NV4_ROWS: out [rows][K].
 *                    NV4_COLS: out [K][out->K], the transpose by segments as in
 *                      nvfp4_quantize, each segment padded with zeros to NV4_F8_BLOCK
 *                      columns (seg_padded_offsets of mx_padded_offsets), so that a block holds
 *                      one segment's rows; out->K >= rows + 127 * nseg, a multiple of
 *                      128; columns at and after seg_padded_offsets[nseg] are not written.
 *                    NV4_ROWS_AND_COLS: NV4_COLS into out and NV4_ROWS into out_rows, of
 *                      which rows behind the last segment are not written.
 *                    NV4_F8_TILES: out [rows][K] in 128 x 128 blocks of nseg equal matrices.
 *   nseg, seg_offsets, seg_padded_offsets   device int32 [nseg+1], for NV4_COLS and
 *                    NV4_ROWS_AND_COLS (nseg alone for NV4_F8_TILES).
 *   rule             NV4_F8_FP32 or NV4_F8_POW2
 * Errors: EINVAL, EALIGN (K % 16, ldx or x not in 16-byte steps, misaligned outputs),
 * EUNSUPPORTED (row_index with NV4_F8_TILES), EHIP.
 */
nv4_status fp8_quantize(const void *x, nv4_dtype xtype, int64_t x_rows, int64_t rows, int64_t K, int64_t ldx,
                        const int32_t *row_index, int layout, int nseg, const int32_t *seg_offsets,
                        const int32_t *seg_padded_offsets, int rule, nv4_f8_tensor *out, nv4_f8_tensor *out_rows,
                        int32_t *dev_status, void *stream);

/*
 * fp8_dequantize -- the values of an FP8 tensor, [q->rows][ldo]: FP32 rounds code * scale once,
 * BF16 that once more; a NaN scale gives NaN.
 * Errors: EINVAL, EALIGN (ldo or out not in 16-byte steps, misaligned q), EHIP.
 */
nv4_status fp8_dequantize(const nv4_f8_tensor *q, void *out, nv4_dtype otype, int64_t ldo, void *stream);

/*
 * fp8_transpose -- each of q's nseg matrices transposed, codes and scales moved as they are: q
 * [nseg*m][K] (nseg >= 1, m % 16 == 0), out [nseg*K][m].  The operand of a data gradient
 * from the forward's weights.  out does not overlap q.
 * Errors: EINVAL (nseg < 1, out's shape), EALIGN (m % 16, misaligned operands), EHIP.
 */
nv4_status fp8_transpose(const nv4_f8_tensor *q, nv4_f8_tensor *out, void *stream);

/*
 * fp8_grouped_gemm -- nvfp4_grouped_gemm's grouping on FP8 operands.
 * NV4_GROUP_M: rows [offsets[e], offsets[e+1]) of A (or A rows a_rows[r]; an index
 *   outside A is clamped into it) times B_e^T; A scaled by rows (nseg == 0), B [E*N][K]
 *   (EPI_NONE) or [E*2N][K] (EPI_SWIGLU: gate rows, then up rows; N % 32 == 0) in 128 x 128
 *   blocks of E matrices (nseg == E); rows [0, min(offsets[E], M_cap)) of C are written and
 *   no others.
 *   q_out (EPI_SWIGLU; NULL otherwise): the epilogue also quantises its FP32 result into this
 *   [M_cap][N] tensor under `rule`, before it is rounded to C's type: with an FP32 C bit for bit what
 *   fp8_quantize makes of C.  C may then be NULL (ctype is not looked at).
 * NV4_GROUP_K: A [N][Kcap], B [M][Kcap] as NV4_COLS lays them out (nseg == 0 both); expert
 *   e contracts over [offsets[e], offsets[e+1]) (multiples of NV4_F8_BLOCK, from
 *   mx_padded_offsets; others are taken to the blocks that they touch); C [E][N][ldc] gets
 *   A_e . B_e^T, zeros for an empty range.
 *   offsets   device int32 [E+1], 1 <= E <= 1024
 * A call's result depends on its arguments alone, bit for bit; a call with other outputs or another
 *   M_cap may add a row's blocks in another order.
 * A, and an expert's part of B (GROUP_K: B), each stay below 4 GiB of codes; C has at most 2^20
 * columns, ldc included.
 * No workspace.  Errors: EINVAL (shapes, an operand's nseg), EALIGN (K % 16, SwiGLU with N % 32,
 * misaligned operands), EUNSUPPORTED (a row index, q_out or SwiGLU with GROUP_K; q_out without
 * SwiGLU), EHIP.
 */
nv4_status fp8_grouped_gemm(const nv4_f8_tensor *A, const nv4_f8_tensor *B, const int32_t *offsets, int E,
                            int64_t M_cap, int64_t N, const int32_t *a_rows, int group_mode, int epilogue,
                            void *C, nv4_dtype ctype, int64_t ldc, nv4_f8_tensor *q_out, int rule, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NV4MOE_FP8_H */

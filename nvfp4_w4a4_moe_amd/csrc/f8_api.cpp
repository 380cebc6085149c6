// C ABI of the FP8 calls (declarations and contracts: include/nv4moe/fp8.h).  Host side only:
// argument validation and dispatch to the kernel launchers.  No call allocates memory or waits
// on the device.
#include <hip/hip_runtime.h>

#include "../../include/nv4moe.h"
#include "api_common.h"
#include "f8_internal.h"

using nv4::aligned;
using nv4::f8_blocks;
using nv4::fail;
using nv4::from_hip;
using nv4::ok;

namespace {

constexpr int64_t kMost32 = 1ll << 31;

bool bad_rule(int rule) { return rule != NV4_F8_FP32 && rule != NV4_F8_POW2; }

// an operand's codes and scales: shape, pointers, alignment
nv4_status check_tensor(const char *fn, const char *name, const nv4_f8_tensor *t) {
  if (!t) return fail(NV4_EINVAL, "%s: %s is NULL", fn, name);
  if (t->rows < 0 || t->K < 0) return fail(NV4_EINVAL, "%s: %s has a negative shape", fn, name);
  if (t->K % 16) return fail(NV4_EALIGN, "%s: %s->K = %lld is not a multiple of 16", fn, name, (long long)t->K);
  if (t->rows >= kMost32 || t->K >= kMost32) return fail(NV4_EINVAL, "%s: %s is too large", fn, name);
  if (t->rows == 0 || t->K == 0) return NV4_OK;
  if (!t->codes || !t->scales) return fail(NV4_EINVAL, "%s: %s has a NULL buffer", fn, name);
  if (!aligned(t->codes, 16) || !aligned(t->scales, 4))
    return fail(NV4_EALIGN, "%s: %s needs 16-byte aligned codes and 4-byte aligned scales", fn, name);
  return NV4_OK;
}

// an input operand: also its scale grouping
nv4_status check_operand(const char *fn, const char *name, const nv4_f8_tensor *t) {
  const nv4_status st = check_tensor(fn, name, t);
  if (st != NV4_OK) return st;
  if (bad_rule(t->rule)) return fail(NV4_EINVAL, "%s: %s has a bad scale rule %d", fn, name, t->rule);
  if (t->nseg < 0 || (t->nseg > 0 && t->rows % t->nseg))
    return fail(NV4_EINVAL, "%s: %s has %lld rows in %d matrices", fn, name, (long long)t->rows, t->nseg);
  return NV4_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- quantisation

nv4_status fp8_quantize(const void *x, nv4_dtype xtype, int64_t x_rows, int64_t rows, int64_t K, int64_t ldx,
                        const int32_t *row_index, int layout, int nseg, const int32_t *seg_offsets,
                        const int32_t *seg_padded_offsets, int rule, nv4_f8_tensor *out, nv4_f8_tensor *out_rows,
                        int32_t *dev_status, void *stream) {
  const char *fn = "fp8_quantize";
  if (xtype != NV4_BF16 && xtype != NV4_F32) return fail(NV4_EINVAL, "%s: bad input dtype", fn);
  if (layout != NV4_ROWS && layout != NV4_COLS && layout != NV4_ROWS_AND_COLS && layout != NV4_F8_TILES)
    return fail(NV4_EINVAL, "%s: bad layout %d", fn, layout);
  if (bad_rule(rule)) return fail(NV4_EINVAL, "%s: bad scale rule %d", fn, rule);
  if (rows < 0 || K < 0 || x_rows < 0) return fail(NV4_EINVAL, "%s: negative shape", fn);
  if (rows >= kMost32 || K >= kMost32 || x_rows >= kMost32 || rows * f8_blocks(K) >= kMost32)
    return fail(NV4_EINVAL, "%s: shape too large", fn);
  if (K % 16) return fail(NV4_EALIGN, "%s: K = %lld is not a multiple of 16", fn, (long long)K);
  if (ldx < K) return fail(NV4_EINVAL, "%s: ldx < K", fn);
  if ((ldx * (xtype == NV4_F32 ? 4 : 2)) % 16 || !aligned(x, 16))
    return fail(NV4_EALIGN, "%s: x and its row stride must be 16-byte aligned", fn);
  if (row_index && layout == NV4_F8_TILES)
    return fail(NV4_EUNSUPPORTED, "%s: row_index is not supported with NV4_F8_TILES", fn);
  if (!row_index && x_rows < rows) return fail(NV4_EINVAL, "%s: x has fewer than `rows` rows", fn);
  if (row_index && rows > 0 && x_rows == 0) return fail(NV4_EINVAL, "%s: row index into an empty x", fn);
  nv4_status st = check_tensor(fn, "out", out);
  if (st != NV4_OK) return st;
  const bool both = layout == NV4_ROWS_AND_COLS, cols = layout == NV4_COLS || both;
  if (both) {
    st = check_tensor(fn, "out_rows", out_rows);
    if (st != NV4_OK) return st;
    if (out_rows->rows != rows || out_rows->K != K) return fail(NV4_EINVAL, "%s: out_rows must be [rows][K]", fn);
  } else if (out_rows) {
    return fail(NV4_EINVAL, "%s: out_rows is for NV4_ROWS_AND_COLS", fn);
  }
  if (layout != NV4_ROWS && (nseg < 1 || nseg > (1 << 20))) return fail(NV4_EINVAL, "%s: bad nseg %d", fn, nseg);
  if (!cols && (out->rows != rows || out->K != K)) return fail(NV4_EINVAL, "%s: out must be [rows][K]", fn);
  if (layout == NV4_F8_TILES) {
    if (rows % nseg) return fail(NV4_EINVAL, "%s: rows must be nseg equal matrices", fn);
    if (nseg * f8_blocks(rows / nseg) * f8_blocks(K) >= kMost32) return fail(NV4_EINVAL, "%s: shape too large", fn);
  }
  if (cols) {
    if (!seg_offsets || !seg_padded_offsets)
      return fail(NV4_EINVAL, "%s: NV4_COLS needs seg_offsets and seg_padded_offsets", fn);
    if (out->rows != K) return fail(NV4_EINVAL, "%s: out must have K rows", fn);
    if (out->K % NV4_F8_BLOCK)
      return fail(NV4_EALIGN, "%s: NV4_COLS needs out->K to be a multiple of %d", fn, NV4_F8_BLOCK);
    if (out->K < rows + (NV4_F8_BLOCK - 1) * (int64_t)nseg)
      return fail(NV4_EINVAL, "%s: out->K must be >= rows + 127 * nseg (padded capacity)", fn);
  }
  out->nseg = layout == NV4_F8_TILES ? nseg : 0;
  out->rule = rule;
  if (both) out_rows->nseg = 0, out_rows->rule = rule;
  if (rows == 0 || K == 0) return ok();
  if (!x) return fail(NV4_EINVAL, "%s: x is NULL", fn);
  if (layout != NV4_ROWS) {
    if (cols && (f8_blocks(rows) + nseg) * f8_blocks(K) >= kMost32) return fail(NV4_EINVAL, "%s: shape too large", fn);
    // a tile of 128 rows is addressed with 32-bit offsets
    if (ldx > (1ll << 22)) return fail(NV4_EINVAL, "%s: ldx is above 2^22 in this layout", fn);
  }
  nv4::F8QuantArgs a{};
  a.x = x;
  a.x_is_f32 = xtype == NV4_F32;
  a.x_rows = x_rows;
  a.rows = rows;
  a.K = K;
  a.ldx = ldx;
  a.row_index = row_index;
  a.layout = layout;
  a.nseg = nseg;
  a.seg_offsets = seg_offsets;
  a.seg_padded_offsets = seg_padded_offsets;
  a.pow2 = rule == NV4_F8_POW2;
  a.codes = out->codes;
  a.scales = out->scales;
  if (both) {
    a.codes2 = out_rows->codes;
    a.scales2 = out_rows->scales;
  }
  a.out_K = out->K;
  a.dev_status = dev_status;
  return from_hip(nv4::launch_f8_quantize(a, static_cast<hipStream_t>(stream)), fn);
}

nv4_status fp8_dequantize(const nv4_f8_tensor *q, void *out, nv4_dtype otype, int64_t ldo, void *stream) {
  const char *fn = "fp8_dequantize";
  const nv4_status st = check_operand(fn, "q", q);
  if (st != NV4_OK) return st;
  if (otype != NV4_BF16 && otype != NV4_F32) return fail(NV4_EINVAL, "%s: bad output dtype", fn);
  if (ldo < q->K) return fail(NV4_EINVAL, "%s: ldo < K", fn);
  if (q->rows * f8_blocks(q->K) >= kMost32) return fail(NV4_EINVAL, "%s: shape too large", fn);
  if ((ldo * (otype == NV4_F32 ? 4 : 2)) % 16 || !aligned(out, 16))
    return fail(NV4_EALIGN, "%s: out and its row stride must be 16-byte aligned", fn);
  if (q->rows == 0 || q->K == 0) return ok();
  if (!out) return fail(NV4_EINVAL, "%s: out is NULL", fn);
  nv4::F8DequantArgs a{};
  a.codes = q->codes;
  a.scales = q->scales;
  a.rows = q->rows;
  a.K = q->K;
  a.nseg = q->nseg;
  a.out = out;
  a.out_is_f32 = otype == NV4_F32;
  a.ldo = ldo;
  return from_hip(nv4::launch_f8_dequantize(a, static_cast<hipStream_t>(stream)), fn);
}

nv4_status fp8_transpose(const nv4_f8_tensor *q, nv4_f8_tensor *out, void *stream) {
  const char *fn = "fp8_transpose";
  nv4_status st = check_operand(fn, "q", q);
  if (st == NV4_OK) st = check_tensor(fn, "out", out);
  if (st != NV4_OK) return st;
  if (q->nseg < 1) return fail(NV4_EINVAL, "%s: q must be scaled in 128 x 128 blocks", fn);
  const int64_t m = q->rows / q->nseg;
  if (m % 16) return fail(NV4_EALIGN, "%s: the matrices' %lld rows are not a multiple of 16", fn, (long long)m);
  if (out->rows != (int64_t)q->nseg * q->K || out->K != m)
    return fail(NV4_EINVAL, "%s: out must be [nseg*K][rows/nseg]", fn);
  if (q->nseg * f8_blocks(m) * f8_blocks(q->K) >= kMost32) return fail(NV4_EINVAL, "%s: shape too large", fn);
  out->nseg = q->nseg;
  out->rule = q->rule;
  if (q->rows == 0 || q->K == 0) return ok();
  if (q->codes == out->codes || q->scales == out->scales) return fail(NV4_EINVAL, "%s: out overlaps q", fn);
  nv4::F8TransposeArgs a{};
  a.codes = q->codes;
  a.scales = q->scales;
  a.nseg = q->nseg;
  a.m = m;
  a.K = q->K;
  a.out_codes = out->codes;
  a.out_scales = out->scales;
  return from_hip(nv4::launch_f8_transpose(a, static_cast<hipStream_t>(stream)), fn);
}

// ---------------------------------------------------------------- grouped GEMM

nv4_status fp8_grouped_gemm(const nv4_f8_tensor *A, const nv4_f8_tensor *B, const int32_t *offsets, int E,
                            int64_t M_cap, int64_t N, const int32_t *a_rows, int group_mode, int epilogue,
                            void *C, nv4_dtype ctype, int64_t ldc, nv4_f8_tensor *q_out, int rule, void *stream) {
  const char *fn = "fp8_grouped_gemm";
  nv4_status st = check_operand(fn, "A", A);
  if (st == NV4_OK) st = check_operand(fn, "B", B);
  if (st != NV4_OK) return st;
  const bool empty = group_mode == NV4_GROUP_K ? A->rows == 0 || B->rows == 0 : M_cap == 0;
  if (!offsets || (!C && !q_out && !empty)) return fail(NV4_EINVAL, "%s: NULL argument", fn);
  if (E < 1 || E > 1024) return fail(NV4_EINVAL, "%s: E must be in [1, 1024]", fn);
  if (group_mode != NV4_GROUP_M && group_mode != NV4_GROUP_K) return fail(NV4_EINVAL, "%s: bad group_mode", fn);
  if (epilogue != NV4_EPI_NONE && epilogue != NV4_EPI_SWIGLU) return fail(NV4_EINVAL, "%s: bad epilogue", fn);
  if (C && ctype != NV4_BF16 && ctype != NV4_F32) return fail(NV4_EINVAL, "%s: bad C dtype", fn);
  if (bad_rule(rule)) return fail(NV4_EINVAL, "%s: bad scale rule %d", fn, rule);
  if (A->K != B->K) return fail(NV4_EINVAL, "%s: A->K != B->K", fn);
  if (A->K == 0) return fail(NV4_EINVAL, "%s: K must be positive", fn);
  if (A->nseg != 0) return fail(NV4_EINVAL, "%s: A must be scaled by rows", fn);
  if (B->nseg != (group_mode == NV4_GROUP_K ? 0 : E))
    return fail(NV4_EINVAL, "%s: B must be scaled by rows (GROUP_K) or in 128 x 128 blocks of E matrices (GROUP_M)", fn);
  const int64_t esz = ctype == NV4_F32 ? 4 : 2;
  if (!aligned(C, esz)) return fail(NV4_EALIGN, "%s: C is not aligned to its type", fn);
  // byte offsets into A and into an expert's part of B are 32-bit; one below 2^32 - 256 marks an
  // absent row
  const int64_t most = 0xFFFFFF00ll;
  if (A->rows * A->K > most || (group_mode == NV4_GROUP_K ? B->rows : B->rows / E) * B->K > most)
    return fail(NV4_EINVAL, "%s: A and an expert's part of B must each stay below 4 GiB of codes", fn);
  const int64_t ncols = group_mode == NV4_GROUP_K ? B->rows : N;
  if (C && ldc < ncols) return fail(NV4_EINVAL, "%s: ldc < columns of C", fn);
  // columns and tiles are counted in 32 bits, a tile's rows of C addressed with 32-bit offsets
  if (ncols > (1ll << 20) || (C && ldc > (1ll << 20))) return fail(NV4_EINVAL, "%s: too many columns", fn);
  if ((group_mode == NV4_GROUP_K ? (int64_t)E * A->rows : M_cap) * ncols > (1ll << 40))
    return fail(NV4_EINVAL, "%s: C is too large", fn);
  if (group_mode == NV4_GROUP_M) {
    const int64_t Nb = epilogue == NV4_EPI_SWIGLU ? 2 * N : N;
    if (N <= 0) return fail(NV4_EINVAL, "%s: N must be positive", fn);
    if (epilogue == NV4_EPI_SWIGLU && N % 32)
      return fail(NV4_EALIGN, "%s: SwiGLU needs N = %lld to be a multiple of 32", fn, (long long)N);
    if (B->rows != (int64_t)E * Nb)
      return fail(NV4_EINVAL, "%s: B->rows = %lld, expected E * %lld", fn, (long long)B->rows, (long long)Nb);
    if (M_cap < 0 || M_cap >= kMost32 || (!a_rows && M_cap > A->rows))
      return fail(NV4_EINVAL, "%s: M_cap exceeds the rows of A", fn);
    if (a_rows && M_cap * 4 > most) return fail(NV4_EINVAL, "%s: too many row indices", fn);  // 32-bit offsets too
    if (a_rows && M_cap > 0 && A->rows == 0) return fail(NV4_EINVAL, "%s: row index into an empty A", fn);
    if (q_out) {
      if (epilogue != NV4_EPI_SWIGLU) return fail(NV4_EUNSUPPORTED, "%s: q_out needs the SwiGLU epilogue", fn);
      st = check_tensor(fn, "q_out", q_out);
      if (st != NV4_OK) return st;
      if (q_out->rows != M_cap || q_out->K != N) return fail(NV4_EINVAL, "%s: q_out must be [M_cap][N]", fn);
      q_out->nseg = 0;
      q_out->rule = rule;
    }
  } else {
    if (epilogue != NV4_EPI_NONE) return fail(NV4_EUNSUPPORTED, "%s: GROUP_K has no SwiGLU epilogue", fn);
    if (a_rows) return fail(NV4_EUNSUPPORTED, "%s: GROUP_K takes no row index", fn);
    if (q_out) return fail(NV4_EUNSUPPORTED, "%s: GROUP_K has no quantised output", fn);
    if (A->K % NV4_F8_BLOCK)
      return fail(NV4_EALIGN, "%s: GROUP_K needs K to be a multiple of %d", fn, NV4_F8_BLOCK);
  }
  if (empty) return ok();
  nv4::F8GemmArgs g{};
  g.a_codes = A->codes;
  g.a_scales = A->scales;
  g.a_rows = A->rows;
  g.K = A->K;
  g.a_rows_index = a_rows;
  g.b_codes = B->codes;
  g.b_scales = B->scales;
  g.b_rows = B->rows;
  g.offsets = offsets;
  g.E = E;
  g.M_cap = M_cap;
  g.N = N;
  g.group_mode = group_mode;
  g.epilogue = epilogue;
  g.pow2 = A->rule == NV4_F8_POW2 && B->rule == NV4_F8_POW2;
  g.C = C;
  g.c_is_f32 = C && ctype == NV4_F32;
  g.ldc = ldc;
  if (q_out) {
    g.q_codes = q_out->codes;
    g.q_scales = q_out->scales;
  }
  g.q_pow2 = rule == NV4_F8_POW2;
  return from_hip(nv4::launch_f8_gemm(g, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"

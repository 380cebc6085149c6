// C ABI of the router's training calls (declarations and contracts: include/nv4moe/router.h).  Host
// side only: argument validation and dispatch to the kernel launchers.  No call allocates memory
// or waits on the device.
#include <hip/hip_runtime.h>

#include "../../include/nv4moe.h"
#include "api_common.h"
#include "router_internal.h"

using nv4::aligned;
using nv4::fail;
using nv4::from_hip;
using nv4::ok;

namespace {

constexpr int kMostSegments = 1 << 16;

// what the loss and its gradient ask of their shapes
nv4_status check_router(const char *fn, const float *logits, int64_t T, int E, int k, const int32_t *topk_ids, int nseg,
                        const int32_t *seg_offsets) {
  if (T < 0) return fail(NV4_EINVAL, "%s: T < 0", fn);
  if (E <= 0 || k <= 0) return fail(NV4_EINVAL, "%s: E and k must be positive", fn);
  if (E > 1024) return fail(NV4_EUNSUPPORTED, "%s: E = %d exceeds 1024", fn, E);
  if (k > 32 || k > E) return fail(NV4_EUNSUPPORTED, "%s: k = %d must be <= min(E, 32)", fn, k);
  if (nseg < 1) return fail(NV4_EINVAL, "%s: bad nseg %d", fn, nseg);
  if (nseg > kMostSegments) return fail(NV4_EUNSUPPORTED, "%s: nseg = %d exceeds %d", fn, nseg, kMostSegments);
  if (!seg_offsets && nseg != 1) return fail(NV4_EINVAL, "%s: %d segments need seg_offsets", fn, nseg);
  if (T >= (1ll << 31)) return fail(NV4_EINVAL, "%s: T is too large", fn);
  if (T > 0 && (!logits || !topk_ids)) return fail(NV4_EINVAL, "%s: NULL pointer", fn);
  return NV4_OK;
}

}  // namespace

extern "C" {

size_t moe_balance_workspace(int64_t T, int E, int nseg) {
  if (T < 0 || E <= 0 || nseg <= 0) return 0;
  return nv4::balance_workspace_bytes(T, E, nseg);
}

nv4_status moe_balance_loss(const float *logits, int64_t T, int E, int k, const int32_t *topk_ids,
                            const uint8_t *mask, int nseg, const int32_t *seg_offsets, int32_t *counts,
                            float *prob_sums, int32_t *tokens, float *loss, void *ws, size_t ws_bytes,
                            int32_t *dev_status, void *stream) {
  const char *fn = "moe_balance_loss";
  const nv4_status st = check_router(fn, logits, T, E, k, topk_ids, nseg, seg_offsets);
  if (st != NV4_OK) return st;
  if (!counts || !prob_sums || !tokens || !loss) return fail(NV4_EINVAL, "%s: NULL output", fn);
  const size_t need = nv4::balance_workspace_bytes(T, E, nseg);
  if (!ws || ws_bytes < need) return fail(NV4_EWORKSPACE, "%s: workspace of %zu bytes required", fn, need);
  if (!aligned(ws, 256)) return fail(NV4_EALIGN, "%s: workspace must be 256-byte aligned", fn);
  nv4::BalanceArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.topk_ids = topk_ids;
  a.mask = mask;
  a.nseg = nseg;
  a.seg_offsets = seg_offsets;
  a.counts = counts;
  a.prob_sums = prob_sums;
  a.tokens = tokens;
  a.loss = loss;
  a.ws = ws;
  a.dev_status = dev_status;
  return from_hip(nv4::launch_balance_loss(a, static_cast<hipStream_t>(stream)), fn);
}

nv4_status moe_balance_backward(const float *logits, int64_t T, int E, int k, const int32_t *topk_ids,
                                const uint8_t *mask, int nseg, const int32_t *seg_offsets, const int32_t *counts,
                                const int32_t *tokens, const float *dloss, const float *dtopk_w, int flags,
                                float *dlogits, int32_t *dev_status, void *stream) {
  const char *fn = "moe_balance_backward";
  const nv4_status st = check_router(fn, logits, T, E, k, topk_ids, nseg, seg_offsets);
  if (st != NV4_OK) return st;
  if (flags & ~NV4_RENORM) return fail(NV4_EINVAL, "%s: unknown flags", fn);
  if (dloss && (!counts || !tokens)) return fail(NV4_EINVAL, "%s: dloss needs counts and tokens", fn);
  if (T == 0) return ok();
  if (!dlogits) return fail(NV4_EINVAL, "%s: dlogits is NULL", fn);
  nv4::BalanceBackwardArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.topk_ids = topk_ids;
  a.mask = mask;
  a.nseg = nseg;
  a.seg_offsets = seg_offsets;
  a.counts = counts;
  a.tokens = tokens;
  a.dloss = dloss;
  a.dtopk_w = dtopk_w;
  a.renorm = (flags & NV4_RENORM) != 0;
  a.dlogits = dlogits;
  a.dev_status = dev_status;
  return from_hip(nv4::launch_balance_backward(a, static_cast<hipStream_t>(stream)), fn);
}

nv4_status moe_combine_backward(const void *dout, nv4_dtype otype, const void *Y, nv4_dtype ytype, int64_t ldy,
                                int64_t rows, const int32_t *token_row, const float *topk_w, int64_t T, int k,
                                int64_t H, void *dY, int64_t lddy, float *dtopk_w, void *stream) {
  const char *fn = "moe_combine_backward";
  if (T < 0 || k <= 0 || H <= 0 || rows < 0) return fail(NV4_EINVAL, "%s: bad shape", fn);
  if (T >= (1ll << 31)) return fail(NV4_EINVAL, "%s: T is too large", fn);
  if (ytype != NV4_BF16 && ytype != NV4_F32) return fail(NV4_EINVAL, "%s: bad Y dtype", fn);
  if (otype != NV4_BF16 && otype != NV4_F32) return fail(NV4_EINVAL, "%s: bad dout dtype", fn);
  if (H % 4) return fail(NV4_EALIGN, "%s: H = %lld is not a multiple of 4", fn, (long long)H);
  const size_t y16 = ytype == NV4_F32 ? 16 : 8;
  if (!aligned(dout, otype == NV4_F32 ? 16 : 8)) return fail(NV4_EALIGN, "%s: dout is not aligned to 4 elements", fn);
  if (dtopk_w) {
    if (ldy < H) return fail(NV4_EINVAL, "%s: ldy < H", fn);
    if (ldy % 4 || !aligned(Y, y16)) return fail(NV4_EALIGN, "%s: Y and its row stride must be aligned to 4 elements", fn);
  }
  if (dY) {
    if (lddy < H) return fail(NV4_EINVAL, "%s: lddy < H", fn);
    if (lddy % 4 || !aligned(dY, y16))
      return fail(NV4_EALIGN, "%s: dY and its row stride must be aligned to 4 elements", fn);
    if (dY == Y || dY == dout) return fail(NV4_EINVAL, "%s: dY overlaps an input", fn);
  }
  if (T == 0) return ok();
  if (!dY && !dtopk_w) return fail(NV4_EINVAL, "%s: no output", fn);
  if (!dout || !token_row || !topk_w || (dtopk_w && !Y && rows > 0)) return fail(NV4_EINVAL, "%s: NULL pointer", fn);
  nv4::CombineBackwardArgs a{};
  a.dout = dout;
  a.dout_is_f32 = otype == NV4_F32;
  a.Y = Y;
  a.y_is_f32 = ytype == NV4_F32;
  a.ldy = ldy;
  a.rows = rows;
  a.token_row = token_row;
  a.topk_w = topk_w;
  a.T = T;
  a.k = k;
  a.H = H;
  a.dY = dY;
  a.lddy = lddy;
  a.dtopk_w = dtopk_w;
  return from_hip(nv4::launch_combine_backward(a, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"

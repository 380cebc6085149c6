"""FP8 calls of the binding (include/nv4moe/fp8.h): E4M3 codes with an FP32 scale for each block of
128 values, 1 x 128 for activations and gradients and 128 x 128 for weights.

    fp8_quantize        quantisation (rows, columns by segment, both, 128 x 128 blocks)
    fp8_dequantize      the values, BF16 or FP32
    fp8_transpose       quantised matrices transposed, exactly
    fp8_grouped_gemm    grouped product (GROUP_M with optional SwiGLU and fused
                        re-quantisation, GROUP_K)

``fp8_moe_forward`` and ``fp8_moe_backward`` compose them with moe_permute and moe_combine as
``moe_forward`` and ``moe_backward`` do for NVFP4.  Segments are padded as MXFP4's are:
mx_padded_offsets and mx_cols_capacity serve both.  Everything here is reachable from the package's
top level.

Matrices may have any row stride of at least their width.  With ``stream`` a call, or a whole
layer, runs on that stream, and what it allocates comes from that stream's pool; the stream waits
for no other, so inputs have to be ready there and results be waited for by whoever reads them.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import (NV4_COLS, NV4_EPI_NONE, NV4_EPI_SWIGLU, NV4_F32, NV4_GROUP_K, NV4_GROUP_M, NV4_ROWS, NV4_ROWS_AND_COLS,
               Routing, _I, _I64, _P, _SIGS, _Stage, load, moe_combine, moe_permute)
from .mxfp4 import _Call, _Layer, _float, _ints, _matrix, _p, _weight_shapes, mx_cols_capacity, mx_padded_offsets

NV4_F8_TILES = 5
NV4_F8_FP32, NV4_F8_POW2 = 0, 1
NV4_F8_BLOCK = 128

__all__ = ["NV4_F8_TILES", "NV4_F8_FP32", "NV4_F8_POW2", "NV4_F8_BLOCK", "F8Tensor", "FP8", "fp8_quantize",
           "fp8_dequantize", "fp8_transpose", "fp8_grouped_gemm", "F8ExpertWeights", "F8TransposedWeights",
           "fp8_quantize_expert_weights", "fp8_transpose_expert_weights", "F8ForwardBuffers", "fp8_alloc_forward",
           "fp8_moe_forward", "F8BackwardBuffers", "fp8_alloc_backward", "fp8_moe_backward"]


class F8Tensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("K", ctypes.c_int64), ("nseg", ctypes.c_int32), ("rule", ctypes.c_int32)]


_T = ctypes.POINTER(F8Tensor)
_SIGS.update({
    "fp8_quantize": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _I, _I, _P, _P, _I, _T, _T, _P, _P]),
    "fp8_dequantize": (_I, [_T, _P, _I, _I64, _P]),
    "fp8_transpose": (_I, [_T, _T, _P]),
    "fp8_grouped_gemm": (_I, [_T, _T, _P, _I, _I64, _I64, _P, _I, _I, _P, _I, _I64, _T, _I, _P]),
})

_U8, _F32 = torch.uint8, torch.float32


def _scale_count(rows: int, K: int, nseg: int) -> int:
    kb = (K + 127) // 128
    return nseg * ((rows // nseg + 127) // 128) * kb if nseg else rows * kb


@dataclass
class FP8:
    """Device FP8 tensor: codes [rows, K] u8 (E4M3 bits), scales FP32.  nseg 0: scales [rows,
    ceil(K/128)]; otherwise the rows are nseg matrices of m rows each and scales [nseg, ceil(m/128),
    ceil(K/128)].  rule NV4_F8_POW2: every scale is a power of two."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    K: int
    nseg: int = 0
    rule: int = NV4_F8_FP32
    rows_out: "FP8 | None" = None  # the row-direction output of NV4_ROWS_AND_COLS

    @staticmethod
    def empty(rows: int, K: int, nseg: int = 0, device="cuda") -> "FP8":
        kb = (K + 127) // 128
        shape = (nseg, (rows // nseg + 127) // 128, kb) if nseg else (rows, kb)
        return FP8(torch.empty((rows, K), dtype=_U8, device=device), torch.empty(shape, dtype=_F32, device=device), rows,
                   K, nseg)

    def c(self, nseg: int | None = None) -> F8Tensor:
        """The C descriptor; nseg: the grouping that a call is about to write."""
        c, s, rows, K = self.codes, self.scales, self.rows, self.K
        n = self.nseg if nseg is None else nseg
        if not (c.dtype is _U8 and s.dtype is _F32 and c.is_contiguous() and s.is_contiguous() and
                c.numel() == rows * K and s.numel() == _scale_count(rows, K, n)):
            raise ValueError(f"FP8 [{rows}, {K}] of nseg {n} needs contiguous uint8 codes and FP32 scales of its shape")
        return F8Tensor(c.data_ptr(), s.data_ptr(), rows, K, n, self.rule)


def _new(call: _Call, rows: int, K: int, nseg: int = 0) -> FP8:
    kb = (K + 127) // 128
    shape = (nseg, (rows // nseg + 127) // 128, kb) if nseg else (rows, kb)
    return FP8(call.empty(_U8, rows, K), call.empty(_F32, *shape), rows, K, nseg)


# ----------------------------------------------------------------------------- quantisation

def fp8_quantize(x: torch.Tensor, layout: int = NV4_ROWS, nseg: int = 1, seg_offsets: torch.Tensor | None = None,
                 seg_padded_offsets: torch.Tensor | None = None, row_index: torch.Tensor | None = None,
                 out: FP8 | None = None, out_K: int | None = None, out_rows: FP8 | None = None,
                 rule: int = NV4_F8_FP32, dev_status: torch.Tensor | None = None, stream=None) -> FP8:
    """FP8-quantise a 2-D BF16/FP32 tensor (row stride x.stride(0)).  With row_index (int32),
    logical row r is x row row_index[r].  NV4_ROWS_AND_COLS returns the column output with the
    row output in its `rows_out` (out_rows, allocated when None); NV4_F8_TILES scales blocks of
    128 x 128 of nseg stacked matrices."""
    ldx = _matrix(x, "x")
    rows, K = x.shape
    call = _Call(stream, x, seg_offsets, seg_padded_offsets, row_index, dev_status, out and out.codes,
                 out and out.scales, out_rows and out_rows.codes, out_rows and out_rows.scales)
    ri = so = sp = ds = None
    if row_index is not None:
        rows, ri = row_index.numel(), _ints(row_index, "row_index")
    if seg_offsets is not None:
        so = _ints(seg_offsets, "seg_offsets", nseg + 1)
    if seg_padded_offsets is not None:
        sp = _ints(seg_padded_offsets, "seg_padded_offsets", nseg + 1)
    if dev_status is not None:
        ds = _ints(dev_status, "dev_status")
    tiles = layout == NV4_F8_TILES
    if tiles and (nseg < 1 or rows % nseg):
        raise ValueError(f"{rows} rows are not {nseg} equal matrices")
    if out is None:
        if layout in (NV4_COLS, NV4_ROWS_AND_COLS):
            out = _new(call, K, out_K if out_K is not None else mx_cols_capacity(rows, nseg))
        else:
            out = _new(call, rows, K, nseg if tiles else 0)
    if layout == NV4_ROWS_AND_COLS and out_rows is None:
        out_rows = _new(call, rows, K)
    scaled = nseg if tiles else 0
    call(load().fp8_quantize, x.data_ptr(), _float(x, "x"), x.shape[0], rows, K, ldx, ri, layout, nseg, so, sp, rule,
         out.c(scaled), None if out_rows is None else out_rows.c(0), ds)
    out.nseg, out.rule, out.rows_out = scaled, rule, out_rows
    if out_rows is not None:
        out_rows.nseg, out_rows.rule, out_rows.rows_out = 0, rule, None
    return out


def fp8_dequantize(q: FP8, out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of q, [rows, K] BF16 or FP32 (code * scale rounded to FP32, and that to BF16)."""
    call = _Call(stream, q.codes, q.scales, out)
    if out is None:
        out = call.empty(out_dtype, q.rows, q.K)
        ldo = q.K
    else:
        ldo = _matrix(out, "out")
        if out.shape != (q.rows, q.K):
            raise ValueError(f"out must be [{q.rows}, {q.K}]")
    call(load().fp8_dequantize, q.c(), out.data_ptr(), _float(out, "out"), ldo)
    return out


def fp8_transpose(q: FP8, out: FP8 | None = None, stream=None) -> FP8:
    """Each of q's nseg matrices transposed (128 x 128 blocks: codes and scales move as they are)."""
    call = _Call(stream, q.codes, q.scales, out and out.codes, out and out.scales)
    if q.nseg < 1:
        raise ValueError("fp8_transpose needs a tensor scaled in 128 x 128 blocks")
    if out is None:
        out = _new(call, q.nseg * q.K, q.rows // q.nseg, q.nseg)
    call(load().fp8_transpose, q.c(), out.c(q.nseg))
    out.nseg, out.rule, out.rows_out = q.nseg, q.rule, None
    return out


# ----------------------------------------------------------------------------- grouped GEMM

def fp8_grouped_gemm(A: FP8, B: FP8, offsets: torch.Tensor, E: int, N: int, M_cap: int | None = None,
                     a_rows: torch.Tensor | None = None, group_mode: int = NV4_GROUP_M, epilogue: int = NV4_EPI_NONE,
                     out_dtype=torch.float32, C: torch.Tensor | None = None, q_out: FP8 | None = None,
                     rule: int = NV4_F8_FP32, want_c: bool = True, stream=None) -> torch.Tensor | None:
    """GROUP_M: C [M_cap, N] = per-expert A_e . B_e^T (SwiGLU: N output columns from 2N rows of
    B per expert).  GROUP_K: C [E, A.rows, B.rows] over per-expert K ranges.  q_out (SwiGLU):
    also the FP8 form of the result under `rule`; with want_c=False that alone.  A block of q_out that is not
    finite has the scale NaN (there is no dev_status)."""
    call = _Call(stream, A.codes, A.scales, B.codes, B.scales, offsets, a_rows, C, q_out and q_out.codes,
                 q_out and q_out.scales)
    if group_mode == NV4_GROUP_K:
        M_cap, N, shape = 0, A.rows, (E, A.rows, B.rows)
    else:
        if M_cap is None:
            M_cap = A.rows if a_rows is None else a_rows.numel()
        shape = (M_cap, N)
        if a_rows is not None and a_rows.numel() < M_cap:
            raise ValueError("a_rows must name a row of A for each of the M_cap rows")
    ldc, ctype = 0, NV4_F32
    if C is not None:
        ctype = _float(C, "C")
        if group_mode == NV4_GROUP_K:
            if C.shape != shape or not C.is_contiguous():
                raise ValueError(f"C must be {list(shape)} and contiguous")
            ldc = shape[-1]
        else:
            if C.dim() != 2 or C.shape[0] < M_cap or C.shape[1] != N:
                raise ValueError(f"C must be {list(shape)} with contiguous rows")
            ldc = _matrix(C, "C")
    elif want_c:
        C = call.empty(out_dtype, *shape)
        ctype, ldc = _float(C, "C"), shape[-1]
    call(load().fp8_grouped_gemm, A.c(), B.c(), _ints(offsets, "offsets", E + 1), E, M_cap, N,
         None if a_rows is None else _ints(a_rows, "a_rows"), group_mode, epilogue, _p(C), ctype, ldc,
         None if q_out is None else q_out.c(0), rule)
    if q_out is not None:
        q_out.nseg, q_out.rule, q_out.rows_out = 0, rule, None
    return C


# ----------------------------------------------------------------------------- layer composition

@dataclass
class F8ExpertWeights:
    """Quantised expert weights in 128 x 128 blocks: W13 [E*2I, H] (per expert gate rows, then up
    rows), W2 [E*H, I]."""
    w13: FP8
    w2: FP8
    E: int
    H: int
    I: int


@dataclass
class F8TransposedWeights:
    """The same values transposed (the operands of the data gradients): W2^T [E*I, H] and
    W13^T [E*H, 2I]."""
    w2t: FP8
    w13t: FP8


def fp8_quantize_expert_weights(W13: torch.Tensor, W2: torch.Tensor, rule: int = NV4_F8_FP32,
                                stream=None) -> F8ExpertWeights:
    """W13 [E, 2I, H] and W2 [E, H, I] (BF16 or FP32) -> FP8 in 128 x 128 blocks of each expert's
    matrix (with I % 128 == 0 none holds both gate and up rows)."""
    E, I2, H = _weight_shapes(W13, W2)
    t = dict(layout=NV4_F8_TILES, nseg=E, rule=rule)
    with _Layer(stream, W13) as layer:  # (weights whose rows are not in one stride are copied here)
        return F8ExpertWeights(layer.made(fp8_quantize(W13.reshape(E * I2, H), **t)),
                               layer.made(fp8_quantize(W2.reshape(E * H, I2 // 2), **t)), E, H, I2 // 2)


def fp8_transpose_expert_weights(w: F8ExpertWeights, stream=None) -> F8TransposedWeights:
    """The transposes that fp8_moe_backward multiplies by: the forward's own values."""
    with _Layer(stream, w.w13.codes) as layer:
        return F8TransposedWeights(layer.made(fp8_transpose(w.w2)), layer.made(fp8_transpose(w.w13)))


@dataclass
class F8ForwardBuffers:
    """Every intermediate of one forward, preallocated so that a forward enqueues kernels only."""
    xq: FP8
    hq: FP8
    hact: torch.Tensor | None   # [R, I] BF16 SwiGLU output, kept when a backward follows
    y: torch.Tensor             # [R, H] expert rows
    out: torch.Tensor           # [T, H]
    pws: torch.Tensor
    rule: int
    routing: Routing | None = None


def fp8_alloc_forward(T: int, H: int, E: int, k: int, I: int, out_dtype=torch.bfloat16, y_dtype=torch.float32,
                      keep_hact: bool = False, rule: int = NV4_F8_FP32, device="cuda") -> F8ForwardBuffers:
    """keep_hact: also keep the BF16 SwiGLU output, which fp8_moe_backward quantises along the
    tokens.  y_dtype: the type of the expert rows between the down product and the combine."""
    R = T * k
    return F8ForwardBuffers(
        xq=FP8.empty(T, H, device=device), hq=FP8.empty(R, I, device=device),
        hact=torch.empty((R, I), dtype=torch.bfloat16, device=device) if keep_hact else None,
        y=torch.empty((R, H), dtype=y_dtype, device=device), out=torch.empty((T, H), dtype=out_dtype, device=device),
        pws=torch.empty(load().moe_permute_workspace(T, E, k), dtype=torch.uint8, device=device), rule=rule)


def fp8_moe_forward(x: torch.Tensor, logits: torch.Tensor, w: F8ExpertWeights, k: int,
                    bufs: F8ForwardBuffers | None = None, flags: int = 0, stream=None,
                    stage_events: list | None = None) -> F8ForwardBuffers:
    """One FP8 expert-layer forward: quantise x, route and permute, gate and up products with
    SwiGLU and re-quantisation in the epilogue, down product, combine (``out``).  As the other layers it takes no
    dev_status: NaN and infinity of x show as NaN in their tokens' rows of out."""
    T, H = x.shape
    R = T * k
    if H != w.H:
        raise ValueError(f"x has {H} columns, the weights {w.H}")
    if logits.shape != (T, w.E):
        raise ValueError(f"logits must be [{T}, {w.E}]")
    if bufs is not None:
        rt = bufs.routing
        if bufs.xq.rows != T or bufs.hq.rows != R or bufs.out.shape != x.shape or not bufs.out.is_contiguous() or \
                rt is not None and (rt.topk_ids.shape != (T, k) or rt.offsets.numel() != w.E + 1):
            raise ValueError(f"bufs are not those of {T} rows of {H} and {k} of {w.E} experts")
    with _Layer(stream, x) as layer:
        st = layer.stream
        if bufs is None:
            bufs = layer.made(fp8_alloc_forward(T, H, w.E, k, w.I, device=x.device))
        with _Stage(stage_events, "quantize_x", st):
            fp8_quantize(x, out=bufs.xq, rule=bufs.rule)
        with _Stage(stage_events, "route_permute", st):
            rt = moe_permute(logits, w.E, k, flags=flags, ws=bufs.pws, out=bufs.routing)
            bufs.routing = layer.made(rt) if bufs.routing is None else rt
        with _Stage(stage_events, "gemm1_swiglu", st):
            fp8_grouped_gemm(bufs.xq, w.w13, rt.offsets, w.E, w.I, M_cap=R, a_rows=rt.row_token,
                             epilogue=NV4_EPI_SWIGLU, C=bufs.hact, want_c=False, q_out=bufs.hq, rule=bufs.rule)
        with _Stage(stage_events, "gemm2", st):
            fp8_grouped_gemm(bufs.hq, w.w2, rt.offsets, w.E, H, M_cap=R, C=bufs.y)
        with _Stage(stage_events, "combine", st):
            moe_combine(bufs.y, rt.token_row, rt.topk_w, out=bufs.out)
    return bufs


@dataclass
class F8BackwardBuffers:
    """Every intermediate and result of one backward (preallocated)."""
    dy2q: FP8               # [R, H]
    dy13q: FP8              # [R, 2I]
    dy2c: FP8               # [H, Kcap]
    hc: FP8                 # [I, Kcap]
    dy13c: FP8              # [2I, Kcap]
    xc: FP8                 # [H, Kcap]
    padded: torch.Tensor    # [E+1] int32
    dhact: torch.Tensor     # [R, I]
    dxperm: torch.Tensor    # [R, H]
    dw2: torch.Tensor       # [E, H, I]
    dw13: torch.Tensor      # [E, 2I, H]


def fp8_alloc_backward(T: int, H: int, E: int, k: int, I: int, dgrad_dtype=torch.bfloat16, wgrad_dtype=torch.float32,
                       device="cuda") -> F8BackwardBuffers:
    R = T * k
    kc = mx_cols_capacity(R, E)
    e = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=device)
    q = lambda rows, K: FP8.empty(rows, K, device=device)
    return F8BackwardBuffers(
        dy2q=q(R, H), dy13q=q(R, 2 * I), dy2c=q(H, kc), hc=q(I, kc), dy13c=q(2 * I, kc), xc=q(H, kc),
        padded=e(E + 1, dtype=torch.int32), dhact=e(R, I, dtype=dgrad_dtype), dxperm=e(R, H, dtype=dgrad_dtype),
        dw2=e(E, H, I, dtype=wgrad_dtype), dw13=e(E, 2 * I, H, dtype=wgrad_dtype))


def fp8_moe_backward(x: torch.Tensor, fwd: F8ForwardBuffers, wt: F8TransposedWeights, dY2: torch.Tensor,
                     dY13: torch.Tensor, bufs: F8BackwardBuffers | None = None, stream=None,
                     stage_events: list | None = None) -> F8BackwardBuffers:
    """The four backward grouped GEMMs of ``moe_backward`` on FP8 operands: gradients and activations
    quantised along their contraction dimension, the forward's weights transposed.  dY2 [R, H]
    and dY13 [R, 2I] are the gradients of the down and the gate/up output rows in expert (permuted)
    row order; the forward kept its SwiGLU output (keep_hact).  SwiGLU's own gradient, which makes dY13 from
    dhact and the gate and up rows, is the caller's, as in the other layers."""
    if fwd.hact is None:
        raise ValueError("the forward kept no SwiGLU output: fp8_alloc_forward(keep_hact=True)")
    T, H = x.shape
    rt = fwd.routing
    E, R, I = rt.offsets.numel() - 1, rt.row_token.numel(), fwd.hact.shape[1]
    if rt.topk_ids.shape[0] != T:
        raise ValueError(f"x has {T} rows, the forward's {rt.topk_ids.shape[0]}")
    if dY2.shape != (R, H) or dY13.shape != (R, 2 * I):
        raise ValueError(f"dY2 must be [{R}, {H}] and dY13 [{R}, {2 * I}]")
    with _Layer(stream, x) as layer:
        st = layer.stream
        if bufs is None:
            bufs = layer.made(fp8_alloc_backward(T, H, E, R // T, I, device=x.device))
        seg = dict(nseg=E, seg_offsets=rt.offsets, seg_padded_offsets=bufs.padded, rule=fwd.rule)
        with _Stage(stage_events, "quantize_dy2", st):
            mx_padded_offsets(rt.offsets, out=bufs.padded)
            fp8_quantize(dY2, layout=NV4_ROWS_AND_COLS, out=bufs.dy2c, out_rows=bufs.dy2q, **seg)
        with _Stage(stage_events, "quantize_dy13", st):
            fp8_quantize(dY13, layout=NV4_ROWS_AND_COLS, out=bufs.dy13c, out_rows=bufs.dy13q, **seg)
        with _Stage(stage_events, "dgrad_hact", st):
            fp8_grouped_gemm(bufs.dy2q, wt.w2t, rt.offsets, E, I, M_cap=R, C=bufs.dhact)
        with _Stage(stage_events, "dgrad_x", st):
            fp8_grouped_gemm(bufs.dy13q, wt.w13t, rt.offsets, E, H, M_cap=R, C=bufs.dxperm)
        with _Stage(stage_events, "quantize_cols_hact", st):
            fp8_quantize(fwd.hact, layout=NV4_COLS, out=bufs.hc, **seg)
        with _Stage(stage_events, "wgrad_w2", st):
            fp8_grouped_gemm(bufs.dy2c, bufs.hc, bufs.padded, E, H, group_mode=NV4_GROUP_K, C=bufs.dw2)
        with _Stage(stage_events, "quantize_cols_x", st):
            fp8_quantize(x, layout=NV4_COLS, out=bufs.xc, row_index=rt.row_token, **seg)
        with _Stage(stage_events, "wgrad_w13", st):
            fp8_grouped_gemm(bufs.dy13c, bufs.xc, bufs.padded, E, 2 * I, group_mode=NV4_GROUP_K, C=bufs.dw13)
    return bufs

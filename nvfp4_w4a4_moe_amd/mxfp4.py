"""MXFP4 calls of the binding (include/nv4moe/mxfp4.h): blocks of 32 E2M1 codes under one
power-of-two scale, the 4-bit format gfx950's matrix instructions multiply as it is stored.

    mxfp4_quantize      quantisation (rows, columns by segment, both, batched columns)
    mxfp4_dequantize    the values, BF16 or FP32 (exact)
    mx_padded_offsets   segment starts for the column layouts
    mxfp4_grouped_gemm  grouped product (GROUP_M with optional SwiGLU and fused
                        re-quantisation, GROUP_K)
    mx_moe_few          a whole expert layer for at most 64 tokens

``mx_moe_forward`` and ``mx_moe_backward`` compose them with moe_permute and moe_combine as
``moe_forward`` and ``moe_backward`` do for NVFP4.  Everything here is reachable from the
package's top level.

Matrices may have any row stride of at least their width.  With ``stream`` a call, or a whole
layer, runs on that stream, and what it allocates comes from that stream's pool; the stream waits
for no other, so inputs have to be ready there and results be waited for by whoever reads them.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
from dataclasses import dataclass, is_dataclass

import torch

from . import (NV4_BF16, NV4_COLS, NV4_COLS_BATCHED, NV4_EPI_NONE, NV4_EPI_SWIGLU, NV4_F32, NV4_GROUP_K, NV4_GROUP_M,
               NV4_ROWS, NV4_ROWS_AND_COLS, Routing, _check, _I, _I64, _P, _SIGS, _Stage, _SZ, load,
               moe_combine, moe_permute)

NV4_MX_FLOOR, NV4_MX_CEIL = 0, 1
NV4_MX_SEGMENT = 128
NV4_MX_FEW_TOKENS = 64

__all__ = ["NV4_MX_FLOOR", "NV4_MX_CEIL", "NV4_MX_SEGMENT", "NV4_MX_FEW_TOKENS", "MXTensor", "MXFP4",
           "mxfp4_scale_stride", "mxfp4_quantize", "mxfp4_dequantize", "mx_padded_offsets", "mx_cols_capacity",
           "mxfp4_grouped_gemm", "MXExpertWeights", "MXTransposedWeights", "mx_quantize_expert_weights",
           "mx_quantize_expert_weights_t", "MXForwardBuffers", "mx_alloc_forward", "mx_moe_forward",
           "MXBackwardBuffers", "mx_alloc_backward", "mx_moe_backward", "mx_moe_few"]


class MXTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("K", ctypes.c_int64)]


_T = ctypes.POINTER(MXTensor)
_SIGS.update({
    "mxfp4_scale_stride": (_I64, [_I64]),
    "mxfp4_quantize": (_I, [_P, _I, _I64, _I64, _I64, _I64, _P, _I, _I, _P, _P, _I, _T, _T, _P, _P]),
    "mxfp4_dequantize": (_I, [_T, _P, _I, _I64, _P]),
    "mx_padded_offsets": (_I, [_P, _I, _P, _P]),
    "mxfp4_grouped_gemm": (_I, [_T, _T, _P, _I, _I64, _I64, _P, _I, _I, _P, _I, _I64, _T, _I, _P]),
    "mx_moe_few_workspace": (_SZ, [_I64, _I, _I, _I64, _I64]),
    "mx_moe_few": (_I, [_P, _I, _I64, _P, _I64, _I, _I, _I, _P, _P, _T, _T, _I64, _I64, _I, _P, _I, _I64, _P, _SZ, _P,
                        _P]),
})


_U8 = torch.uint8


def mxfp4_scale_stride(K: int) -> int:
    """Bytes between two rows of scales: K/32 rounded up to a multiple of 4."""
    return (K // 32 + 3) // 4 * 4


@dataclass
class MXFP4:
    """Device MXFP4 tensor: codes [rows, K/2] u8, scales [rows, mxfp4_scale_stride(K)] u8
    (E8M0, zeros behind the last block)."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    K: int
    rows_out: "MXFP4 | None" = None  # the row-direction output of NV4_ROWS_AND_COLS

    @staticmethod
    def empty(rows: int, K: int, device="cuda") -> "MXFP4":
        return MXFP4(torch.empty((rows, K // 2), dtype=torch.uint8, device=device),
                     torch.empty((rows, mxfp4_scale_stride(K)), dtype=torch.uint8, device=device), rows, K)

    def own(self) -> MXTensor:
        """c() of a tensor that the binding has just made."""
        return MXTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.K)

    def c(self) -> MXTensor:
        c, s, rows, K = self.codes, self.scales, self.rows, self.K
        if not (c.dtype is s.dtype is _U8 and c.is_contiguous() and s.is_contiguous() and
                c.numel() == rows * (K // 2) and s.numel() == rows * ((K // 32 + 3) // 4 * 4)):
            raise ValueError(f"MXFP4 [{rows}, {K}] needs contiguous uint8 codes and scales of its shape")
        return MXTensor(c.data_ptr(), s.data_ptr(), rows, K)


# ----------------------------------------------------------------------------- arguments

_TYPES = {torch.bfloat16: NV4_BF16, torch.float32: NV4_F32}


def _float(t: torch.Tensor, name: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be BF16 or FP32, not {t.dtype}")
    return code


def _matrix(t: torch.Tensor, name: str) -> int:
    """The row stride of a 2-D tensor with contiguous rows (the width where there is one row at
    most, whose stride means nothing)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    if shape[0] <= 1:
        return shape[1]
    if stride[0] < shape[1]:
        raise ValueError(f"{name} has rows that overlap (row stride {stride[0]}, width {shape[1]})")
    return stride[0]


def _ints(t: torch.Tensor | None, name: str, n: int | None = None):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be contiguous int32" + ("" if n is None else f" of {n} elements"))
    return t.data_ptr()


# the device's current stream as an address, without the Stream object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


class _Call:
    """One call's device and stream: every tensor has to be on the device of the first one, and the
    launch goes to the given stream or to that device's current one.  Memory comes from the pool
    of that stream: a block of the current stream's pool may still be in use by kernels queued
    there, which another stream does not wait for."""

    __slots__ = ("index", "device", "given", "stream")

    def __init__(self, stream, first: torch.Tensor, *others):
        index = first.get_device()
        for t in others:
            if t is not None and t.get_device() != index:
                raise ValueError(f"tensors on {first.device} and {t.device} in one call")
        self.device = first.device
        if not first.is_cuda:
            raise ValueError(f"tensors must be on a GPU, not on {first.device}")
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream of {stream.device} for tensors on {self.device}")
        self.index, self.given = index, None
        self.stream = _raw_stream(index)
        if stream is not None and stream.cuda_stream != self.stream:
            self.given, self.stream = stream, stream.cuda_stream

    def scratch(self, dtype, *shape) -> torch.Tensor:
        """Memory that the call alone uses: free for the stream's next work when the call returns."""
        if self.given is None:
            return torch.empty(*shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.given):
            return torch.empty(*shape, dtype=dtype, device=self.device)

    def empty(self, dtype, *shape) -> torch.Tensor:
        """An output: the caller's stream, where it is read next, keeps it from reuse as well."""
        t = self.scratch(dtype, *shape)
        if self.given is not None:
            t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def mx(self, rows: int, K: int) -> MXFP4:
        return MXFP4(self.empty(_U8, rows, K // 2), self.empty(_U8, rows, (K // 32 + 3) // 4 * 4), rows, K)

    def __call__(self, fn, *args):
        if torch.cuda.current_device() == self.index:
            status = fn(*args, self.stream)
        else:
            with torch.cuda.device(self.index):
                status = fn(*args, self.stream)
        if status:
            _check(status)


def _p(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=None)
def _few_workspace(T: int, E: int, k: int, H: int, I: int) -> int:
    return load().mx_moe_few_workspace(T, E, k, H, I)


# ----------------------------------------------------------------------------- quantisation

def mx_cols_capacity(R: int, E: int) -> int:
    """Column capacity of a segment-transposed operand: R rows, each of E segments padded to
    NV4_MX_SEGMENT."""
    return (R + (NV4_MX_SEGMENT - 1) * E + NV4_MX_SEGMENT - 1) // NV4_MX_SEGMENT * NV4_MX_SEGMENT


def mx_padded_offsets(offsets: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Segment starts with every segment padded to NV4_MX_SEGMENT, from int32 offsets [nseg+1]."""
    call = _Call(stream, offsets, out)
    if out is None:
        out = call.empty(torch.int32, *offsets.shape)
    n = offsets.numel()
    call(load().mx_padded_offsets, _ints(offsets, "offsets"), n - 1, _ints(out, "out", n))
    return out


def mxfp4_quantize(x: torch.Tensor, layout: int = NV4_ROWS, nseg: int = 1, seg_offsets: torch.Tensor | None = None,
                   seg_padded_offsets: torch.Tensor | None = None, row_index: torch.Tensor | None = None,
                   out: MXFP4 | None = None, out_K: int | None = None, out_rows: MXFP4 | None = None,
                   rule: int = NV4_MX_FLOOR, dev_status: torch.Tensor | None = None, stream=None) -> MXFP4:
    """MXFP4-quantise a 2-D BF16/FP32 tensor (row stride x.stride(0)).  With row_index (int32),
    logical row r is x row row_index[r].  NV4_ROWS_AND_COLS returns the column output with the
    row output in its `rows_out` (out_rows, allocated when None)."""
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
    if out is not None:
        c = out.c()
    else:
        if layout == NV4_COLS_BATCHED:
            out = call.mx(nseg * K, rows // max(nseg, 1))
        elif layout == NV4_ROWS:
            out = call.mx(rows, K)
        else:
            out = call.mx(K, out_K if out_K is not None else mx_cols_capacity(rows, nseg))
        c = out.own()
    if layout == NV4_ROWS_AND_COLS and out_rows is None:
        out_rows = call.mx(rows, K)
    call(load().mxfp4_quantize, x.data_ptr(), _float(x, "x"), x.shape[0], rows, K, ldx, ri, layout, nseg, so, sp, rule,
         c, None if out_rows is None else out_rows.c(), ds)
    out.rows_out = out_rows
    return out


def mxfp4_dequantize(q: MXFP4, out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of q, [rows, K] BF16 or FP32 (both hold them exactly)."""
    call = _Call(stream, q.codes, q.scales, out)
    if out is None:
        out = call.empty(out_dtype, q.rows, q.K)
        ldo = q.K
    else:
        ldo = _matrix(out, "out")
        if out.shape != (q.rows, q.K):
            raise ValueError(f"out must be [{q.rows}, {q.K}]")
    call(load().mxfp4_dequantize, q.c(), out.data_ptr(), _float(out, "out"), ldo)
    return out


# ----------------------------------------------------------------------------- grouped GEMM

def mxfp4_grouped_gemm(A: MXFP4, B: MXFP4, offsets: torch.Tensor, E: int, N: int, M_cap: int | None = None,
                       a_rows: torch.Tensor | None = None, group_mode: int = NV4_GROUP_M, epilogue: int = NV4_EPI_NONE,
                       out_dtype=torch.float32, C: torch.Tensor | None = None, q_out: MXFP4 | None = None,
                       rule: int = NV4_MX_FLOOR, want_c: bool = True, stream=None) -> torch.Tensor | None:
    """GROUP_M: C [M_cap, N] = per-expert A_e . B_e^T (SwiGLU: N output columns from 2N rows of
    B per expert).  GROUP_K: C [E, A.rows, B.rows] over per-expert K ranges.  q_out (SwiGLU):
    also the MXFP4 form of the result; with want_c=False that alone."""
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
    call(load().mxfp4_grouped_gemm, A.c(), B.c(), _ints(offsets, "offsets", E + 1), E, M_cap, N,
         None if a_rows is None else _ints(a_rows, "a_rows"), group_mode, epilogue, _p(C), ctype, ldc,
         None if q_out is None else q_out.c(), rule)
    return C


# ----------------------------------------------------------------------------- layer composition

class _Layer:
    """Makes the given stream, or else the tensors' device, current while a layer's calls are queued
    there: what they allocate comes from that stream's pool (as for one call, see _Call), and the
    calls that know only the current device find it."""

    def __init__(self, stream, x: torch.Tensor):
        if not x.is_cuda:
            raise ValueError(f"tensors must be on a GPU, not on {x.device}")
        if stream is not None and stream.device != x.device:
            raise ValueError(f"stream of {stream.device} for tensors on {x.device}")
        self.caller = torch.cuda.current_stream(x.device)
        if stream is not None and stream != self.caller:
            self.on = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != x.get_device():
            self.on = torch.cuda.device(x.device)
        else:
            self.on = contextlib.nullcontext()

    def __enter__(self):
        self.on.__enter__()
        self.stream = torch.cuda.current_stream()
        return self

    def __exit__(self, *exc):
        return self.on.__exit__(*exc)

    def made(self, bufs):
        """`bufs`, which the layer has allocated and returns: the caller's stream keeps their tensors
        from reuse as well."""
        if self.stream != self.caller:
            for v in vars(bufs).values():
                if isinstance(v, torch.Tensor):
                    v.record_stream(self.caller)
                elif is_dataclass(v):  # a quantised tensor
                    self.made(v)
        return bufs


@dataclass
class MXExpertWeights:
    """Quantised expert weights: W13 [E*2I, H] (per expert gate rows, then up rows), W2 [E*H, I]."""
    w13: MXFP4
    w2: MXFP4
    E: int
    H: int
    I: int


def _weight_shapes(W13: torch.Tensor, W2: torch.Tensor):
    E, I2, H = W13.shape
    if I2 % 2 or W2.shape not in ((E, H, I2 // 2), (E * H, I2 // 2)):
        raise ValueError(f"W13 [E, 2I, H] and W2 [E, H, I] must fit together, not {list(W13.shape)} and {list(W2.shape)}")
    return E, I2, H


@dataclass
class MXTransposedWeights:
    """Expert weights transposed and re-quantised along their new contraction dimension (the
    operands of the data gradients): W2^T [E*I, H] and W13^T [E*H, 2I]."""
    w2t: MXFP4
    w13t: MXFP4


def mx_quantize_expert_weights(W13: torch.Tensor, W2: torch.Tensor, rule: int = NV4_MX_FLOOR,
                               stream=None) -> MXExpertWeights:
    """W13 [E, 2I, H] and W2 [E, H, I] (BF16 or FP32) -> MXFP4 along their last dimension."""
    E, I2, H = _weight_shapes(W13, W2)
    with _Layer(stream, W13) as layer:  # (weights whose rows are not in one stride are copied here)
        return MXExpertWeights(layer.made(mxfp4_quantize(W13.reshape(E * I2, H), rule=rule)),
                               layer.made(mxfp4_quantize(W2.reshape(E * H, I2 // 2), rule=rule)), E, H, I2 // 2)


def mx_quantize_expert_weights_t(W13: torch.Tensor, W2: torch.Tensor, rule: int = NV4_MX_FLOOR,
                                 stream=None) -> MXTransposedWeights:
    """W13 [E, 2I, H] and W2 [E, H, I] -> per-expert transposes in MXFP4."""
    E, I2, H = _weight_shapes(W13, W2)
    t = dict(layout=NV4_COLS_BATCHED, nseg=E, rule=rule)
    with _Layer(stream, W13) as layer:
        return MXTransposedWeights(layer.made(mxfp4_quantize(W2.reshape(E * H, I2 // 2), **t)),
                                   layer.made(mxfp4_quantize(W13.reshape(E * I2, H), **t)))


@dataclass
class MXForwardBuffers:
    """Every intermediate of one forward, preallocated so that a forward enqueues kernels only."""
    xq: MXFP4
    hq: MXFP4
    hact: torch.Tensor | None   # [R, I] BF16 SwiGLU output, kept when a backward follows
    y: torch.Tensor             # [R, H] expert rows
    out: torch.Tensor           # [T, H]
    pws: torch.Tensor
    rule: int
    routing: Routing | None = None


def mx_alloc_forward(T: int, H: int, E: int, k: int, I: int, out_dtype=torch.bfloat16, y_dtype=torch.float32,
                     keep_hact: bool = False, rule: int = NV4_MX_FLOOR, device="cuda") -> MXForwardBuffers:
    """keep_hact: also keep the BF16 SwiGLU output, which mx_moe_backward quantises along the
    tokens.  y_dtype: the type of the expert rows between the down product and the combine."""
    R = T * k
    return MXForwardBuffers(
        xq=MXFP4.empty(T, H, device), hq=MXFP4.empty(R, I, device),
        hact=torch.empty((R, I), dtype=torch.bfloat16, device=device) if keep_hact else None,
        y=torch.empty((R, H), dtype=y_dtype, device=device), out=torch.empty((T, H), dtype=out_dtype, device=device),
        pws=torch.empty(load().moe_permute_workspace(T, E, k), dtype=torch.uint8, device=device), rule=rule)


def mx_moe_forward(x: torch.Tensor, logits: torch.Tensor, w: MXExpertWeights, k: int,
                   bufs: MXForwardBuffers | None = None, flags: int = 0, stream=None,
                   stage_events: list | None = None) -> MXForwardBuffers:
    """One MXFP4 expert-layer forward: quantise x, route and permute, gate and up products with
    SwiGLU and re-quantisation in the epilogue, down product, combine (``out``)."""
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
            bufs = layer.made(mx_alloc_forward(T, H, w.E, k, w.I, device=x.device))
        with _Stage(stage_events, "quantize_x", st):
            mxfp4_quantize(x, out=bufs.xq, rule=bufs.rule)
        with _Stage(stage_events, "route_permute", st):
            rt = moe_permute(logits, w.E, k, flags=flags, ws=bufs.pws, out=bufs.routing)
            bufs.routing = layer.made(rt) if bufs.routing is None else rt
        with _Stage(stage_events, "gemm1_swiglu", st):
            mxfp4_grouped_gemm(bufs.xq, w.w13, rt.offsets, w.E, w.I, M_cap=R, a_rows=rt.row_token,
                               epilogue=NV4_EPI_SWIGLU, C=bufs.hact, want_c=False, q_out=bufs.hq, rule=bufs.rule)
        with _Stage(stage_events, "gemm2", st):
            mxfp4_grouped_gemm(bufs.hq, w.w2, rt.offsets, w.E, H, M_cap=R, C=bufs.y)
        with _Stage(stage_events, "combine", st):
            moe_combine(bufs.y, rt.token_row, rt.topk_w, out=bufs.out)
    return bufs


@dataclass
class MXBackwardBuffers:
    """Every intermediate and result of one backward (preallocated)."""
    dy2q: MXFP4             # [R, H]
    dy13q: MXFP4            # [R, 2I]
    dy2c: MXFP4             # [H, Kcap]
    hc: MXFP4               # [I, Kcap]
    dy13c: MXFP4            # [2I, Kcap]
    xc: MXFP4               # [H, Kcap]
    padded: torch.Tensor    # [E+1] int32
    dhact: torch.Tensor     # [R, I]
    dxperm: torch.Tensor    # [R, H]
    dw2: torch.Tensor       # [E, H, I]
    dw13: torch.Tensor      # [E, 2I, H]


def mx_alloc_backward(T: int, H: int, E: int, k: int, I: int, dgrad_dtype=torch.bfloat16, wgrad_dtype=torch.float32,
                      device="cuda") -> MXBackwardBuffers:
    R = T * k
    kc = mx_cols_capacity(R, E)
    e = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=device)
    return MXBackwardBuffers(
        dy2q=MXFP4.empty(R, H, device), dy13q=MXFP4.empty(R, 2 * I, device), dy2c=MXFP4.empty(H, kc, device),
        hc=MXFP4.empty(I, kc, device), dy13c=MXFP4.empty(2 * I, kc, device), xc=MXFP4.empty(H, kc, device),
        padded=e(E + 1, dtype=torch.int32), dhact=e(R, I, dtype=dgrad_dtype), dxperm=e(R, H, dtype=dgrad_dtype),
        dw2=e(E, H, I, dtype=wgrad_dtype), dw13=e(E, 2 * I, H, dtype=wgrad_dtype))


def mx_moe_backward(x: torch.Tensor, fwd: MXForwardBuffers, wt: MXTransposedWeights, dY2: torch.Tensor,
                    dY13: torch.Tensor, bufs: MXBackwardBuffers | None = None, stream=None,
                    stage_events: list | None = None) -> MXBackwardBuffers:
    """The four backward grouped GEMMs of ``moe_backward`` on MXFP4 operands, each re-quantised
    along its contraction dimension.  dY2 [R, H] and dY13 [R, 2I] are the gradients of the down
    and the gate/up output rows in expert (permuted) row order; the forward kept its SwiGLU
    output (keep_hact)."""
    if fwd.hact is None:
        raise ValueError("the forward kept no SwiGLU output: mx_alloc_forward(keep_hact=True)")
    T, H = x.shape
    rt = fwd.routing
    E, R, I = rt.offsets.numel() - 1, rt.row_token.numel(), fwd.hact.shape[1]
    if rt.topk_ids.shape[0] != T:
        raise ValueError(f"x has {T} rows, the forward's {rt.topk_ids.shape[0]}")
    with _Layer(stream, x) as layer:
        st = layer.stream
        if bufs is None:
            bufs = layer.made(mx_alloc_backward(T, H, E, R // T, I, device=x.device))
        seg = dict(nseg=E, seg_offsets=rt.offsets, seg_padded_offsets=bufs.padded, rule=fwd.rule)
        with _Stage(stage_events, "quantize_dy2", st):
            mx_padded_offsets(rt.offsets, out=bufs.padded)
            mxfp4_quantize(dY2, layout=NV4_ROWS_AND_COLS, out=bufs.dy2c, out_rows=bufs.dy2q, **seg)
        with _Stage(stage_events, "quantize_dy13", st):
            mxfp4_quantize(dY13, layout=NV4_ROWS_AND_COLS, out=bufs.dy13c, out_rows=bufs.dy13q, **seg)
        with _Stage(stage_events, "dgrad_hact", st):
            mxfp4_grouped_gemm(bufs.dy2q, wt.w2t, rt.offsets, E, I, M_cap=R, C=bufs.dhact)
        with _Stage(stage_events, "dgrad_x", st):
            mxfp4_grouped_gemm(bufs.dy13q, wt.w13t, rt.offsets, E, H, M_cap=R, C=bufs.dxperm)
        with _Stage(stage_events, "quantize_cols_hact", st):
            mxfp4_quantize(fwd.hact, layout=NV4_COLS, out=bufs.hc, **seg)
        with _Stage(stage_events, "wgrad_w2", st):
            mxfp4_grouped_gemm(bufs.dy2c, bufs.hc, bufs.padded, E, H, group_mode=NV4_GROUP_K, C=bufs.dw2)
        with _Stage(stage_events, "quantize_cols_x", st):
            mxfp4_quantize(x, layout=NV4_COLS, out=bufs.xc, row_index=rt.row_token, **seg)
        with _Stage(stage_events, "wgrad_w13", st):
            mxfp4_grouped_gemm(bufs.dy13c, bufs.xc, bufs.padded, E, 2 * I, group_mode=NV4_GROUP_K, C=bufs.dw13)
    return bufs


# ----------------------------------------------------------------------------- a few tokens

def mx_moe_few(x: torch.Tensor, logits: torch.Tensor | None, w: MXExpertWeights, k: int,
               topk_ids: torch.Tensor | None = None, topk_w: torch.Tensor | None = None, flags: int = 0,
               out_dtype=torch.bfloat16, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
               rule: int = NV4_MX_FLOOR, dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The layer of ``mx_moe_forward`` for at most NV4_MX_FEW_TOKENS tokens (a decode step) in
    two to four kernels: x [T, H], logits FP32 [T, E] -> out [T, H].  With logits None, topk_ids
    (int32 [T, k]) and topk_w (FP32) are the routing; otherwise they receive it when given."""
    ldx = _matrix(x, "x")
    T, H = x.shape
    call = _Call(stream, x, logits, w.w13.codes, w.w13.scales, w.w2.codes, w.w2.scales, topk_ids, topk_w, out, ws,
                 dev_status)
    if H != w.H:
        raise ValueError(f"x has {H} columns, the weights {w.H}")
    if logits is not None and (logits.dtype != torch.float32 or not logits.is_contiguous() or
                               logits.shape != (T, w.E)):
        raise ValueError(f"logits must be contiguous FP32 [{T}, {w.E}]")
    if topk_w is not None and (topk_w.dtype != torch.float32 or not topk_w.is_contiguous() or topk_w.numel() != T * k):
        raise ValueError(f"topk_w must be contiguous FP32 [{T}, {k}]")
    if out is None:
        out = call.empty(out_dtype, T, H)
    elif out.shape != x.shape:
        raise ValueError(f"out must be [{T}, {H}]")
    if ws is None:
        ws = call.scratch(_U8, max(_few_workspace(T, w.E, k, H, w.I), 256))
    elif ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be contiguous uint8")
    call(load().mx_moe_few, x.data_ptr(), _float(x, "x"), ldx, _p(logits), T, w.E, k, flags,
         _ints(topk_ids, "topk_ids", T * k), _p(topk_w), w.w13.c(), w.w2.c(), H, w.I, rule, out.data_ptr(),
         _float(out, "out"), _matrix(out, "out"), ws.data_ptr(), ws.numel(), _ints(dev_status, "dev_status"))
    return out

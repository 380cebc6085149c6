"""The training side of the router (include/nv4moe/router.h):

    moe_balance_loss      per-expert counts, probability sums, the balance loss and the z loss
    moe_balance_backward  the gradient of the logits, of both losses and of the routing weights
    moe_combine_backward  the gradients of moe_combine: the expert rows' and the routing weights'

    rt = moe_permute(logits, E, k)                          # the forward's routing
    b = moe_balance_loss(logits, rt.topk_ids)               # total = loss + (coefs * b.loss).sum()
    dY, dw = moe_combine_backward(dout, y, rt.token_row, rt.topk_w)
    dlogits = moe_balance_backward(logits, rt.topk_ids, b, coefs, dtopk_w=dw)

Everything here is reachable from the package's top level; streams and memory are as in mxfp4.py.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _I, _I64, _P, _SIGS, _SZ, load
from .mxfp4 import _Call, _float, _ints, _matrix, _p

__all__ = ["MoeBalance", "moe_balance_loss", "moe_balance_backward", "moe_combine_backward"]

_SIGS.update({
    "moe_balance_workspace": (_SZ, [_I64, _I, _I]),
    "moe_balance_loss": (_I, [_P, _I64, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _SZ, _P, _P]),
    "moe_balance_backward": (_I, [_P, _I64, _I, _I, _P, _P, _I, _P, _P, _P, _P, _P, _I, _P, _P, _P]),
    "moe_combine_backward": (_I, [_P, _I, _P, _I, _I64, _I64, _P, _P, _I64, _I, _I64, _P, _I64, _P, _P]),
})


@dataclass
class MoeBalance:
    """What moe_balance_loss returns.  counts, prob_sums and tokens are sums over tokens: ranks of
    a data-parallel job may add theirs before moe_balance_backward."""
    loss: torch.Tensor       # [2] FP32: balance, z
    counts: torch.Tensor     # [nseg, E] int32
    prob_sums: torch.Tensor  # [nseg, E] FP32
    tokens: torch.Tensor     # [nseg] int32


def _floats(t: torch.Tensor | None, name: str, shape):
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be contiguous FP32 {list(shape)}")
    return t.data_ptr()


def _router(logits, topk_ids, mask, seg_offsets):
    """Shapes and pointers of what the loss and its gradient share."""
    if logits.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != logits.shape[0]:
        raise ValueError(f"logits [T, E] and topk_ids [T, k] must fit together, not {list(logits.shape)} and "
                         f"{list(topk_ids.shape)}")
    (T, E), k = logits.shape, topk_ids.shape[1]
    lg = _floats(logits, "logits", (T, E))
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous() or mask.shape != (T,)):
        raise ValueError(f"mask must be contiguous bool or uint8 [{T}]")
    if seg_offsets is not None and (seg_offsets.dim() != 1 or seg_offsets.numel() < 2):
        raise ValueError("seg_offsets must be [nseg + 1]")
    nseg = 1 if seg_offsets is None else seg_offsets.numel() - 1
    return T, E, k, nseg, (lg, T, E, k, _ints(topk_ids, "topk_ids"), _p(mask), nseg, _ints(seg_offsets, "seg_offsets"))


def moe_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, mask: torch.Tensor | None = None,
                     seg_offsets: torch.Tensor | None = None, out: MoeBalance | None = None,
                     ws: torch.Tensor | None = None, dev_status: torch.Tensor | None = None, stream=None) -> MoeBalance:
    """Counts and losses of the routing topk_ids (int32 [T, k]) of logits (FP32 [T, E]), over the
    tokens whose mask (bool [T]) is set, for each of the segments [seg_offsets[s], seg_offsets[s+1])
    (int32 [nseg+1]; None: all tokens as one).  loss[0] is 1 for even routing."""
    T, E, k, nseg, args = _router(logits, topk_ids, mask, seg_offsets)
    call = _Call(stream, logits, topk_ids, mask, seg_offsets, ws, dev_status, *(() if out is None else vars(out).values()))
    if out is None:
        out = MoeBalance(call.empty(torch.float32, 2), call.empty(torch.int32, nseg, E),
                         call.empty(torch.float32, nseg, E), call.empty(torch.int32, nseg))
    lib = load()
    if ws is None:
        ws = call.scratch(torch.uint8, lib.moe_balance_workspace(T, E, nseg))
    elif ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be contiguous uint8")
    call(lib.moe_balance_loss, *args, _ints(out.counts, "counts", nseg * E), _floats(out.prob_sums, "prob_sums", (nseg, E)),
         _ints(out.tokens, "tokens", nseg), _floats(out.loss, "loss", (2,)), ws.data_ptr(), ws.numel(),
         _ints(dev_status, "dev_status"))
    return out


def moe_balance_backward(logits: torch.Tensor, topk_ids: torch.Tensor, balance: MoeBalance | None = None,
                         dloss: torch.Tensor | None = None, dtopk_w: torch.Tensor | None = None,
                         mask: torch.Tensor | None = None, seg_offsets: torch.Tensor | None = None, flags: int = 0,
                         out: torch.Tensor | None = None, dev_status: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """The gradient of the logits [T, E]: of the two losses (dloss FP32 [2] on the device, with the
    counts and tokens of `balance`, mask and segments as in moe_balance_loss) and of the routing
    weights (dtopk_w FP32 [T, k], flags NV4_RENORM as moe_permute had it).  out may be logits."""
    T, E, k, nseg, args = _router(logits, topk_ids, mask, seg_offsets)
    if dloss is not None and balance is None:
        raise ValueError("dloss needs the counts and tokens of moe_balance_loss")
    counts, tokens = (balance.counts, balance.tokens) if dloss is not None else (None, None)
    call = _Call(stream, logits, topk_ids, mask, seg_offsets, counts, tokens, dloss, dtopk_w, out, dev_status)
    if out is None:
        out = call.empty(torch.float32, T, E)
    call(load().moe_balance_backward, *args, _ints(counts, "counts", nseg * E), _ints(tokens, "tokens", nseg),
         _floats(dloss, "dloss", (2,)), _floats(dtopk_w, "dtopk_w", (T, k)), flags, _floats(out, "out", (T, E)),
         _ints(dev_status, "dev_status"))
    return out


def moe_combine_backward(dout: torch.Tensor, Y: torch.Tensor, token_row: torch.Tensor, topk_w: torch.Tensor,
                         dY: torch.Tensor | None = None, dtopk_w: torch.Tensor | None = None, want_dy: bool = True,
                         want_dw: bool = True, stream=None):
    """The gradients of out = moe_combine(Y, token_row, topk_w): (dY [R, H] of Y's type, dtopk_w FP32
    [T, k]) from dout [T, H].  want_dy=False or want_dw=False: None in its place (unless its
    buffer is given).  Rows of dY that no token names are not written."""
    T, H = dout.shape
    if not dout.is_contiguous():
        raise ValueError("dout must be contiguous")
    if Y.dim() != 2 or Y.shape[1] != H:
        raise ValueError(f"Y must have {H} columns")
    if token_row.dim() != 2 or token_row.shape[0] != T:
        raise ValueError(f"token_row must be [{T}, k]")
    k = token_row.shape[1]
    call = _Call(stream, dout, Y, token_row, topk_w, dY, dtopk_w)
    if dY is None and want_dy:
        dY = call.empty(Y.dtype, *Y.shape)
    elif dY is not None and (dY.shape != Y.shape or dY.dtype != Y.dtype):
        raise ValueError(f"dY must be {list(Y.shape)} of Y's type")
    if dtopk_w is None and want_dw:
        dtopk_w = call.empty(torch.float32, T, k)
    call(load().moe_combine_backward, dout.data_ptr(), _float(dout, "dout"), Y.data_ptr(), _float(Y, "Y"), _matrix(Y, "Y"),
         Y.shape[0], _ints(token_row, "token_row"), _floats(topk_w, "topk_w", (T, k)), T, k, H, _p(dY),
         0 if dY is None else _matrix(dY, "dY"), _floats(dtopk_w, "dtopk_w", (T, k)))
    return dY, dtopk_w

"""MXFP4 block quantisation and its expert layer, written out step by step.

TEST INFRASTRUCTURE ONLY (see the package docstring).

MXFP4 is the OCP Microscaling (MX) v1.0 format of the E2M1 elements that the pages' NVFP4
also uses: 32 elements under one E8M0 scale 2^e, no tensor scale.  The specification leaves
the choice of e open and gives one rule:

    floor   e = floor(log2 max|v|) - 2, 2 being E2M1's largest exponent; elements above
            6 * 2^e saturate
    ceil    e = the smallest with max|v| <= 6 * 2^e

Readings taken: e is clamped to >= -127 (E8M0's smallest), an all-zero block has e = -127, and
a block with a NaN or infinity has scale byte 255 (E8M0's NaN) and codes 0.  Elements round to
the nearest E2M1 value, ties to the even code.
"""

from __future__ import annotations

import numpy as np

from . import formats as F
from . import moe

BLOCK = 32
SEGMENT = 128
FLOOR, CEIL = 0, 1


def scale_bytes(amax: np.ndarray, rule: int = FLOOR) -> np.ndarray:
    """E8M0 byte of each block from its max|v| (FP64 holding FP32 values)."""
    a = np.asarray(amax, np.float64)
    m, ex = np.frexp(np.where(np.isfinite(a) & (a > 0), a, 1.0))   # a = m 2^ex, m in [0.5, 1)
    e = ex - 1 - 2
    if rule == CEIL:
        e = e + (m > 0.75)                                         # a > 6 2^e = 0.75 2^ex
    b = np.clip(e, -127, 127) + 127
    b = np.where(a == 0, 0, b)
    return np.where(np.isfinite(a), b, 255).astype(np.uint8)


def quantize(x: np.ndarray, rule: int = FLOOR) -> tuple[np.ndarray, np.ndarray]:
    """Blocks along the last dimension (a multiple of 32): codes (one per element), bytes."""
    v = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(v), axis=-1)
    b = scale_bytes(amax, rule)
    bad = b == 255
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.ldexp(np.where(bad[..., None], 0.0, v), 127 - b.astype(np.int64)[..., None])
    # every quotient is a power-of-two multiple of an FP32 value: clipping to [-8, 8] and
    # rounding to FP32 keeps its side of every rounding border
    c = F.e2m1_encode(np.clip(y, -8, 8).astype(np.float32))
    c = np.where(bad[..., None], 0, c)
    return c.reshape(x.shape).astype(np.uint8), b


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """FP64 values of unpacked codes [.., K] and bytes [.., >= K/32]."""
    K = codes.shape[-1]
    b = scales[..., :K // BLOCK].astype(np.int64)
    v = F.e2m1_decode(codes).astype(np.float64).reshape(*codes.shape[:-1], -1, BLOCK)
    v = np.ldexp(v, b[..., None] - 127)
    v = np.where(b[..., None] == 255, np.nan, v)
    return v.reshape(codes.shape)


def rounded(x: np.ndarray, rule: int = FLOOR) -> np.ndarray:
    return values(*quantize(x, rule))


def padded_offsets(offsets: np.ndarray) -> np.ndarray:
    n = np.diff(offsets)
    return np.concatenate([[0], np.cumsum((n + SEGMENT - 1) // SEGMENT * SEGMENT)]).astype(np.int64)


def by_segment(x: np.ndarray, offsets: np.ndarray) -> np.ndarray:
    """Rows [offsets[s], offsets[s+1]) at their padded positions, zeros between, transposed:
    [cols, padded total]."""
    po = padded_offsets(offsets)
    out = np.zeros((po[-1], x.shape[1]), np.float64)
    for s in range(len(offsets) - 1):
        n = offsets[s + 1] - offsets[s]
        out[po[s]:po[s] + n] = x[offsets[s]:offsets[s + 1]]
    return out.T


def layer(x, ids, w, W13v, W2v, rule: int = FLOOR):
    """out [T, H] FP64 of the expert layer on x [T, H] with the weights' MXFP4 values W13v
    [E, 2I, H] and W2v [E, H, I], and per token and choice the FP64 SwiGLU row h, the sums of
    |products| of gate and up, and the gate and up values (for error bounds)."""
    T, k = ids.shape
    I = W2v.shape[2]
    xv = rounded(x, rule)
    h = np.zeros((T, k, I))
    gu, ab = np.zeros((T, k, 2 * I)), np.zeros((T, k, 2 * I))
    out = np.zeros((T, x.shape[1]))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            gu[t, j] = W13v[e] @ xv[t]
            ab[t, j] = np.abs(W13v[e]) @ np.abs(xv[t])
            h[t, j] = moe.swiglu(gu[t, j][None])[0]
            out[t] += w[t, j] * (W2v[e] @ rounded(h[t, j], rule))
    return out, h, gu, ab

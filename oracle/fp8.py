"""FP8 (E4M3) quantisation with an FP32 scale for each block of 128, written out step by step.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The element format is OCP OFP8's E4M3 (maximum 448).  A block is 128 consecutive elements of a row
(the last one may be shorter) or 128 x 128 elements of a matrix.  Readings taken, with A = max|v|:

    fp32    S = min(fp32(448 / A), 2^126)
    pow2    S = the largest power of two, at most 2^126, with A * S <= 448
    A = 0   S = 1

The stored scale is G = fp32(1 / S), an element's code E4M3(fp32(v * S)) to nearest even, its value
e4m3(code) * G.  A block with a NaN or infinity has the scale NaN and codes 0.
"""

from __future__ import annotations

import numpy as np

from . import formats as F

BLOCK = 128
FP32, POW2 = 0, 1
MOST = np.float32(2.0 ** 126)


def factors(amax: np.ndarray, rule: int = FP32) -> tuple[np.ndarray, np.ndarray]:
    """S and G (FP32) of blocks with these max|v| (FP32 values)."""
    a = np.asarray(amax, np.float32)
    ok = np.isfinite(a) & (a > 0)
    safe = np.where(ok, a, np.float32(1))
    if rule == POW2:
        m, e = np.frexp(safe.astype(np.float64))          # a = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
        S = np.ldexp(1.0, np.minimum(9 - e - (m > 0.875), 126)).astype(np.float32)
    else:
        with np.errstate(over="ignore"):
            S = np.minimum(F.f32_div(np.float32(448), safe), MOST)
    S = np.where(ok | ~np.isfinite(a), S, np.float32(1))
    G = F.f32_div(np.float32(1), S)
    return S, np.where(np.isfinite(a), G, np.float32(np.nan))


def encode(y: np.ndarray) -> np.ndarray:
    """FP32 values below 448 (1 + 2^-23) in magnitude -> E4M3 bytes, the sign kept."""
    y = np.asarray(y, np.float32)
    return (F.e4m3_encode(np.abs(y)) | (np.signbit(y).astype(np.uint8) << 7)).astype(np.uint8)


def _blocks(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.float32)
    pad = -x.shape[-1] % BLOCK
    x = np.concatenate([x, np.zeros((*x.shape[:-1], pad), np.float32)], -1) if pad else x
    return x.reshape(*x.shape[:-1], -1, BLOCK)


def quantize(x: np.ndarray, rule: int = FP32) -> tuple[np.ndarray, np.ndarray]:
    """Blocks along the last dimension: codes (one per element), scales FP32."""
    K = x.shape[-1]
    b = _blocks(x)
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(b), axis=-1)
    amax = np.where(np.isfinite(b).all(-1), amax, np.float32(np.inf))
    S, G = factors(amax, rule)
    bad = ~np.isfinite(amax)[..., None]
    y = F.f32_mul(np.where(bad, np.float32(0), b), S[..., None])
    codes = np.where(bad, np.uint8(0), encode(y)).astype(np.uint8)
    return codes.reshape(*x.shape[:-1], -1)[..., :K], G


def quantize_tiles(x: np.ndarray, rule: int = FP32) -> tuple[np.ndarray, np.ndarray]:
    """One matrix [m, K] in 128 x 128 blocks: codes [m, K], scales [ceil(m/128), ceil(K/128)]."""
    m, K = x.shape
    codes, G = np.zeros((m, K), np.uint8), np.zeros((-(-m // BLOCK), -(-K // BLOCK)), np.float32)
    for i in range(G.shape[0]):
        for j in range(G.shape[1]):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            b = np.asarray(x[at], np.float32)
            ok = np.isfinite(b).all()
            S, G[i, j] = factors(np.float32(np.max(np.abs(b)) if ok else np.inf), rule)
            if ok:
                codes[at] = encode(F.f32_mul(b, S))
    return codes, G


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """FP64 values of codes [.., K] under row blocks' scales [.., ceil(K/128)]."""
    return F.e4m3_decode(codes) * np.repeat(scales.astype(np.float64), BLOCK, -1)[..., :codes.shape[-1]]


def tile_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """FP64 values of one matrix's codes under its blocks' scales."""
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0), BLOCK, 1)
    return F.e4m3_decode(codes) * s[:codes.shape[0], :codes.shape[1]]

"""The SwiGLU of the MXFP4 kernels over its whole range of gates, from sums that are exact."""

import numpy as np
import pytest
import torch

import synth
from oracle import moe
from tests.gpu_util import dev_bf16, host, same_bits
from tests.test_gpu_mx import check_codes

pytestmark = pytest.mark.gpu

H = I = 256


def gates_and_ups(rows):
    """x [rows, H] and W13 [2I, H] whose products are exact (three elements of a block each, all of them
    codes under the block's scale), gates from -288 to 288 and down to 2^-5, mostly negative."""
    r = synth.rng(rows)
    x = np.zeros((rows, H))
    x[:, :3] = np.array([1.0, 2.0, 0.5])[np.arange(rows) % 3][:, None]
    W = np.zeros((2 * I, H))
    g = np.stack([r.choice([4.0, 6.0], I), r.choice([0.5, 1, 1.5, 2, 3, 4, 6], I), r.choice([0, 0.5, 1, 3, 6], I)], 1)
    W[:I, :3] = g * np.exp2(r.integers(-7, 4, I))[:, None] * np.where(r.random(I) < 0.8, -1, 1)[:, None]
    W[I:, 0] = r.choice([4.0, 6.0, -4.0, -6.0], I) * np.exp2(r.integers(-4, 3, I))
    p = x @ W.T
    return x, W, p[:, :I], p[:, I:]


def test_error_grows_with_the_gate(gpu_lib):
    """g / (1 + exp(-g)) u as the kernels compute it: -g log2(e) in FP32 (the constant within 0.224
    2^-24, one rounding: 1.224 2^-24 |g| of the exponential's value), exp2 and reciprocal within one
    unit in the last place (2 2^-24 each), the sum and two products with one rounding each: in all
    (1.224 |g| + 7) 2^-24 of the result, and 1.25 and 8 with the products of these.  A reciprocal
    below FP32's smallest normal 2^-126 may be zero, and is where the exponential overflows."""
    rows = 6
    x, W, g, u = gates_and_ups(rows)
    assert g.min() < -100 and (np.abs(g) < 0.1).any() and ((g > -87) & (g < -60)).sum() > 5 and g.max() > 50
    xq, wq = gpu_lib.mxfp4_quantize(dev_bf16(x)), gpu_lib.mxfp4_quantize(dev_bf16(W))
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    exact = host(gpu_lib.mxfp4_grouped_gemm(xq, wq, off, 1, 2 * I))
    assert np.array_equal(exact, np.concatenate([g, u], 1))
    h = host(gpu_lib.mxfp4_grouped_gemm(xq, wq, off, 1, I, epilogue=gpu_lib.NV4_EPI_SWIGLU)).astype(np.float64)
    ref = moe.swiglu(np.concatenate([g, u], 1))
    tol = np.abs(ref) * (1.25 * np.abs(g) + 8) * 2.0 ** -24 + np.abs(g * u) * 2.0 ** -126
    assert (np.abs(h - ref) <= tol).all(), float(np.max(np.abs(h - ref) / (tol + 1e-300)))


@pytest.mark.parametrize("T", [2, 3, 7])   # each of the three ways through the few-token layer
def test_few_takes_the_same_values(gpu_lib, T):
    """With W2 the identity and one expert the layer returns the re-quantised SwiGLU rows: those of the
    grouped product, bit for bit, since the sums are exact."""
    x, W, *_ = gates_and_ups(T)
    w = gpu_lib.mx_quantize_expert_weights(dev_bf16(W[None]), dev_bf16(np.eye(H, I)[None]))
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    q = gpu_lib.MXFP4.empty(T, I)
    C = gpu_lib.mxfp4_grouped_gemm(gpu_lib.mxfp4_quantize(dev_bf16(x)), w.w13, off, 1, I, q_out=q,
                                   epilogue=gpu_lib.NV4_EPI_SWIGLU)
    check_codes(q, host(C))
    out = gpu_lib.mx_moe_few(dev_bf16(x), torch.zeros(T, 1, device="cuda"), w, 1, out_dtype=torch.float32)
    assert same_bits(out + 0.0, gpu_lib.mxfp4_dequantize(q, torch.float32) + 0.0)   # (-0 as 0)

"""MXFP4 at the ends of its range: every scale byte dequantised, products under scales whose product
is a subnormal or overflows, and the few-token layer between very small activations and very large weights."""

import numpy as np
import pytest
import torch

import synth
from oracle import mxfp4 as M
from oracle import nvfp4 as Q
from tests.gpu_util import dev_bf16, dev_f32, dev_i32, host
from tests.test_gpu_mx import check_codes, few_reference, unpacked, vals

pytestmark = pytest.mark.gpu


def tensor(gpu_lib, codes, scales):
    """An MXFP4 tensor of packed codes [rows, K/2] and scale bytes [rows, K/32]."""
    rows, K = codes.shape[0], 2 * codes.shape[1]
    s = np.zeros((rows, gpu_lib.mxfp4_scale_stride(K)), np.uint8)
    s[:, :K // 32] = scales
    return gpu_lib.MXFP4(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda(), rows, K)


def test_every_scale_byte_dequantised(gpu_lib):
    """Values under 2^-127 are subnormals of either type; those of 2^128 and more are infinity."""
    codes = synth.rng(1).integers(0, 256, (256, 48), dtype=np.uint8)
    scales = np.stack([np.arange(256), np.arange(256)[::-1], (np.arange(256) * 7) % 256], 1).astype(np.uint8)
    with np.errstate(over="ignore"):
        want = M.values(Q.unpack_codes(codes), scales).astype(np.float32)
    assert np.isinf(want).any() and (np.abs(want[want != 0]) < 2.0 ** -126).any()
    for dt in (torch.float32, torch.bfloat16):
        assert np.array_equal(host(gpu_lib.mxfp4_dequantize(tensor(gpu_lib, codes, scales), dt)), want, equal_nan=True)


def test_products_under_every_pair_of_scales(gpu_lib):
    """3 * 3 + 1 * 1 under 2^(ea + eb): exact wherever FP32 holds it, infinity above."""
    by = np.array([0, 1, 2, 3, 20, 64, 100, 120, 126, 127, 128, 140, 200, 230, 250, 252, 253, 254], np.uint8)
    codes = np.zeros((len(by), 16), np.uint8)
    codes[:, 0], codes[:, 3] = 0x05, 0x20
    q = tensor(gpu_lib, codes, by[:, None])
    C = gpu_lib.mxfp4_grouped_gemm(q, q, dev_i32(np.array([0, len(by)])), 1, len(by))
    with np.errstate(over="ignore"):
        e = by.astype(int) - 127
        want = np.ldexp(10.0, e[:, None] + e[None, :]).astype(np.float32)
    assert np.array_equal(host(C), want)


def test_largest_blocks_by_the_ceil_rule(gpu_lib):
    """From 1.75 * 2^127 on the nearest code under 2^126 is 4: the stored value is 2^128."""
    x = np.zeros((3, 32), np.float32)
    x[:, 0] = [1.7 * 2.0 ** 127, 1.75 * 2.0 ** 127, -3.4e38]
    q = gpu_lib.mxfp4_quantize(dev_f32(x), rule=M.CEIL)
    check_codes(q, x, M.CEIL)
    assert unpacked(q)[1][:, 0].tolist() == [253] * 3
    assert host(gpu_lib.mxfp4_dequantize(q, torch.float32))[:, 0].tolist() == [3 * 2.0 ** 126, np.inf, -np.inf]


@pytest.mark.parametrize("T,E,k", [(2, 6, 2), (9, 40, 3), (30, 4, 2)])   # each of the three ways through it
def test_few_between_small_and_large(gpu_lib, T, E, k):
    H, I, s = 160, 64, 2.0 ** 110
    x = (synth.activations(T, H, 1) / s).astype(np.float32)
    W13, W2 = synth.weights((E, 2 * I, H), 2) * s, synth.weights((E, H, I), 3)
    w = gpu_lib.mx_quantize_expert_weights(dev_bf16(W13), dev_bf16(W2))
    ids, wts = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    out = gpu_lib.mx_moe_few(dev_bf16(x), dev_f32(synth.logits_softmax(T, E, 4)), w, k, topk_ids=ids, topk_w=wts,
                             out_dtype=torch.float32)
    ref, tol = few_reference(x, host(ids), host(wts).astype(np.float64), vals(w.w13).reshape(E, 2 * I, H),
                             vals(w.w2).reshape(E, H, I))
    assert np.abs(ref).max() > 1e-4 and (np.abs(host(out) - ref) <= tol).all()

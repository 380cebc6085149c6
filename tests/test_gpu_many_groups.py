"""Calls of more work than one dimension of a launch counts (2^32 work-items): the FP8 conversions and the router's
gradients at sizes that their contracts allow."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev_f32, dev_i32, same_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    """Up to 150 GB a test, given back behind it."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("yt", [F32, BF16])
def test_combine_backward(gpu_lib, yt):
    """One workgroup a token: 2^24 tokens are 2^32 work-items of 256."""
    T, H = (1 << 24) + 5, 8
    dout, Y = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda").to(yt)
    row = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, 1)
    w = torch.rand(T, 1, device="cuda")
    dY, dw = gpu_lib.moe_combine_backward(dout, Y, row, w)
    assert torch.equal(dY.flip(0), (w * dout).to(yt))
    y = Y.flip(0).float()
    assert ((dw[:, 0].double() - (dout.double() * y).sum(1)).abs() <= H * 2.0 ** -24 * (dout * y).abs().sum(1)).all()


def test_balance_backward(gpu_lib):
    """Eight work-items a token where experts are few: 2^29 tokens."""
    T = (1 << 29) + 7
    l, ids = torch.rand(T, 1, device="cuda"), torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    b = gpu_lib.moe_balance_loss(l, ids)
    assert b.tokens.item() == b.counts.item() == T
    g = gpu_lib.moe_balance_backward(l, ids, b, dev_f32(np.array([1.0, float(T)])))
    # one expert: p = 1, lse = l and c_j - sum c p = 0; 2 T / T lse within the coefficient's three roundings and the product's
    # (T is rounded to 2^29, which is 2^-26 off)
    assert ((g - 2 * l).abs() <= 6 * 2.0 ** -24 * 2 * l).all()


def test_rows(gpu_lib):
    """64 blocks a workgroup of 256: 2^30 blocks, quantised and back."""
    R, K = (1 << 30) + 77, 16
    x = torch.randn(3, K, device="cuda", dtype=BF16)
    index = torch.zeros(R, dtype=torch.int32, device="cuda")
    index[-70:], index[-1] = 1, 2
    q, t = gpu_lib.fp8_quantize(x, row_index=index), gpu_lib.fp8_quantize(x)
    del index
    at = torch.cat([torch.arange(0, R, 4093), torch.arange(R - 300, R)]).cuda()
    src = (at >= R - 70).long() + (at == R - 1).long()
    assert torch.equal(q.codes[at], t.codes[src]) and torch.equal(q.scales[at], t.scales[src])
    d = gpu_lib.fp8_dequantize(q)
    assert torch.equal(d[at], gpu_lib.fp8_dequantize(t)[src])


@pytest.mark.parametrize("dt,K", [(BF16, 2064), (F32, 1040)])
def test_tiles(gpu_lib, dt, K):
    """A workgroup of 256 (FP32: 512) for each block: 2^20 matrices of one row."""
    E = 1 << 20
    x = torch.randn(E, K, device="cuda", dtype=BF16).to(dt)
    assert E * -(-K // 128) * (256 if dt == BF16 else 512) > 1 << 32
    q = gpu_lib.fp8_quantize(x, layout=gpu_lib.NV4_F8_TILES, nseg=E)
    r = gpu_lib.fp8_quantize(x)                     # blocks of one row are the row's own
    assert torch.equal(q.codes, r.codes) and torch.equal(q.scales[:, 0], r.scales)


def test_transpose(gpu_lib):
    E, m, K = (1 << 24) + 3, 16, 16
    g = torch.Generator("cuda").manual_seed(1)
    q = gpu_lib.FP8.empty(E * m, K, E)
    q.codes.random_(0, 127, generator=g)
    q.scales.uniform_(generator=g)
    t = gpu_lib.fp8_transpose(q)
    assert torch.equal(t.codes.view(E, K, m), q.codes.view(E, m, K).transpose(1, 2))
    assert torch.equal(t.scales.flatten(), q.scales.flatten())


@pytest.mark.parametrize("both", [False, True])
def test_segments(gpu_lib, both):
    """2^20 segments of FP32 rows, all of them empty but the last: as that one alone."""
    E, K, R = 1 << 20, 1040, 300
    x = torch.randn(R, K, device="cuda")
    n = 384
    off, padded = (torch.zeros(E + 1, dtype=torch.int32, device="cuda") for _ in range(2))
    off[-1], padded[-1] = R, n
    run = lambda o, p, s: gpu_lib.fp8_quantize(x, layout=gpu_lib.NV4_ROWS_AND_COLS if both else gpu_lib.NV4_COLS, nseg=s,
                                               seg_offsets=o, seg_padded_offsets=p)
    ref, got = run(dev_i32(np.array([0, R])), dev_i32(np.array([0, n])), 1), run(off, padded, E)
    assert (-(-R // 128) + E) * -(-K // 128) * 512 > 1 << 32
    assert torch.equal(got.codes[:, :n], ref.codes[:, :n]) and torch.equal(got.scales[:, :3], ref.scales[:, :3])
    if both:
        assert same_bits(got.rows_out.codes, ref.rows_out.codes) and same_bits(got.rows_out.scales, ref.rows_out.scales)

"""Calls of more work than one dimension of a launch counts (2^32 work-items): the combine, the routing and the MXFP4
conversions at sizes that their contracts allow."""

import numpy as np
import pytest
import torch

from tests.gpu_util import dev_i32
from tests.test_gpu_many_groups import BF16, F32, memory  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("yt,k", [(F32, 1), (BF16, 1), (F32, 3)])
def test_combine(gpu_lib, yt, k):
    T, H = (1 << 24) + 5, 8
    Y = torch.randn(T, H, device="cuda").to(yt)
    row = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    row = row.view(T, 1).repeat(1, k)
    w = torch.zeros(T, k, device="cuda")
    w[:, k - 1] = torch.rand(T, device="cuda")
    assert torch.equal(gpu_lib.moe_combine(Y, row, w), w[:, k - 1:] * Y.flip(0).float())


@pytest.mark.parametrize("E,lanes", [(2, 32), (129, 64)])
def test_route(gpu_lib, E, lanes):
    """A wave of 64 for one token, or for two up to 128 experts."""
    T = (1 << 32) // lanes + 9
    l = torch.empty(T, E, device="cuda").uniform_()
    rt = gpu_lib.moe_permute(l, E, 1)
    want = torch.cat([l[i:i + (1 << 24)].argmax(1) for i in range(0, T, 1 << 24)])
    top = torch.cat([l[i:i + (1 << 24)].amax(1) for i in range(0, T, 1 << 24)])
    # (of equal logits the first expert; argmax may give another)
    ids = rt.topk_ids[:, 0].long()
    assert torch.equal(l.gather(1, ids[:, None])[:, 0], top) and (ids == want).float().mean() > 0.999
    assert torch.equal(rt.offsets[1:].long(), torch.bincount(ids, minlength=E).cumsum(0))
    assert torch.equal(rt.row_token[rt.token_row[:, 0].long()], torch.arange(T, dtype=torch.int32, device="cuda"))


def test_gather(gpu_lib):
    """Four rows a workgroup of 256."""
    T, K = (1 << 26) + 5, 32
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    ids[::2] = 1
    src, dst = gpu_lib.NVFP4.empty(T, K, 1), gpu_lib.NVFP4.empty(T, K, 1)
    src.codes.random_(0, 256)
    src.scales.random_(0, 127)
    rt = gpu_lib.moe_permute(None, 2, 1, topk_ids=ids, gather_src=src, gather_dst=dst)
    # (in parts: torch's own gather of so many rows is cut off as well)
    for t, c, z in zip(rt.row_token.long().split(1 << 22), dst.codes.split(1 << 22), dst.scales.split(1 << 22)):
        assert torch.equal(c, src.codes[t]) and torch.equal(z, src.scales[t])


def test_mx_rows(gpu_lib):
    R, K = (1 << 29) + 77, 32
    x = torch.randn(3, K, device="cuda", dtype=BF16)
    index = torch.zeros(R, dtype=torch.int32, device="cuda")
    index[-70:], index[-1] = 1, 2
    q, t = gpu_lib.mxfp4_quantize(x, row_index=index), gpu_lib.mxfp4_quantize(x)
    at = torch.cat([torch.arange(0, R, 4093), torch.arange(R - 300, R)]).cuda()
    src = index[at].long()
    assert torch.equal(q.codes[at], t.codes[src]) and torch.equal(q.scales[at], t.scales[src])
    d = gpu_lib.mxfp4_dequantize(q)
    assert torch.equal(d[at], gpu_lib.mxfp4_dequantize(t)[src])


@pytest.mark.parametrize("both", [False, True])
def test_mx_segments(gpu_lib, both):
    """2^20 segments of FP32 rows, all of them empty but the last: as that one alone."""
    E, K, R, n = 1 << 20, 1152, 300, 384
    x = torch.randn(R, K, device="cuda")
    off, padded = (torch.zeros(E + 1, dtype=torch.int32, device="cuda") for _ in range(2))
    off[-1], padded[-1] = R, n
    run = lambda o, p, s: gpu_lib.mxfp4_quantize(x, layout=gpu_lib.NV4_ROWS_AND_COLS if both else gpu_lib.NV4_COLS, nseg=s,
                                                 seg_offsets=o, seg_padded_offsets=p)
    ref, got = run(dev_i32(np.array([0, R])), dev_i32(np.array([0, n])), 1), run(off, padded, E)
    assert (R + 127 * E) // 128 * (K // 64) * 256 > 1 << 32
    assert torch.equal(got.codes[:, :n // 2], ref.codes[:, :n // 2])
    assert torch.equal(got.scales[:, :n // 32], ref.scales[:, :n // 32])
    if both:
        assert torch.equal(got.rows_out.codes, ref.rows_out.codes) and torch.equal(got.rows_out.scales, ref.rows_out.scales)

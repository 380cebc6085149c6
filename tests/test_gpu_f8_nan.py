"""Blocks with NaN scales in the FP8 product: NaN in exactly the results that such a block belongs to, in every kernel
and by every way that scales take (multiply-adds, a scale for each weight row, the matrix instruction's exponents), and
through the re-quantisation.  (Elsewhere integers under power-of-two scales: every order of adding gives the same bits.)"""

import numpy as np
import pytest
import torch

from oracle import fp8 as M
from tests.gpu_util import dev_i32, same_bits
from tests.test_gpu_f8_tiles import BF16, COLUMNS, F32, KINDS, coded, counts_of, reference, values

pytestmark = pytest.mark.gpu


def spoil_rows(q, at):
    """Non-finite blocks as the quantiser leaves them: scale NaN, codes 0."""
    for row, block in at:
        q.scales[row, block] = float("nan")
        q.codes[row, block * 128:(block + 1) * 128] = 0


def spoil_tiles(q, at):
    m = q.rows // q.nseg
    for e, rb, block in at:
        q.scales[e, rb, block] = float("nan")
        q.codes[e * m + rb * 128:e * m + min(rb * 128 + 128, m), block * 128:(block + 1) * 128] = 0


def agrees(got, ref):
    """Equal bits, and NaN exactly where the reference is."""
    return torch.equal(got.isnan(), ref.isnan()) and same_bits(got.nan_to_num(nan=0.0), ref.nan_to_num(nan=0.0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [272, 896])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_rows(gpu_lib, kind, K, rule, dt):
    counts, N = counts_of(kind), COLUMNS[kind]
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R, last = int(off[-1]), (K - 1) // 128
    a, b = coded(gpu_lib, R, K, 0, 1, rule), coded(gpu_lib, E * N, K, E, 2, rule)
    spoil_rows(a, [(0, 0), (R - 1, last), (R // 2, 1)])
    full = int(np.argmax(counts))
    clean = reference(a, b, off, E, N).to(dt)
    assert 0 < clean.isnan().any(1).sum() <= 3 and clean.isnan().any(1).sum() * N == clean.isnan().sum()
    run = lambda **o: gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, M_cap=R, out_dtype=dt, **o)
    assert agrees(run(), clean)
    spoil_tiles(b, [(full, 0, last), (E - 1, (N - 1) // 128, 0)])
    ref = reference(a, b, off, E, N).to(dt)
    assert agrees(run(), ref) and (R == 3 or (~ref.isnan()).any())       # (three rows: all of them are spoiled)
    index = torch.randint(0, R, (R,), device="cuda", dtype=torch.int32)
    assert agrees(run(a_rows=index), reference(a, b, off, E, N, index).to(dt))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_swiglu_and_its_quantisation(gpu_lib, kind, rule):
    counts, N, K = counts_of(kind), (COLUMNS[kind] // 64 + 1) * 32, 400
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R, full = int(off[-1]), int(np.argmax(counts))
    a, b = coded(gpu_lib, R, K, 0, 1, rule), coded(gpu_lib, E * 2 * N, K, E, 2, rule)
    a.scales.mul_(2.0 ** -6)
    spoil_rows(a, [(0, 0), (R - 1, 3), (R // 2, 1)])
    spoil_tiles(b, [(full, 0, 2), (E - 1, (2 * N - 1) // 128, 0)])      # a block of gate rows, one of up rows
    raw = reference(a, b, off, E, 2 * N)
    nan = (raw[:, :N] + raw[:, N:]).isnan()
    o = dict(M_cap=R, epilogue=gpu_lib.NV4_EPI_SWIGLU)
    C = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, **o)
    assert torch.equal(C.isnan(), nan) and (R == 3 or (~nan).any()) and nan.any()
    want = gpu_lib.fp8_quantize(C, rule=rule)
    blocks = torch.nn.functional.pad(nan, (0, -N % 128)).view(R, -1, 128).any(2)
    assert torch.equal(want.scales.isnan(), blocks)
    for dt in (F32, BF16, None):
        q = gpu_lib.FP8.empty(R, N)
        got = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, q_out=q, rule=rule, want_c=dt is not None,
                                       out_dtype=dt or F32, **o)
        assert got is None if dt is None else agrees(got, C.to(dt))
        assert agrees(q.scales, want.scales) and same_bits(q.codes, want.codes)
        assert (q.codes[blocks.repeat_interleave(128, 1)[:, :N]] == 0).all()
    assert agrees(gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, out_dtype=BF16, **o), C.bfloat16())


@pytest.mark.parametrize("blocks", [[1], [3, 0, 1, 0, 7], [2] * 40])
@pytest.mark.parametrize("n,m", [(16, 16), (300, 130)])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_weight_gradients(gpu_lib, blocks, n, m, rule, dt):
    """In one block of a live range: that expert's row or column, and no other expert's."""
    E, off = len(blocks), 128 * np.concatenate([[0], np.cumsum(blocks)])
    a, b = coded(gpu_lib, n, int(off[-1]), 0, 1, rule), coded(gpu_lib, m, int(off[-1]), 0, 2, rule)
    spoil_rows(a, [(n - 1, int(off[-1]) // 128 - 1)])
    spoil_rows(b, [(5, 0)])
    av, bv = values(a), values(b)
    ref = torch.stack([av[:, off[e]:off[e + 1]] @ bv[:, off[e]:off[e + 1]].T for e in range(E)]).to(dt)
    assert ref[-1, n - 1].isnan().all() and ref[0, :, 5].isnan().all()
    got = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, 0, group_mode=gpu_lib.NV4_GROUP_K, out_dtype=dt)
    assert agrees(got, ref)

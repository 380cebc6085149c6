"""The FP8 product's kernels and tiles, each at problems large or small enough that it is the one taken.

The operands are integers under scales that are powers of two, so that every way of adding gives the same FP32
sums, exactly: a product is compared bit for bit, whichever kernel it comes from."""

import numpy as np
import pytest
import torch

import synth
from oracle import fp8 as M
from oracle import moe
from tests.gpu_util import dev_i32, host, same_bits

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def coded(lib, rows, K, nseg, seed, rule):
    """Codes of integers up to 8, scales 1/2, 1 and 2: sums of less than 2^16 products stay below 2^24 quarters."""
    g = torch.Generator("cuda").manual_seed(seed)
    v = torch.randint(-8, 9, (rows, K), device="cuda", generator=g).float()
    q = lib.FP8.empty(rows, K, nseg)
    q.codes.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    q.scales.copy_(torch.randint(-1, 2, q.scales.shape, device="cuda", generator=g).float().exp2())
    q.rule = rule
    return q


def values(q):
    """FP32 values of rows or of tiles (exact)."""
    v = q.codes.view(torch.float8_e4m3fn).float()
    s = q.scales.view(q.rows if q.nseg == 0 else -1, (q.K + 127) // 128)
    if q.nseg:
        s = q.scales.view(q.nseg, -1, (q.K + 127) // 128).repeat_interleave(128, 1)[:, :q.rows // q.nseg]
        s = s.reshape(q.rows, -1)
    return v * s.repeat_interleave(128, 1)[:, :q.K]


def reference(a, b, off, E, n, index=None):
    """FP32 sums by expert: exact, as every sum of these integers is."""
    av, bv = values(a), values(b).view(E, n, -1)
    av = av if index is None else av[index.long()]
    return torch.cat([av[off[e]:off[e + 1]] @ bv[e].T for e in range(E)])


def counts_of(kind):
    r = synth.rng(5)
    return {"few": [5, 0, 33], "few rows of many": [0, 1] * 3 + [0],
            "small": list(r.integers(0, 40, 64)), "small, one hot": [0, 1500] + [3] * 62,
            "medium": [700, 0, 1301], "large": [3000, 129, 5171]}[kind]


# columns that make each kernel the one taken; with SwiGLU half of them
COLUMNS = {"few": 72, "few rows of many": 33, "small": 290, "small, one hot": 290, "medium": 300, "large": 1500}
KINDS = list(COLUMNS)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [112, 272, 896])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_rows(gpu_lib, kind, K, rule, dt):
    counts, N = counts_of(kind), COLUMNS[kind]
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    a, b = coded(gpu_lib, R, K, 0, 1, rule), coded(gpu_lib, E * N, K, E, 2, rule)
    ref = reference(a, b, off, E, N).to(dt)
    C = torch.full((R + 2, N), 3.0, dtype=dt, device="cuda")
    gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, M_cap=R, C=C)
    assert same_bits(C[:R].contiguous(), ref) and (C[R:] == 3).all()
    # gathered rows, the rows of C an odd number of elements apart, not all of them asked for
    index = torch.randint(0, R, (R,), device="cuda", dtype=torch.int32)
    ref = reference(a, b, off, E, N, index).to(dt)
    big = torch.full(((R + 2) * (N + 3) + 1,), 3.0, dtype=dt, device="cuda")
    C = big[1:].view(R + 2, N + 3)[:, :N]
    gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, M_cap=R - 1, a_rows=index, C=C)
    assert same_bits(C[:R - 1].contiguous(), ref[:R - 1].contiguous())
    C[:R - 1] = 3
    assert (big == 3).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [112, 528])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_swiglu_and_its_quantisation(gpu_lib, kind, K, rule):
    """FP32, BF16 and quantised results of the same exact sums, with and without one another."""
    counts, N = counts_of(kind), (COLUMNS[kind] // 64 + 1) * 32
    E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    R = int(off[-1])
    a, b = coded(gpu_lib, R, K, 0, 1, rule), coded(gpu_lib, E * 2 * N, K, E, 2, rule)
    a.scales.mul_(2.0 ** -6)        # (gates small enough for exp to matter)
    a = gpu_lib.FP8(a.codes, a.scales, R, K, rule=rule)
    o = dict(M_cap=R, epilogue=gpu_lib.NV4_EPI_SWIGLU)
    raw = reference(a, b, off, E, 2 * N).double()
    g, u = raw[:, :N], raw[:, N:]
    ref = g / (1 + torch.exp(-g)) * u
    C = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, **o)
    # (gates whose exp leaves FP32's range give 0)
    assert ((C - ref).abs() <= ref.abs() * (1.25 * g.abs() + 8) * 2.0 ** -24 + (g * u).abs() * 2.0 ** -125).all()
    for dt in (F32, BF16, None):
        q = gpu_lib.FP8.empty(R + 1, N)
        q.codes.fill_(0xEE)
        q.scales.fill_(7.0)
        part = gpu_lib.FP8(q.codes[:R], q.scales[:R], R, N)
        got = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, q_out=part, rule=rule, want_c=dt is not None,
                                       out_dtype=dt or F32, **o)
        assert got is None if dt is None else same_bits(got, C.to(dt))
        want = gpu_lib.fp8_quantize(C, rule=rule)
        assert same_bits(part.codes, want.codes) and same_bits(part.scales, want.scales)
        assert (q.codes[R] == 0xEE).all() and (q.scales[R] == 7).all()
    assert same_bits(gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, out_dtype=BF16, **o), C.bfloat16())


@pytest.mark.parametrize("blocks", [[1], [3, 0, 1, 0, 7], [2] * 40, [0, 0], [5, 1, 60]])
@pytest.mark.parametrize("n,m", [(16, 16), (300, 130), (768, 521)])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_weight_gradients(gpu_lib, blocks, n, m, rule):
    E, off = len(blocks), 128 * np.concatenate([[0], np.cumsum(blocks)])
    K = max(int(off[-1]), 128)
    a, b = coded(gpu_lib, n, K, 0, 1, rule), coded(gpu_lib, m, K, 0, 2, rule)
    av, bv = values(a), values(b)
    ref = torch.stack([av[:, off[e]:off[e + 1]] @ bv[:, off[e]:off[e + 1]].T for e in range(E)])
    for dt in (F32, BF16):
        C = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, 0, group_mode=gpu_lib.NV4_GROUP_K, out_dtype=dt)
        assert same_bits(C, ref.to(dt))


@pytest.mark.parametrize("hot", [0, 63])
def test_every_row_in_one_expert(gpu_lib, hot):
    """As many experts as make the mean few rows, and all of them in one: each kernel's tiles behind the first."""
    for R, N in ((40, 1100), (3000, 300), (60, 33)):
        E, K = 64, 400
        off = np.where(np.arange(E + 1) > hot, R, 0)
        a, b = coded(gpu_lib, R, K, 0, 1, M.FP32), coded(gpu_lib, E * N, K, E, 2, M.FP32)
        got = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N)
        assert same_bits(got, reference(a, b, off, E, N))


def test_many_experts(gpu_lib):
    """1024 experts: more than one border for each lane and thread that looks for a tile."""
    r = synth.rng(3)
    for R, N, K in ((1, 16, 128), (30, 16, 160), (5000, 40, 272)):
        E = 1024
        off = np.concatenate([[0], np.cumsum(r.multinomial(R, r.dirichlet(np.full(E, 0.3))))])
        a, b = coded(gpu_lib, R, K, 0, 1, M.FP32), coded(gpu_lib, E * N, K, E, 2, M.FP32)
        assert same_bits(gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N), reference(a, b, off, E, N))


def test_offsets_outside_the_contract_stay_in_bounds(gpu_lib):
    """Offsets that fall, are negative or lie behind M_cap: taken as empty or cut off, nothing behind C."""
    E, K, N, R = 4, 160, 40, 50
    a, b = coded(gpu_lib, R, K, 0, 1, M.FP32), coded(gpu_lib, E * N, K, E, 2, M.FP32)
    for off in ([0, 20, 10, 40, 50], [-5, 10, 20, 30, 90], [7, 7, 7, 7, 7], [60, 70, 80, 90, 100], [0, -3, 0, 50, 10]):
        big = torch.full((R + 64, N), 3.0, device="cuda")
        gpu_lib.fp8_grouped_gemm(a, b, dev_i32(np.array(off)), E, N, M_cap=R, C=big[:R])
        assert (big[R:] == 3).all()


def test_a_chain_of_stages_in_the_last_block(gpu_lib):
    """K of one block, of one element group behind a block, and as many stages as the ring has slots."""
    for K in (16, 128, 144, 256, 384, 400):
        for counts, N in (([300, 1, 700, 2, 900], 300), ([7] * 64, 300), ([3000, 5300], 1536)):
            E, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
            a, b = coded(gpu_lib, int(off[-1]), K, 0, 1, M.FP32), coded(gpu_lib, E * N, K, E, 2, M.FP32)
            index = torch.randint(0, int(off[-1]), (int(off[-1]),), device="cuda", dtype=torch.int32)
            got = gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, M_cap=int(off[-1]), a_rows=index, out_dtype=BF16)
            assert same_bits(got, reference(a, b, off, E, N, index).bfloat16())

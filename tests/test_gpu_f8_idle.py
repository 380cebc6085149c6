"""The FP8 product where workgroups have no tile, or fewer stages than their ring has slots: their loads have nothing
to fetch, whatever K is.  (Integers under power-of-two scales: every order of adding gives the same bits.)"""

import numpy as np
import pytest
import torch

from oracle import fp8 as M
from tests.gpu_util import dev_i32, same_bits
from tests.test_gpu_f8_tiles import coded, reference, values

pytestmark = pytest.mark.gpu


# experts, rows that C has room for, columns: the kernel for few rows, and tiles of 64, 128 and 256 rows
@pytest.mark.parametrize("E,R,N", [(4, 40, 64), (64, 2000, 320), (2, 900, 320), (2, 9000, 1536)])
@pytest.mark.parametrize("K", [16, 144, 4112])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_rows(gpu_lib, E, R, N, K, rule):
    a = coded(gpu_lib, R, K, 0, 1, rule)
    for epi in (gpu_lib.NV4_EPI_NONE, gpu_lib.NV4_EPI_SWIGLU):
        b = coded(gpu_lib, E * N * (2 if epi else 1), K, E, 2, rule)
        for dt in (torch.float32, torch.bfloat16):
            for gather in (None, torch.arange(R - 1, -1, -1, device="cuda", dtype=torch.int32)):
                for used in (0, 1, 70 if R > 100 else 20):
                    off = np.array([0] + [used] * E)
                    C = torch.full((R, N), 3.0, dtype=dt, device="cuda")
                    gpu_lib.fp8_grouped_gemm(a, b, dev_i32(off), E, N, M_cap=R, a_rows=gather, epilogue=epi, C=C)
                    assert (C[used:] == 3).all()
                    if epi == gpu_lib.NV4_EPI_NONE:
                        ref = reference(a, b, off, E, N, gather)
                        assert same_bits(C[:used].contiguous(), ref.to(dt))


@pytest.mark.parametrize("E,n,m", [(1, 16, 16), (3, 300, 130), (40, 768, 520)])
@pytest.mark.parametrize("rule", [M.FP32, M.POW2])
def test_weight_gradients(gpu_lib, E, n, m, rule):
    """No range at all, and one block in the last expert."""
    K = 128 * 33
    a, b = coded(gpu_lib, n, K, 0, 1, rule), coded(gpu_lib, m, K, 0, 2, rule)
    av, bv = values(a), values(b)
    for lo, hi in ((0, 0), (K, K), (K - 128, K)):
        off = dev_i32(np.array([lo] * E + [hi]))
        for dt in (torch.float32, torch.bfloat16):
            C = gpu_lib.fp8_grouped_gemm(a, b, off, E, 0, group_mode=gpu_lib.NV4_GROUP_K, out_dtype=dt)
            assert (C[:-1] == 0).all() and same_bits(C[-1], (av[:, lo:hi] @ bv[:, lo:hi].T).to(dt))

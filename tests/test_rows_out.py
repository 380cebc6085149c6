"""A tensor that is quantised into again keeps no row-direction output of an earlier call."""

import pytest

import nvfp4_w4a4_moe_amd as nv4
from tests.test_f8_binding import gpu  # noqa: F401 (the stand-in library)
from tests.test_mx_binding import i32, ten


@pytest.mark.parametrize("quantize", ["fp8_quantize", "mxfp4_quantize"])
def test_the_row_output_is_the_last_calls(gpu, quantize):  # noqa: F811
    q, x = getattr(nv4, quantize), ten(9, 128)
    seg = dict(nseg=2, seg_offsets=i32(0, 5, 9), seg_padded_offsets=i32(0, 128, 256))
    both = q(x, layout=nv4.NV4_ROWS_AND_COLS, **seg)
    old = both.rows_out
    assert old.rows == 9
    assert q(x, layout=nv4.NV4_ROWS_AND_COLS, out=both, **seg).rows_out is not old
    assert q(x, layout=nv4.NV4_COLS, out=both, **seg) is both and both.rows_out is None


def test_other_calls_into_the_same_tensor(gpu):  # noqa: F811
    from tests.test_f8_binding import f8
    stale = f8(9, 32)
    a, b, off = f8(9, 128), f8(64, 128, 1), i32(0, 9)
    out = f8(9, 32)
    out.rows_out = stale
    nv4.fp8_grouped_gemm(a, b, off, 1, 32, epilogue=nv4.NV4_EPI_SWIGLU, q_out=out, want_c=False)
    assert out.rows_out is None
    t = f8(128, 64, 1)
    t.rows_out = stale
    assert nv4.fp8_transpose(b, out=t) is t and t.rows_out is None

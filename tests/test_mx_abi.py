"""The MXFP4 calls without a GPU: every declared function is exported and bound, and each
documented refusal happens on the host, before anything is launched."""

import ctypes
import os
import re

import pytest
import torch

import nvfp4_w4a4_moe_amd as nv4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nv4moe", "mxfp4.h")
P = ctypes.c_void_p(0x1000)
EINVAL, EALIGN, EUNSUPPORTED, EWORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv4.LIB_PATH):
        pytest.fail("libnv4moe.so is not built")
    return nv4.load()


def mx(rows, K, codes=0x1000, scales=0x1000):
    return nv4.MXTensor(codes, scales, rows, K)


def test_declared_functions_are_exported_and_bound(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", src, flags=re.M))
    assert names == {"mxfp4_scale_stride", "mxfp4_quantize", "mxfp4_dequantize", "mx_padded_offsets",
                     "mxfp4_grouped_gemm", "mx_moe_few_workspace", "mx_moe_few"}
    for n in names:
        assert hasattr(lib, n) and n in nv4._SIGS
    assert '#include "nv4moe/mxfp4.h"' in open(os.path.join(ROOT, "include", "nv4moe.h")).read()
    assert [lib.mxfp4_scale_stride(k) for k in (0, 32, 96, 128, 160, 2048)] == [0, 4, 4, 4, 8, 64]
    assert [nv4.mxfp4_scale_stride(k) for k in (0, 32, 96, 128, 160, 2048)] == [0, 4, 4, 4, 8, 64]


def test_header_compiles_as_c(tmp_path):
    import subprocess
    f = tmp_path / "t.c"
    f.write_text('#include "nv4moe/mxfp4.h"\nint main(void) { return (int)mxfp4_scale_stride(0); }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                        str(f)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _quantize(lib, **o):
    d = dict(x=P, xt=0, xr=64, rows=64, K=96, ldx=96, ri=None, layout=1, nseg=1, so=None, sp=None, rule=0,
             out=mx(64, 96), out_rows=None)
    d.update(o)
    return lib.mxfp4_quantize(d["x"], d["xt"], d["xr"], d["rows"], d["K"], d["ldx"], d["ri"], d["layout"], d["nseg"],
                              d["so"], d["sp"], d["rule"], d["out"], d["out_rows"], None, None)


@pytest.mark.parametrize("want,o", [
    (EALIGN, dict(K=80, out=mx(64, 80))), (EALIGN, dict(ldx=100)), (EALIGN, dict(x=ctypes.c_void_p(0x1008))),
    (EALIGN, dict(xt=1, ldx=98)), (EALIGN, dict(out=mx(64, 96, codes=0x1008))),
    (EALIGN, dict(out=mx(64, 96, scales=0x1002))),
    (EINVAL, dict(ldx=88)), (EINVAL, dict(xt=2)), (EINVAL, dict(layout=0)), (EINVAL, dict(layout=5)),
    (EINVAL, dict(rule=2)), (EINVAL, dict(rows=-1)), (EINVAL, dict(K=-32)), (EINVAL, dict(xr=63)),
    (EINVAL, dict(out=None)), (EINVAL, dict(out=mx(63, 96))), (EINVAL, dict(out=mx(64, 64))),
    (EINVAL, dict(x=None)), (EINVAL, dict(out=mx(64, 96, codes=None))), (EINVAL, dict(out_rows=mx(64, 96))),
    (EINVAL, dict(ri=P, xr=0)), (EINVAL, dict(rows=1 << 31, xr=1 << 31, out=mx(1 << 31, 96))),
    # columns by segment
    (EINVAL, dict(layout=2, out=mx(96, 256))), (EINVAL, dict(layout=2, so=P, sp=P, out=mx(95, 256))),
    (EALIGN, dict(layout=2, so=P, sp=P, out=mx(96, 224))), (EINVAL, dict(layout=2, so=P, sp=P, out=mx(96, 128))),
    (EINVAL, dict(layout=2, so=P, sp=P, nseg=0, out=mx(96, 256))),
    (EINVAL, dict(layout=4, so=P, sp=P, out=mx(96, 256))),
    (EINVAL, dict(layout=4, so=P, sp=P, out=mx(96, 256), out_rows=mx(63, 96))),
    # batched
    (EALIGN, dict(layout=3, nseg=3, out=mx(288, 21))), (EALIGN, dict(layout=3, nseg=4, out=mx(384, 16))),
    (EINVAL, dict(layout=3, nseg=2, out=mx(96, 32))), (EUNSUPPORTED, dict(layout=3, nseg=2, ri=P, out=mx(192, 32))),
])
def test_quantize_refuses(lib, want, o):
    assert _quantize(lib, **o) == want
    assert lib.nv4_last_error().startswith(b"mxfp4_quantize")


def test_empty_calls_succeed(lib):
    assert _quantize(lib, rows=0, xr=0, x=None, out=mx(0, 96)) == 0
    assert _quantize(lib, K=0, ldx=0, out=mx(64, 0)) == 0
    assert lib.mxfp4_dequantize(mx(0, 96), None, 0, 96, None) == 0
    assert lib.mxfp4_grouped_gemm(mx(0, 96, None, None), mx(64, 96), P, 2, 0, 32, None, 0, 0, P, 0, 32, None, 0,
                                  None) == 0
    assert lib.mx_moe_few(None, 0, 64, None, 0, 4, 2, 0, None, None, mx(4 * 64, 64), mx(4 * 64, 32), 64, 32, 0, None, 0,
                          64, None, 0, None, None) == 0


def test_dequantize_and_offsets_refuse(lib):
    d = lambda q=mx(64, 96), out=P, ot=0, ldo=96: lib.mxfp4_dequantize(q, out, ot, ldo, None)
    assert d(q=None) == EINVAL and d(q=mx(64, 80)) == EALIGN and d(q=mx(64, 96, codes=0x1001)) == EALIGN
    assert d(ot=2) == EINVAL and d(ldo=95) == EINVAL and d(ldo=100) == EALIGN and d(out=None) == EINVAL
    assert d(out=ctypes.c_void_p(0x1008)) == EALIGN
    o = lambda a=P, n=4, b=P: lib.mx_padded_offsets(a, n, b, None)
    assert o(a=None) == EINVAL and o(b=None) == EINVAL and o(n=0) == EINVAL and o(n=1025) == EINVAL


def _gemm(lib, **o):
    d = dict(A=mx(100, 96), B=mx(4 * 48, 96), off=P, E=4, M=100, N=48, ri=None, mode=0, epi=0, C=P, ct=1, ldc=48, q=None,
             rule=0)
    d.update(o)
    return lib.mxfp4_grouped_gemm(d["A"], d["B"], d["off"], d["E"], d["M"], d["N"], d["ri"], d["mode"], d["epi"], d["C"],
                                  d["ct"], d["ldc"], d["q"], d["rule"], None)


@pytest.mark.parametrize("want,o", [
    (EINVAL, dict(A=None)), (EINVAL, dict(off=None)), (EINVAL, dict(C=None)), (EINVAL, dict(E=0)),
    (EINVAL, dict(E=1025)), (EINVAL, dict(mode=2)), (EINVAL, dict(epi=2)), (EINVAL, dict(ct=2)), (EINVAL, dict(rule=7)),
    (EINVAL, dict(A=mx(100, 64))), (EALIGN, dict(A=mx(100, 80), B=mx(192, 80))),
    (EINVAL, dict(A=mx(100, 0), B=mx(192, 0))), (EINVAL, dict(N=0)), (EINVAL, dict(N=47)), (EINVAL, dict(ldc=47)),
    (EINVAL, dict(M=101)), (EINVAL, dict(M=-1)), (EALIGN, dict(C=ctypes.c_void_p(0x1002))),
    (EINVAL, dict(ldc=(1 << 22) + 1)), (EINVAL, dict(ri=P, A=mx(0, 96))),
    (EINVAL, dict(A=mx(1 << 27, 96), M=1)),                        # above 4 GiB of codes
    (EUNSUPPORTED, dict(q=mx(100, 48))),                             # quantised result without SwiGLU
    (EALIGN, dict(epi=1, B=mx(4 * 96, 96), q=mx(100, 48))),          # N % 32
    (EINVAL, dict(epi=1, N=32, B=mx(4 * 64, 96), q=mx(99, 32))),
    (EINVAL, dict(epi=1)),                                           # B rows != E * 2N
    (EUNSUPPORTED, dict(mode=1, epi=1, A=mx(8, 128), B=mx(48, 128))),
    (EUNSUPPORTED, dict(mode=1, ri=P, A=mx(8, 128), B=mx(48, 128))),
    (EUNSUPPORTED, dict(mode=1, q=mx(8, 32), A=mx(8, 128), B=mx(48, 128))),
    (EALIGN, dict(mode=1, A=mx(8, 96), B=mx(48, 96))),               # GROUP_K: K % 128
])
def test_gemm_refuses(lib, want, o):
    assert _gemm(lib, **o) == want
    assert lib.nv4_last_error().startswith(b"mxfp4_grouped_gemm")


def test_sizes_behind_32_bit_offsets_are_refused(lib):
    n = 1 << 22
    assert _gemm(lib, E=1, N=n, ldc=n, M=1, A=mx(100, 2112), B=mx(n, 2112)) == EINVAL  # one expert above 4 GiB
    assert b"4 GiB" in lib.nv4_last_error()
    assert _gemm(lib, ri=P, M=1 << 30) == EINVAL and b"row indices" in lib.nv4_last_error()
    seg = dict(layout=2, so=P, sp=P, out=mx(96, 256))
    assert _quantize(lib, ldx=n + 8, **seg) == EINVAL and b"2^22" in lib.nv4_last_error()
    assert _quantize(lib, ldx=n + 8, layout=3, nseg=2, out=mx(192, 32)) == EINVAL


def _few(lib, **o):
    d = dict(x=P, xt=0, ldx=64, lg=P, T=3, E=4, k=2, fl=0, ids=None, w=None, w13=mx(4 * 64, 64), w2=mx(4 * 64, 32), H=64,
             I=32, rule=0, out=P, ot=0, ldo=64, ws=P, wsb=1 << 20)
    d.update(o)
    return lib.mx_moe_few(d["x"], d["xt"], d["ldx"], d["lg"], d["T"], d["E"], d["k"], d["fl"], d["ids"], d["w"], d["w13"],
                          d["w2"], d["H"], d["I"], d["rule"], d["out"], d["ot"], d["ldo"], d["ws"], d["wsb"], None, None)


@pytest.mark.parametrize("want,o", [
    (EINVAL, dict(T=-1)), (EUNSUPPORTED, dict(T=65)), (EINVAL, dict(E=0)), (EUNSUPPORTED, dict(E=1025)),
    (EINVAL, dict(k=0)), (EUNSUPPORTED, dict(k=5)), (EUNSUPPORTED, dict(E=64, k=33)), (EINVAL, dict(fl=2)),
    (EINVAL, dict(lg=None, fl=1)), (EINVAL, dict(rule=2)), (EINVAL, dict(xt=2)), (EINVAL, dict(ot=2)),
    (EINVAL, dict(H=0)), (EALIGN, dict(H=80)), (EALIGN, dict(I=16)), (EINVAL, dict(w13=mx(4 * 32, 64))),
    (EINVAL, dict(w13=None)),
    (EINVAL, dict(H=1 << 17, I=1 << 15, w13=mx(4 << 16, 1 << 17), w2=mx(4 << 17, 1 << 15))), (EINVAL, dict(w2=mx(4 * 64, 64))), (EALIGN, dict(w2=mx(4 * 64, 32, codes=0x1004))),
    (EINVAL, dict(x=None)), (EINVAL, dict(out=None)), (EINVAL, dict(lg=None)), (EINVAL, dict(lg=None, ids=P)),
    (EINVAL, dict(ldx=56)), (EINVAL, dict(ldo=63)), (EALIGN, dict(ldx=68)), (EALIGN, dict(x=ctypes.c_void_p(0x1004))),
    (EALIGN, dict(out=ctypes.c_void_p(0x1001))), (EWORKSPACE, dict(ws=None)), (EWORKSPACE, dict(wsb=100)),
    (EALIGN, dict(ws=ctypes.c_void_p(0x1080))),
])
def test_few_refuses(lib, want, o):
    assert _few(lib, **o) == want
    assert lib.nv4_last_error().startswith(b"mx_moe_few")


def test_few_workspace_grows_with_its_shape(lib):
    f = lib.mx_moe_few_workspace
    assert 0 < f(1, 8, 2, 64, 32) < f(64, 128, 8, 2048, 768)
    assert f(65, 8, 2, 64, 32) == 0 and f(-1, 8, 2, 64, 32) == 0 and f(4, 0, 2, 64, 32) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        nv4.mxfp4_quantize(x)
    q = nv4.MXFP4.empty(4, 64, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        nv4.mxfp4_dequantize(q)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        nv4.mxfp4_grouped_gemm(q, q, off, 1, 4)
    w = nv4.MXExpertWeights(nv4.MXFP4.empty(2 * 64, 64, "cpu"), nv4.MXFP4.empty(2 * 64, 32, "cpu"), 2, 64, 32)
    with pytest.raises(ValueError, match="GPU"):
        nv4.mx_moe_few(x, torch.zeros(4, 2), w, 1)
    with pytest.raises(ValueError, match="contiguous rows"):
        nv4.mxfp4_quantize(x.t())
    with pytest.raises(ValueError, match="contiguous uint8"):
        nv4.MXFP4(q.codes[:, ::2], q.scales, 4, 64).c()
    with pytest.raises(TypeError, match="BF16 or FP32"):
        from nvfp4_w4a4_moe_amd import mxfp4
        mxfp4._float(x.half(), "x")

"""The FP8 and router calls without a GPU: every declared function is exported and bound, and each
documented refusal happens on the host, before anything is launched."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

import nvfp4_w4a4_moe_amd as nv4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, Q = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x2000)
EINVAL, EALIGN, EUNSUPPORTED, EWORKSPACE = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv4.LIB_PATH):
        pytest.fail("libnv4moe.so is not built")
    return nv4.load()


def f8(rows, K, nseg=0, rule=0, codes=0x1000, scales=0x1000):
    return nv4.F8Tensor(codes, scales, rows, K, nseg, rule)


@pytest.mark.parametrize("header,want", [
    ("fp8.h", {"fp8_quantize", "fp8_dequantize", "fp8_transpose", "fp8_grouped_gemm"}),
    ("router.h", {"moe_balance_workspace", "moe_balance_loss", "moe_balance_backward", "moe_combine_backward"})])
def test_declared_functions_are_exported_and_bound(lib, tmp_path, header, want):
    path = os.path.join(ROOT, "include", "nv4moe", header)
    src = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    names = set(re.findall(r"^\s*[a-z_0-9]+\s+([a-z_0-9]+)\s*\(", src, flags=re.M))
    assert names == want
    for n in names:
        assert hasattr(lib, n) and n in nv4._SIGS
    assert f'#include "nv4moe/{header}"' in open(os.path.join(ROOT, "include", "nv4moe.h")).read()
    f = tmp_path / "t.c"
    f.write_text(f'#include "nv4moe/{header}"\nint main(void) {{ return 0; }}\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                        str(f)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _quantize(lib, **o):
    d = dict(x=P, xt=0, xr=64, rows=64, K=80, ldx=80, ri=None, layout=1, nseg=1, so=None, sp=None, rule=0,
             out=f8(64, 80), out_rows=None)
    d.update(o)
    return lib.fp8_quantize(d["x"], d["xt"], d["xr"], d["rows"], d["K"], d["ldx"], d["ri"], d["layout"], d["nseg"],
                            d["so"], d["sp"], d["rule"], d["out"], d["out_rows"], None, None)


@pytest.mark.parametrize("want,o", [
    (EALIGN, dict(K=72, out=f8(64, 72))), (EALIGN, dict(ldx=84)), (EALIGN, dict(x=ctypes.c_void_p(0x1008))),
    (EALIGN, dict(xt=1, ldx=82)), (EALIGN, dict(out=f8(64, 80, codes=0x1008))),
    (EALIGN, dict(out=f8(64, 80, scales=0x1002))),
    (EINVAL, dict(ldx=72)), (EINVAL, dict(xt=2)), (EINVAL, dict(layout=0)), (EINVAL, dict(layout=3)), (EINVAL, dict(layout=6)),
    (EINVAL, dict(rule=2)), (EINVAL, dict(rows=-1)), (EINVAL, dict(K=-16)), (EINVAL, dict(xr=63)),
    (EINVAL, dict(out=None)), (EINVAL, dict(out=f8(63, 80))), (EINVAL, dict(out=f8(64, 64))),
    (EINVAL, dict(x=None)), (EINVAL, dict(out=f8(64, 80, codes=None))), (EINVAL, dict(out_rows=f8(64, 80))),
    (EINVAL, dict(ri=P, xr=0)), (EINVAL, dict(rows=1 << 31, xr=1 << 31, out=f8(1 << 31, 80))),
    # columns by segment
    (EINVAL, dict(layout=2, out=f8(80, 256))), (EINVAL, dict(layout=2, so=P, sp=P, out=f8(79, 256))),
    (EALIGN, dict(layout=2, so=P, sp=P, out=f8(80, 224))), (EINVAL, dict(layout=2, so=P, sp=P, out=f8(80, 128))),
    (EINVAL, dict(layout=2, so=P, sp=P, nseg=0, out=f8(80, 256))),
    (EINVAL, dict(layout=2, so=P, sp=P, ldx=(1 << 22) + 8, out=f8(80, 256))),
    (EINVAL, dict(layout=4, so=P, sp=P, out=f8(80, 256))),
    (EINVAL, dict(layout=4, so=P, sp=P, out=f8(80, 256), out_rows=f8(63, 80))),
    # 128 x 128 blocks
    (EINVAL, dict(layout=5, nseg=3)), (EINVAL, dict(layout=5, nseg=0)), (EUNSUPPORTED, dict(layout=5, nseg=2, ri=P)),
    (EINVAL, dict(layout=5, nseg=2, out=f8(63, 80))),
])
def test_quantize_refuses(lib, want, o):
    assert _quantize(lib, **o) == want
    assert lib.nv4_last_error().startswith(b"fp8_quantize")


def test_empty_calls_succeed(lib):
    assert _quantize(lib, rows=0, xr=0, x=None, out=f8(0, 80)) == 0
    assert _quantize(lib, K=0, ldx=0, out=f8(64, 0)) == 0
    assert lib.fp8_dequantize(f8(0, 80), None, 0, 80, None) == 0
    assert lib.fp8_transpose(f8(0, 80, 2), f8(160, 0), None) == 0
    assert lib.fp8_grouped_gemm(f8(0, 80, codes=None, scales=None), f8(64, 80, 2), P, 2, 0, 32, None, 0, 0, P, 0, 32, None,
                                0, None) == 0
    assert lib.moe_balance_backward(None, 0, 8, 2, None, None, 1, None, None, None, None, None, 0, None, None, None) == 0
    assert lib.moe_combine_backward(None, 0, None, 0, 64, 0, None, None, 0, 2, 64, None, 0, None, None) == 0


def test_what_a_call_writes_is_described(lib):
    """Grouping and rule of the outputs (an empty call: nothing is launched)."""
    o, r = f8(0, 80, 9, 9), f8(0, 80, 9, 9)
    assert _quantize(lib, rows=0, xr=0, x=None, rule=1, out=o) == 0 and (o.nseg, o.rule) == (0, 1)
    assert _quantize(lib, rows=0, xr=0, x=None, layout=5, nseg=4, out=o) == 0 and (o.nseg, o.rule) == (4, 0)
    c = f8(80, 128, 9, 9)
    assert _quantize(lib, rows=0, xr=0, x=None, layout=4, so=P, sp=P, rule=1, out=c, out_rows=r) == 0
    assert (c.nseg, c.rule, r.nseg, r.rule) == (0, 1, 0, 1)
    t = f8(160, 0, 9, 9)
    assert lib.fp8_transpose(f8(0, 80, 2, 1), t, None) == 0 and (t.nseg, t.rule) == (2, 1)


def test_dequantize_and_transpose_refuse(lib):
    d = lambda q=f8(64, 80), out=P, ot=0, ldo=80: lib.fp8_dequantize(q, out, ot, ldo, None)
    assert d(q=None) == EINVAL and d(q=f8(64, 72)) == EALIGN and d(q=f8(64, 80, codes=0x1001)) == EALIGN
    assert d(ot=2) == EINVAL and d(ldo=79) == EINVAL and d(ldo=84) == EALIGN and d(out=None) == EINVAL
    assert d(out=ctypes.c_void_p(0x1008)) == EALIGN and d(q=f8(64, 80, 3)) == EINVAL and d(q=f8(64, 80, 0, 2)) == EINVAL
    t = lambda q=f8(64, 80, 2), out=f8(160, 32, codes=0x2000, scales=0x2000): lib.fp8_transpose(q, out, None)
    assert t(q=f8(64, 80)) == EINVAL and t(q=f8(66, 80, 2)) == EALIGN and t(q=None) == EINVAL and t(out=None) == EINVAL
    assert t(out=f8(160, 48, codes=0x2000, scales=0x2000)) == EINVAL and t(q=f8(64, 80, 3)) == EINVAL
    assert t(out=f8(160, 32)) == EINVAL and b"overlap" in lib.nv4_last_error()


def _gemm(lib, **o):
    d = dict(A=f8(100, 80), B=f8(4 * 48, 80, 4), off=P, E=4, M=100, N=48, ri=None, mode=0, epi=0, C=P, ct=1, ldc=48, q=None,
             rule=0)
    d.update(o)
    return lib.fp8_grouped_gemm(d["A"], d["B"], d["off"], d["E"], d["M"], d["N"], d["ri"], d["mode"], d["epi"], d["C"],
                                d["ct"], d["ldc"], d["q"], d["rule"], None)


@pytest.mark.parametrize("want,o", [
    (EINVAL, dict(A=None)), (EINVAL, dict(off=None)), (EINVAL, dict(C=None)), (EINVAL, dict(E=0)),
    (EINVAL, dict(E=1025)), (EINVAL, dict(mode=2)), (EINVAL, dict(epi=2)), (EINVAL, dict(ct=2)), (EINVAL, dict(rule=7)),
    (EINVAL, dict(A=f8(100, 64))), (EALIGN, dict(A=f8(100, 72), B=f8(192, 72, 4))),
    (EINVAL, dict(A=f8(100, 0), B=f8(192, 0, 4))), (EINVAL, dict(N=0)), (EINVAL, dict(N=47)), (EINVAL, dict(ldc=47)),
    (EINVAL, dict(M=101)), (EINVAL, dict(M=-1)), (EALIGN, dict(C=ctypes.c_void_p(0x1002))),
    (EINVAL, dict(ldc=(1 << 20) + 1)), (EINVAL, dict(ri=P, A=f8(0, 80))), (EINVAL, dict(ri=P, M=1 << 30)),
    (EINVAL, dict(A=f8(1 << 26, 80), M=1)),                         # above 4 GiB of codes
    (EINVAL, dict(A=f8(100, 80, 1))), (EINVAL, dict(B=f8(192, 80))), (EINVAL, dict(B=f8(192, 80, 2))),  # scale grouping
    (EINVAL, dict(A=f8(100, 80, 0, 2))),
    (EUNSUPPORTED, dict(q=f8(100, 48))),                             # quantised result without SwiGLU
    (EALIGN, dict(epi=1, B=f8(4 * 96, 80, 4), q=f8(100, 48))),       # SwiGLU: N % 32
    (EINVAL, dict(epi=1, N=32, B=f8(4 * 64, 80, 4), q=f8(99, 32))),
    (EINVAL, dict(epi=1, N=64)),                                     # B rows != E * 2N
    (EUNSUPPORTED, dict(mode=1, epi=1, A=f8(8, 128), B=f8(48, 128))),
    (EUNSUPPORTED, dict(mode=1, ri=P, A=f8(8, 128), B=f8(48, 128))),
    (EUNSUPPORTED, dict(mode=1, q=f8(8, 32), A=f8(8, 128), B=f8(48, 128))),
    (EALIGN, dict(mode=1, A=f8(8, 80), B=f8(48, 80))),               # GROUP_K: K % 128
    (EINVAL, dict(mode=1, A=f8(8, 128), B=f8(48, 128, 4))),
])
def test_gemm_refuses(lib, want, o):
    assert _gemm(lib, **o) == want
    assert lib.nv4_last_error().startswith(b"fp8_grouped_gemm")


def _router(**o):
    d = dict(lg=P, T=16, E=8, k=2, ids=P, mask=None, nseg=1, so=None)
    d.update(o)
    return [d[n] for n in ("lg", "T", "E", "k", "ids", "mask", "nseg", "so")]


ROUTER = [(EINVAL, dict(T=-1)), (EINVAL, dict(E=0)), (EINVAL, dict(k=0)), (EUNSUPPORTED, dict(E=1025)),
          (EUNSUPPORTED, dict(k=9)), (EUNSUPPORTED, dict(E=64, k=33)), (EINVAL, dict(nseg=0)),
          (EUNSUPPORTED, dict(nseg=65537, so=P)), (EINVAL, dict(nseg=2)), (EINVAL, dict(lg=None)), (EINVAL, dict(ids=None)),
          (EINVAL, dict(T=1 << 31))]


@pytest.mark.parametrize("want,o", ROUTER)
def test_balance_refuses(lib, want, o):
    assert lib.moe_balance_loss(*_router(**o), P, P, P, P, P, 1 << 30, None, None) == want
    assert lib.nv4_last_error().startswith(b"moe_balance_loss")
    assert lib.moe_balance_backward(*_router(**o), P, P, P, P, 0, P, None, None) == want
    assert lib.nv4_last_error().startswith(b"moe_balance_backward")


def test_balance_buffers_are_checked(lib):
    f = lambda c=P, p=P, t=P, l=P, ws=P, n=1 << 20: lib.moe_balance_loss(*_router(), c, p, t, l, ws, n, None, None)
    assert f(c=None) == f(p=None) == f(t=None) == f(l=None) == EINVAL
    need = lib.moe_balance_workspace(16, 8, 1)
    assert need > 0 and f(ws=None) == EWORKSPACE and f(n=need - 1) == EWORKSPACE and f(ws=ctypes.c_void_p(0x1080)) == EALIGN
    w = lib.moe_balance_workspace
    assert w(16, 8, 1) < w(65536, 8, 1) < w(65536, 128, 1) < w(65536, 128, 40) and w(-1, 8, 1) == w(1, 0, 1) == w(1, 8, 0) == 0
    b = lambda c=P, t=P, dl=P, fl=0, out=P: lib.moe_balance_backward(*_router(), c, t, dl, None, fl, out, None, None)
    assert b(c=None) == b(t=None) == b(fl=2) == b(out=None) == EINVAL


@pytest.mark.parametrize("want,o", [
    (EINVAL, dict(T=-1)), (EINVAL, dict(k=0)), (EINVAL, dict(H=0)), (EINVAL, dict(rows=-1)), (EINVAL, dict(yt=2)),
    (EINVAL, dict(ot=2)), (EALIGN, dict(H=62)), (EINVAL, dict(ldy=60)), (EALIGN, dict(ldy=66)), (EINVAL, dict(lddy=60)),
    (EALIGN, dict(lddy=66)), (EALIGN, dict(dout=ctypes.c_void_p(0x1004))), (EALIGN, dict(Y=ctypes.c_void_p(0x1004))),
    (EALIGN, dict(dY=ctypes.c_void_p(0x2004))), (EALIGN, dict(yt=1, Y=ctypes.c_void_p(0x1008))), (EINVAL, dict(dout=None)),
    (EINVAL, dict(Y=None)), (EINVAL, dict(row=None)), (EINVAL, dict(w=None)), (EINVAL, dict(dY=None, dw=None)),
    (EINVAL, dict(dY=P)), (EINVAL, dict(T=1 << 31))])
def test_combine_backward_refuses(lib, want, o):
    d = dict(dout=P, ot=0, Y=P, yt=0, ldy=64, rows=32, row=P, w=P, T=16, k=2, H=64, dY=Q, lddy=64, dw=P)
    d.update(o)
    assert lib.moe_combine_backward(d["dout"], d["ot"], d["Y"], d["yt"], d["ldy"], d["rows"], d["row"], d["w"], d["T"],
                                    d["k"], d["H"], d["dY"], d["lddy"], d["dw"], None) == want
    assert lib.nv4_last_error().startswith(b"moe_combine_backward")


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = nv4.FP8.empty(4, 64, device="cpu")
    w = nv4.FP8.empty(8, 64, 2, device="cpu")
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    lg, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    b = nv4.MoeBalance(torch.zeros(2), torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, 8),
                       torch.zeros(1, dtype=torch.int32))
    for call in (lambda: nv4.fp8_quantize(x), lambda: nv4.fp8_dequantize(q), lambda: nv4.fp8_transpose(w),
                 lambda: nv4.fp8_grouped_gemm(q, w, off, 2, 4), lambda: nv4.moe_balance_loss(lg, ids),
                 lambda: nv4.moe_balance_backward(lg, ids, b, torch.zeros(2)),
                 lambda: nv4.moe_combine_backward(x, x, ids, torch.zeros(4, 2)),
                 lambda: nv4.fp8_quantize_expert_weights(torch.zeros(2, 64, 32), torch.zeros(2, 32, 32)),
                 lambda: nv4.fp8_moe_forward(x, torch.zeros(4, 2), nv4.F8ExpertWeights(w, w, 2, 64, 32), 1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="contiguous rows"):
        nv4.fp8_quantize(x.t())
    for bad in (nv4.FP8(q.codes[:, ::2], q.scales, 4, 64), nv4.FP8(q.codes, q.scales.half(), 4, 64),
                nv4.FP8(q.codes, q.scales, 4, 64, 1), nv4.FP8(w.codes, w.scales[:1], 8, 64, 2)):
        if bad.nseg == 1:
            bad.scales = torch.zeros(3)
        with pytest.raises(ValueError, match="contiguous uint8"):
            bad.c()
    for bad, o in ((dict(logits=lg.half()), {}), (dict(logits=lg.t()), {}), (dict(topk_ids=ids[:3]), {}),
                   (dict(topk_ids=ids.long()), {}), ({}, dict(mask=torch.zeros(3, dtype=torch.bool))),
                   ({}, dict(mask=torch.zeros(4))), ({}, dict(seg_offsets=torch.zeros(1, dtype=torch.int32)))):
        a = dict(logits=lg, topk_ids=ids) | bad
        with pytest.raises(ValueError):
            nv4.moe_balance_loss(a["logits"], a["topk_ids"], **o)
    with pytest.raises(ValueError, match="counts"):
        nv4.moe_balance_backward(lg, ids, None, torch.zeros(2))


"""The FP8 product's DMAs are written in assembly, for which the compiler adds no wait states.  In the assembly that it
makes of these kernels: a buffer load reads a scalar register that a vector instruction (a lane read, a comparison) wrote
at least five wait states before, and m0, which the DMAs write and the compiler takes for its own, is used by nothing
else."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from nvfp4_w4a4_moe_amd import build

FILES = ["f8_gemm_large.hip", "f8_gemm_medium.hip", "f8_gemm_small.hip"]
STATES = 5


def scalars(text):
    out = set()
    for lo, hi, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def instructions(asm):
    """(line, mnemonic, operands) of the code in order; None where a function begins."""
    for n, line in enumerate(asm.splitlines(), 1):
        text = line.split(";")[0].strip()
        if re.match(r"_Z\w+:", text):
            yield n, None, []
        elif text and text[0] not in ".#" and not text.endswith(":"):
            op, _, rest = text.partition(" ")
            yield n, op, [x.strip() for x in rest.split(",")]


def written_by_vector(op, args):
    if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
        return scalars(args[0])
    if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_", op) or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")):
        return scalars(args[1])
    return set()


def short_waits(asm):
    """Buffer loads to LDS that read a scalar register too soon: [(line, register, wait states)], and how many there are."""
    since, loads, short = {}, 0, []
    for n, op, args in instructions(asm):
        if op is None:
            since = {}
            continue
        if op.startswith("buffer_load") and any("lds" in a.split() for a in args):
            loads += 1
            short += [(n, r, since[r]) for a in args[1:] for r in scalars(a) if since.get(r, STATES) < STATES]
        passed = int(args[0], 0) + 1 if op == "s_nop" else 1
        since = {r: w + passed for r, w in since.items() if w + passed < STATES}
        if op.startswith("s_") and args and not op.startswith(("s_cmp", "s_cbranch", "s_waitcnt", "s_nop", "s_barrier")):
            for r in scalars(args[0]):
                since.pop(r, None)
        since.update({r: 0 for r in written_by_vector(op, args)})
    return loads, short


def test_the_scan_counts_wait_states():
    asm = "_Z1kv:\n v_readlane_b32 s4, v1, 0\n s_mov_b32 m0, s9\n s_nop {}\n buffer_load_dword v0, s[4:7], s8 offen lds\n"
    assert short_waits(asm.format(2)) == (1, [(5, 4, 4)]) and short_waits(asm.format(3)) == (1, [])
    assert short_waits(asm.format(0).replace("s_mov_b32 m0, s9", "s_mov_b32 s4, 0")) == (1, [])
    asm = "_Z1kv:\n v_cmp_eq_u32_e64 s[8:9], v1, v2\n buffer_load_dwordx4 v0, s[4:7], s8 offen nt lds ; comment\n"
    assert short_waits(asm) == (1, [(3, 8, 0)])


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    out = tmp_path_factory.mktemp("asm")
    flags = [f for f in build.HIP_FLAGS if f != "-fPIC"]

    def compile(name):
        to = out / (name + ".s")
        r = subprocess.run([build.hipcc(), *flags, "-fPIC", "-x", "hip", "-S", "--offload-device-only",
                            os.path.join(build.CSRC, name), "-o", str(to)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return to.read_text()

    with ThreadPoolExecutor(max_workers=len(FILES)) as ex:
        return dict(zip(FILES, ex.map(compile, FILES)))


@pytest.mark.parametrize("name", FILES)
def test_scalar_operands_of_the_dmas_have_landed(listings, name):
    loads, short = short_waits(listings[name])
    assert loads > 100 and short == []


@pytest.mark.parametrize("name", FILES)
def test_only_the_dmas_use_m0(listings, name):
    asm = listings[name]
    blocks = re.findall(r"#ASMSTART\n(.*?)#ASMEND", asm, flags=re.S)
    inside = sum(len(re.findall(r"\bm0\b", b)) for b in blocks if "lds" in b)
    code = "\n".join(" ".join([op, *args]) for _, op, args in instructions(asm) if op)
    assert inside > 100 and len(re.findall(r"\bm0\b", code)) == inside

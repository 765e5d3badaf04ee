"""What the prompt kernel's loads in assembly rely on, seen in its compiled form (no
GPU): the compiler does not look into assembly, and cannot be told that m0 is written.
"""
import importlib.util
import os
import re
import subprocess

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_group_quantized_amd")


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    spec = importlib.util.spec_from_file_location("q4g128_build_flags", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        hipcc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = str(tmp_path_factory.mktemp("asm") / "attn_prefill.s")
    cmd = [hipcc] + build.COMPILE_FLAGS + ["-x", "hip", "--cuda-device-only", "-S",
                                           os.path.join(build.CSRC, "attn_prefill.hip"), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True, timeout=600)
    with open(out) as f:
        return [line.strip() for line in f]


def blocks(lines):
    """The instructions of each piece of assembly, in order."""
    found, inside = [], None
    for line in lines:
        if line.startswith(";;#ASMSTART"):
            inside = []
        elif line.startswith(";;#ASMEND"):
            found.append(inside)
            inside = None
        elif inside is not None and line:
            inside.append(line)
    return found


def wait_states(instruction):
    return int(instruction.split()[1]) + 1 if instruction.startswith("s_nop") else 1


def test_only_the_loads_use_m0(lines):
    loads = [b for b in blocks(lines) if any("global_load_lds" in i for i in b)]
    assert len(loads) > 100
    for b in loads:
        assert [i.split()[0] for i in b] == ["s_mov_b32", "s_nop", "global_load_lds_dwordx4"], b
        assert b[0].startswith("s_mov_b32 m0, s")
    code = [line.split(";")[0] for line in lines]
    assert sum(bool(re.search(r"\bm0\b", line)) for line in code) == len(loads)


def test_scalar_bases_are_waited_for(lines):
    """A memory operation needs five wait states after a vector instruction (which reads a lane, say a spilled
    scalar's) has written its scalar base: they lie within the assembly, whatever stands before it."""
    scalar = [b for b in blocks(lines) if re.search(r"global_load_lds_dwordx4 v\d+, s\[", b[-1] if b else "")]
    assert len(scalar) > 100
    for b in scalar:
        assert sum(wait_states(i) for i in b[:-1]) >= 5, b

"""The kernels of drafted tokens and latent rows in their compiled form (no GPU): what their loads in assembly rely on,
and the rescaling of outputs in accumulation registers.
"""
import importlib.util
import os
import re
import subprocess

import pytest

from test_attention_assembly import PKG, blocks, wait_states

SOURCES = ["attn_tree.hip", "latent_prefill.hip", "latent_attn.hip", "latent_expand.hip"]


@pytest.fixture(scope="module", params=SOURCES)
def lines(request, tmp_path_factory):
    spec = importlib.util.spec_from_file_location("q4g128_build_flags", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        hipcc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = str(tmp_path_factory.mktemp("asm") / "kernel.s")
    cmd = [hipcc] + build.COMPILE_FLAGS + ["-x", "hip", "--cuda-device-only", "-S",
                                           os.path.join(build.CSRC, request.param), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True, timeout=600)
    with open(out) as f:
        return [line.strip() for line in f]


def test_loads_and_what_else_is_in_assembly(lines):
    """m0 is written by the loads alone; a memory operation needs five wait states after a vector instruction has
    written its scalar base, and they lie within the assembly; an accumulation register that has just been written
    needs waits before a product reads it, which stand behind the rescaling."""
    found = [b for b in blocks(lines) if b]
    loads = [b for b in found if any("global_load_lds" in i for i in b)]
    assert len(loads) > 20
    for b in loads:
        assert [i.split()[0] for i in b] == ["s_mov_b32", "s_nop", "global_load_lds_dwordx4"], b
        assert re.match(r"s_mov_b32 m0, (s\d|vcc_)", b[0])
        if re.search(r"global_load_lds_dwordx4 v\d+, (s\[|vcc)", b[-1]):
            assert sum(wait_states(i) for i in b[:-1]) >= 5, b
    code = [line.split(";")[0] for line in lines]
    assert sum(bool(re.search(r"\bm0\b", line)) for line in code) == len(loads)
    scaled = [b for b in found if any("accvgpr" in i for i in b)]
    for b in scaled:
        assert [i.split()[0] for i in b] == ["v_accvgpr_read_b32", "v_mul_f32", "v_accvgpr_write_b32"], b
    assert bool(scaled) == (["s_nop 7"] in found)


def test_scratch(lines):
    """Outputs, queries and weights stay in registers (the prompt kernels keep a few addresses elsewhere)."""
    sizes = [int(m.group(1)) for m in (re.match(r"\.private_segment_fixed_size:\s+(\d+)", line) for line in lines) if m]
    assert len(sizes) >= 4
    prompt = any("attn_prefill_kernel" in line for line in lines)
    assert max(sizes) <= (64 if prompt else 0), sizes

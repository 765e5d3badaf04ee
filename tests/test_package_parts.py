"""What the package needs for what: the products only the library; the cache and
attention calls their compiled binding too.  No GPU.
"""
import os
import shutil
import subprocess
import sys

import pytest

q4 = pytest.importorskip("int4_group_quantized_amd")

PKG = os.path.dirname(os.path.abspath(q4.__file__))

USE = """
import torch
import int4_group_quantized_amd as q4
assert q4.library().q4g128_gemv(None, None, None, None, None, 1, 128, None) == q4.Q4_EINVAL
for call in (q4.q4g128_rope_append, q4.q4g128_attn_decode, q4.q4g128_attn_prefill):
    try:
        call(*[torch.zeros(1)] * 7)
    except ImportError as e:
        assert "build.py" in str(e), e
    else:
        raise AssertionError("no ImportError")
try:
    q4.q4g128_gemv(*[torch.zeros(1, 1)] * 4)
except ValueError:
    print("products work")
"""


@pytest.mark.parametrize("binding", ["missing", "of another build"])
def test_products_without_the_compiled_binding(tmp_path, binding):
    pkg = tmp_path / "int4_group_quantized_amd"
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    os.symlink(os.path.join(PKG, "libq4g128.so"), pkg / "libq4g128.so")
    if binding != "missing":
        (pkg / "_binding.so").write_bytes(b"not a module")
    got = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "products work" in got.stdout, got.stderr

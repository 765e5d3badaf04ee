"""What the package needs for what: the products only the library; the cache and
attention calls their compiled binding too; the library's build no torch.  No GPU.
"""
import importlib.util
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


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py with its compiler calls recorded, writing to a temporary directory."""
    spec = importlib.util.spec_from_file_location("q4g128_build_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.done = []
    monkeypatch.setattr(mod, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(mod, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(mod, "_compile", lambda src, verbose: src)
    monkeypatch.setattr(mod, "_link", lambda objs, name, path, verbose: mod.done.append(name))

    def run(cmd, what, verbose):
        mod.done.append(what)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(mod, "_run", run)
    return mod


def test_build_with_torch(build):
    assert build.build_library() == build.LIB_PATH
    assert build.done == [build.LIB_NAME, build.DIAG_NAME, build.BINDING_SOURCE, "the binding"]
    assert os.path.exists(build.BINDING_PATH)


@pytest.mark.parametrize("without", ["torch", "headers"])
def test_build_without_torch(build, monkeypatch, tmp_path, capsys, without):
    """The libraries are built and returned; a binding of an earlier build does not stay."""
    if without == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    else:
        import torch
        monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    open(build.BINDING_PATH, "w").close()
    assert build.build_library() == build.LIB_PATH
    assert build.done == [build.LIB_NAME, build.DIAG_NAME]
    assert not os.path.exists(build.BINDING_PATH)
    assert "binding" in capsys.readouterr().out

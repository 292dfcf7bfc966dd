"""What importing the package needs: the library, the binding's module, and CUDA in torch only for the device side."""
import importlib.util
import os
import pathlib
import shutil
import subprocess
import sys

import pytest

PACKAGE = pathlib.Path(__file__).resolve().parents[1] / "huffman_decode_canonical_b200"


def _import(tmp_path, leave_out, code):
    """Runs `code` where the package is a copy without some of its built files: (exit code, output, errors)"""
    there = tmp_path / PACKAGE.name
    there.mkdir()
    for name in ("__init__.py", "libentro.so", "_binding.so"):
        if name not in leave_out:
            shutil.copy(PACKAGE / name, there / name)
    done = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True, timeout=300, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    return done.returncode, done.stdout, done.stderr


@pytest.mark.parametrize("missing", ["libentro.so", "_binding.so"])
def test_a_missing_build_says_how_to_build(tmp_path, missing):
    leave_out = ("libentro.so", "_binding.so") if missing == "libentro.so" else (missing,)
    code, _, err = _import(tmp_path, leave_out, "import huffman_decode_canonical_b200")
    last = err.strip().splitlines()[-1]
    assert code != 0 and last.startswith("ImportError") and missing in last and "build.py" in last and "circular" not in last


_HOST_ONLY = """
import numpy as np, torch
torch.version.cuda = None
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    delattr(torch._C, name)
import huffman_decode_canonical_b200 as entro
w = np.random.default_rng(0).standard_normal((40, 64)).astype(np.float32)
blob = entro.encode(w, bits=4)
assert entro.Blob.from_bytes(blob.to_bytes()).info()["n"] == 40 * 64
for call in (lambda: entro.quantize_tokens(torch.zeros(2, 32, dtype=torch.bfloat16)),
             lambda: entro.attention_prompt(*[torch.zeros(2, 2, 64, dtype=torch.bfloat16)] * 3, torch.tensor([0, 2], dtype=torch.int32))):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("taken")
print("good")
"""


def test_the_host_side_needs_no_cuda_in_torch(tmp_path):
    code, out, err = _import(tmp_path, ("_binding.so",), _HOST_ONLY)
    assert code == 0 and out.strip() == "good", err[-2000:]


def test_another_torch_or_interpreter_builds_the_binding_again(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_builder_under_test", PACKAGE / "build.py")
    builder = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(builder)
    import sysconfig

    import torch
    made_for = tmp_path / "made_for.txt"
    monkeypatch.setattr(builder, "BINDING_MADE_FOR", str(made_for))
    monkeypatch.setattr(builder, "_stale", lambda *a: False)  # by its sources the module is up to date
    assert builder._binding_stale()
    made_for.write_text(builder._binding_abi())
    assert not builder._binding_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert builder._binding_stale()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu")
        assert builder._binding_stale()
    assert not builder._binding_stale()

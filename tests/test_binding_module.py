"""The binding without the CPython module of the block-scaled calls, and without
torch (no GPU needed)."""

import importlib.metadata
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_the_module_is_built_and_loads(tp):
    from megatron_tensor_transformer_gate_gb300 import build
    assert os.path.exists(build.pycall_path())
    out = python("from megatron_tensor_transformer_gate_gb300 import binding as"
                 " b\nm = b._load()\n"
                 "print(m.__name__, m.quantize(1, 2, 3, None, None, None))")
    assert out.split()[0].endswith("._tpcall") and out.split()[1] == "None"


def test_calls_of_the_library_need_neither_module_nor_torch(tp):
    # what counts bytes and operations is reached by ctypes alone
    out = python("import sys\nsys.modules['torch'] = None\n"
                 "from megatron_tensor_transformer_gate_gb300 import binding as"
                 " b\nb.lib()\n"
                 "print(b.comm_bytes(b.SCOPE_MLP, 64, 128, 2, b.BF16)"
                 "['payload_bytes'])\n"
                 "assert not any('_tpcall' in m for m in sys.modules)")
    assert int(out) > 0


def test_without_the_module_the_python_checks_make_the_calls(tp, monkeypatch,
                                                             tmp_path):
    from megatron_tensor_transformer_gate_gb300 import build
    monkeypatch.setattr(build, "pycall_path", lambda: str(tmp_path / "no.so"))
    monkeypatch.setattr(tp, "_tpcall", None)
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = tp.fp8_block_empty(4, 256, device="cpu")
    with pytest.warns(UserWarning, match="not built"), \
            pytest.raises(ValueError, match="not on a GPU"):
        tp.quantize_fp8_block(x, q, s)
    for name in ("quantize", "swiglu", "swiglu_bwd", "norm", "gemm"):
        assert getattr(tp._tpcall, name)(x, q, s) is None


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    from megatron_tensor_transformer_gate_gb300 import build
    here = build.pycall_path()
    monkeypatch.setattr(importlib.metadata, "version", lambda _: "0.1")
    assert build.pycall_path() != here
    assert here.endswith(".so") and sys.implementation.cache_tag[-3:] in here


def test_the_library_is_built_without_the_module(tp, monkeypatch, tmp_path,
                                                 capsys):
    from megatron_tensor_transformer_gate_gb300 import build
    monkeypatch.setattr(build, "pycall_path", lambda: str(tmp_path / "no.so"))
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda n: None
                        if n in ("g++", "c++") else which(n))
    assert build.build() == build.LIB
    assert "g++ not found" in capsys.readouterr().err
    fake = tmp_path / "g++"
    fake.write_text("#!/bin/sh\necho no headers >&2\nexit 1\n")
    fake.chmod(0o755)
    monkeypatch.setattr(build.shutil, "which", lambda n: str(fake)
                        if n == "g++" else which(n))
    assert build.build() == build.LIB
    assert "no headers" in capsys.readouterr().err
    assert not (tmp_path / "no.so").exists()

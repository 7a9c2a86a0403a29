"""The compiled part of the binding: loaded only by the operators that need it,
and refused, with what to do, when it is missing or was built for another
Python or PyTorch."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "mxfp8_w8a8_quantized_b200"


@pytest.fixture(scope="module")
def build():
    from mxfp8_w8a8_quantized_b200 import build
    build.build()
    return build


@pytest.fixture
def copy(build, tmp_path):
    """The package as installed (no sources), in a folder of its own."""
    d = tmp_path / PKG
    d.mkdir()
    for name in os.listdir(os.path.join(ROOT, PKG)):
        if name.endswith(".py") or name.endswith(".so"):
            shutil.copy(os.path.join(ROOT, PKG, name), d / name)
    return tmp_path


def _run(where, code):
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    r = subprocess.run([sys.executable, "-c", code], cwd=where, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


CHECK = """
import torch
from mxfp8_w8a8_quantized_b200 import mxfp8 as mx, build
assert mx.scale_bytes(129, 512) == 2 * 4 * 512 and mx.mxfp4_scale_bytes(1, 32) == 512
assert mx._lib.mxfp8_rmsnorm_quantize(None, 0, None, 0, None, 0, None, 0, 1e-6, 0, 64, None, None, 1, None) == 0
try:
    mx.quantize(torch.zeros(4, 64))
except ValueError:
    pass                                    # the older operators' own refusal
x = torch.zeros(4, 64, dtype=torch.bfloat16)
for call in (lambda: mx.mxfp4_quantize(x), lambda: mx.rmsnorm_quantize(x, x[0]), lambda: mx.gated_quantize(x, x)):
    try:
        call()
        raise SystemExit("not refused")
    except %s as e:
        assert %r in str(e), e
"""
HINT = "python -m mxfp8_w8a8_quantized_b200.build"


def test_whole(copy):
    _run(copy, CHECK % ("ValueError", "must be"))


def test_without_the_compiled_part(copy):
    os.remove(copy / PKG / "_native.so")
    _run(copy, CHECK % ("ImportError", HINT))


def test_compiled_for_another_version(copy, build):
    so = copy / PKG / "_native.so"
    tag = build.native_tag().encode()
    data = so.read_bytes()
    assert tag in data
    so.write_bytes(data.replace(tag, tag.replace(b"torch ", b"torch 0")[:len(tag)]))
    _run(copy, CHECK % ("ImportError", HINT))
    _run(copy, CHECK % ("ImportError", "another Python or PyTorch"))


def test_a_binary_of_another_version_is_rebuilt(build, tmp_path, monkeypatch):
    assert build.native_problem() is None and build.up_to_date()
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0.1")
    assert "another Python or PyTorch" in build.native_problem() and not build.up_to_date()


def test_the_library_is_built_without_pytorch(build, monkeypatch):
    monkeypatch.setattr(build, "_has_torch", lambda: False)
    monkeypatch.setattr(build, "NATIVE", os.path.join(ROOT, PKG, "no_such_binding.so"))
    calls = []
    monkeypatch.setattr(build, "_build_native", lambda: calls.append(1))
    assert build.up_to_date() and build.build() == build.LIB and not calls

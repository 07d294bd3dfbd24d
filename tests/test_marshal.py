"""The binding's compiled tensor checks on tensors that have a GPU's device but
no plain sizes or memory: an exception each, in a process of its own, since an
unhandled C++ one would end it.  Fake tensors need no GPU."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SETUP = """
import sys, torch
sys.path.insert(0, %r)
import convolution_conv2d_forward_amd as cc
from torch._subclasses.fake_tensor import FakeTensorMode
d = cc.linear_desc_create(cc.make_linear_params(8, 8))
def refused(x, kind):
    assert x.is_cuda
    try:
        cc.linear_forward(d, x, x, None, None, x, stream=0)
    except kind as e:
        assert "x: " in str(e), e
        return
    raise SystemExit("accepted")
""" % ROOT


@pytest.mark.parametrize("case", [
    """
def f(t):
    refused(t, TypeError)
    return t
with FakeTensorMode():
    torch.func.vmap(f)(torch.empty(3, 2, 8, device="cuda"))
""", """
from torch.fx.experimental.symbolic_shapes import ShapeEnv
m = FakeTensorMode(shape_env=ShapeEnv())
x = m.from_tensor(torch.empty(2, 8), static_shapes=False)
with m:
    x = x.to("cuda")
refused(x, (TypeError, RuntimeError))
""", """
with FakeTensorMode():
    x = torch.empty(2, 8, device="cuda")
refused(x, TypeError)
""", """
with FakeTensorMode():
    x = torch.sparse_coo_tensor(torch.zeros(2, 1, dtype=torch.long, device="cuda"), torch.ones(1, device="cuda"), (2, 8))
refused(x, TypeError)
"""], ids=["vmap", "symbolic sizes", "no memory", "sparse"])
def test_tensors_without_plain_memory_are_refused(case):
    r = subprocess.run([sys.executable, "-c", SETUP + case], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_missing_checks_are_named_before_a_descriptor_is_made(monkeypatch):
    import convolution_conv2d_forward_amd as cc
    from convolution_conv2d_forward_amd import attention
    made = []
    monkeypatch.setattr(attention, "_tensor", None)
    monkeypatch.setitem(sys.modules, "convolution_conv2d_forward_amd._marshal", None)
    monkeypatch.setattr(attention._lib, "linear_desc_create", lambda *a: made.append(a) or 0)
    with pytest.raises(ImportError, match="_marshal.so"):
        cc.linear_desc_create(cc.make_linear_params(8, 8))
    assert not made, "a handle that nothing would destroy"


def _build_script(monkeypatch, path):
    import importlib.util
    spec = importlib.util.spec_from_file_location("_build", os.path.join(ROOT, "convolution_conv2d_forward_amd", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    monkeypatch.setattr(m, "MARSHAL", str(path))
    return m


def test_library_builds_without_torch(monkeypatch, tmp_path, capsys):
    m = _build_script(monkeypatch, tmp_path / "_marshal.so")
    monkeypatch.setitem(sys.modules, "torch", None)
    m._build_marshal(False)
    assert "_marshal.so is not built" in capsys.readouterr().out and not os.listdir(tmp_path)


def test_checks_build_with_the_librarys_own_compiler(monkeypatch, tmp_path):
    m = _build_script(monkeypatch, tmp_path / "_marshal.so")
    monkeypatch.setenv("CXX", "/nonexistent/compiler")
    m._build_marshal(False)
    assert os.listdir(tmp_path) == ["_marshal.so"]

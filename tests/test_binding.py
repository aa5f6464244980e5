"""The compiled part of the binding (_mok_bind.so): what works without it.  Each case in a process of its own; no
GPU needed."""
import subprocess
import sys

import pytest

from helpers import ROOT


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


USE = """
import torch
from mixture_experts_layer_build_gb300 import mok
assert mok.mok_workspace_bytes(mok.make_config(), mok.make_shape(16, 128, 128, 4, 2)) > 0
layer = mok.Layer(16, 128, 128, 4, 2, device="cpu")  # the routed layer is there
x = torch.zeros((4, 64), dtype=torch.bfloat16)
plan = mok.FFN(4, 64, 64, device="cpu")
for call in (lambda: mok.rmsnorm_forward(x, x[0], 1e-6), lambda: mok.rmsnorm_backward(x, x[0], x[0], x),
             lambda: plan.forward(x, x, x, x), lambda: plan.backward(x, x, x, x, x)):
    try:
        call()
    except ImportError as e:
        print(e, "/", e.__cause__)
"""


def test_the_routed_layer_does_without_it():
    out = python("import sys\nsys.modules['mixture_experts_layer_build_gb300._mok_bind'] = None" + USE).splitlines()
    assert len(out) == 4 and all("_mok_bind" in line and "build()" in line for line in out), out


def test_the_library_is_linked_when_the_binding_does_not_compile(monkeypatch, tmp_path):
    """A host without Python's or torch's headers still gets libmok.so, and an error."""
    from mixture_experts_layer_build_gb300 import build
    linked = []
    for name in ("LIB", "BIND"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))

    class Done:
        stdout = stderr = ""

        def __init__(self, returncode):
            self.returncode = returncode

    def fake(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        bad = cmd[-3].endswith("mok_bind.cpp")
        if not bad:
            open(out, "w").close()
            linked.append(out)
        return Done(1 if bad else 0)
    monkeypatch.setattr(build.subprocess, "run", fake)
    with pytest.raises(RuntimeError, match="mok_bind"):
        build.build()
    assert (tmp_path / "LIB").exists() and not (tmp_path / "BIND").exists()


def test_a_binding_of_another_torch_is_not_used():
    out = python("import torch\ntorch.__version__ = '0.0.1'" + USE).splitlines()
    assert len(out) == 4 and all("0.0.1" in line.split("/", 1)[1] for line in out), out


def test_the_binding_is_rebuilt_for_another_torch(monkeypatch):
    from mixture_experts_layer_build_gb300 import build
    import torch
    assert not build.bind_stale() and torch.__version__ in build.bind_target()
    monkeypatch.setattr(build, "bind_target", lambda: "torch 0.0.1, python 3.12")
    assert build.bind_stale()

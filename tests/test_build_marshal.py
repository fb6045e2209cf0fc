"""The library is built with nvcc alone; the wrappers' extension module is extra, and is built for one torch."""
import os
import subprocess
import sys

import pytest

from kalman_delta_rule_b200 import binding as B
from kalman_delta_rule_b200 import build


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """The library's objects are up to date; it is linked anew, to a place of its own."""
    build.build()
    out = str(tmp_path / "libkdn.so")
    monkeypatch.setattr(build, "OUT", out)
    return out


def test_the_library_is_linked_whatever_becomes_of_the_module(fresh, monkeypatch):
    def broken(force=False):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(build, "build_marshal", broken)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert os.path.getsize(fresh) > 0


@pytest.mark.parametrize("what", ["torch", "g++"])
def test_without_torch_or_a_host_compiler(fresh, monkeypatch, what):
    if what == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)      # `import torch` raises ImportError
    else:
        import shutil
        monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None)
    with pytest.warns(UserWarning, match="not built: no " + what.replace("+", "\\+")):
        assert build.build() == fresh
    assert os.path.getsize(fresh) > 0


def test_another_torch_builds_the_module_again(monkeypatch, tmp_path):
    import torch
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("module")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_kdn_marshal.so"))
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    build.build_marshal()
    build.build_marshal()
    assert len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.0")
    build.build_marshal()
    build.build_marshal()
    assert len(runs) == 2 and any("9.9.0" in a for a in runs[1])


def test_a_module_of_another_torch_is_not_used(monkeypatch, tmp_path):
    import torch
    build.build()
    assert B._native_module(torch).abi == build.marshal_abi()
    monkeypatch.setattr(torch, "__version__", "9.9.0")
    with pytest.warns(UserWarning, match="was built for"):
        assert B._native_module(torch) is None
    monkeypatch.setattr(B, "MARSHAL_PATH", str(tmp_path / "none.so"))
    with pytest.warns(UserWarning, match="not built"):
        assert B._native_module(torch) is None
    bad = tmp_path / "bad.so"
    bad.write_text("no module")
    monkeypatch.setattr(B, "MARSHAL_PATH", str(bad))
    with pytest.warns(UserWarning, match="cannot be loaded"):
        assert B._native_module(torch) is None


@pytest.mark.gpu
def test_the_wrappers_without_the_module(kdn, monkeypatch, tmp_path):
    import torch
    from tests import test_gpu_linear as TL
    x = TL.make(3, 2, 70, 2, 64, 32, "bf16", grads=True)
    a = (x["q"], x["k"], x["v"], x["g"])

    def calls():
        S = x["S0"].clone()
        o, last = kdn.linear_forward(*a, S0=x["S0"])
        y = kdn.layer_norm(o)
        n = kdn.layer_norm_backward(x["do"], o, None, y[1], y[2])
        g = kdn.linear_backward(*a, x["do"], S0=x["S0"])
        step = kdn.linear_decode_step(*(t[:, 0].contiguous() for t in a), S)
        many = kdn.linear_decode_tokens(*a, S)
        return [o, last, *y, n["dx"], *g.values(), step, many, S]
    want = calls()
    monkeypatch.setattr(kdn, "_native_mod", None)
    monkeypatch.setattr(kdn, "MARSHAL_PATH", str(tmp_path / "none.so"))
    with pytest.warns(UserWarning, match="not built"):
        got = calls()
    assert kdn._native_mod is kdn._NoNative
    assert all(torch.equal(u, v) for u, v in zip(want, got))

"""The library and the calls of the paged cache where their quick binding (_binding.so) cannot be built or loaded."""
import os
import warnings

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from online_softmax_fa2_gb300 import build as ofa_build
from online_softmax_fa2_gb300 import paged


@pytest.fixture(scope="module", autouse=True)
def built():
    ofa_build.build()


def test_the_library_is_linked_without_a_compiler_for_the_binding(monkeypatch, tmp_path):
    monkeypatch.setattr(ofa_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(ofa_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(ofa_build, "STAMP", str(tmp_path / "_binding.stamp"), raising=False)
    (tmp_path / "_binding.so").write_bytes(b"of older sources")
    os.utime(tmp_path / "_binding.so", (0, 0))
    run = ofa_build.subprocess.run

    def no_gxx(cmd, **kw):
        if "g++" in os.path.basename(cmd[0]):
            raise FileNotFoundError("g++")
        return run(cmd, **kw)

    monkeypatch.setattr(ofa_build.subprocess, "run", no_gxx)
    with pytest.warns(RuntimeWarning, match="quick binding"):
        assert ofa_build.build() == str(tmp_path / "lib.so")
    assert os.path.exists(tmp_path / "lib.so") and not os.path.exists(tmp_path / "_binding.so")


@pytest.mark.parametrize("content", [None, b"no module"])
def test_without_a_binding_there_is_a_warning_and_no_more(monkeypatch, tmp_path, content):
    monkeypatch.setattr(ofa_build, "BINDING", str(tmp_path / "_binding.so"))
    if content:
        (tmp_path / "_binding.so").write_bytes(content)
    monkeypatch.setattr(paged, "_quick", None)
    with pytest.warns(RuntimeWarning, match="quick binding"):
        assert paged._binding() is False
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert paged._binding() is False  # said once


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The binding and its stamp in a folder of their own, as a build has left them."""
    for name in ("BINDING", "STAMP"):
        old = getattr(ofa_build, name)
        new = tmp_path / os.path.basename(old)
        new.write_bytes(open(old, "rb").read())
        monkeypatch.setattr(ofa_build, name, str(new))


def test_a_binding_of_another_torch_is_built_anew(elsewhere):
    assert ofa_build.binding_is_current()
    before = os.stat(ofa_build.BINDING).st_mtime_ns
    ofa_build.build()
    assert os.stat(ofa_build.BINDING).st_mtime_ns == before  # nothing to do
    with open(ofa_build.STAMP, "w") as f:
        f.write(ofa_build.binding_stamp().replace("torch ", "torch 0."))
    assert not ofa_build.binding_is_current()
    ofa_build.build()
    assert ofa_build.binding_is_current() and os.stat(ofa_build.BINDING).st_mtime_ns > before
    os.remove(ofa_build.STAMP)  # of no known origin
    assert not ofa_build.binding_is_current()


def test_a_binding_of_another_torch_is_not_loaded(elsewhere, monkeypatch):
    monkeypatch.setattr(paged, "_quick", None)
    stamp = ofa_build.binding_stamp()
    monkeypatch.setattr(ofa_build, "binding_stamp", lambda: stamp + " and another")
    with pytest.warns(RuntimeWarning, match="another torch"):
        assert paged._binding() is False


@pytest.mark.gpu
def test_the_calls_run_without_a_binding(monkeypatch, tmp_path):
    from paged_helpers import paged_inputs
    s = paged_inputs([1, 3], [40, 90], 4, 2, 64, 16, poison=False)
    k, v = (torch.randn(4, 2, 64, device="cuda").bfloat16() for _ in "kv")
    calls = [lambda: ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"]),
             lambda: ofa.attn_paged_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"])[0]]
    want = [c() for c in calls]
    monkeypatch.setattr(ofa_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(paged, "_quick", None)
    with pytest.warns(RuntimeWarning, match="quick binding"):
        got = [c() for c in calls]
    assert all(torch.equal(a, b) for a, b in zip(got, want))

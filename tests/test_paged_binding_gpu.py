"""The quick binding (csrc/binding.cpp) against the Python one (paged.py): the same results, the same refusals, and calls that it
leaves alone."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from online_softmax_fa2_gb300 import paged
from paged_helpers import angles, paged_inputs
from paged_q8_helpers import q8_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture
def count(monkeypatch):
    """Counts of calls that the quick binding took and left; slow() makes it leave all."""
    taken = {"yes": 0, "no": 0}
    real, off = paged._quick_call, []

    def quick(*a):
        r = None if off else real(*a)
        taken["no" if r is None else "yes"] += 1
        return r

    monkeypatch.setattr(paged, "_quick_call", quick)
    taken["slow"] = lambda on: off.append(1) if on else off.clear()
    return taken


def both(count, f):
    count["slow"](False)
    a = f()
    assert count["yes"] == 1 and count["no"] == 0, "left to Python"
    count["slow"](True)
    b = f()
    count.update(yes=0, no=0)
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    for x, y in zip(a, b):
        assert x.shape == y.shape and x.dtype == y.dtype and x.stride() == y.stride() and torch.equal(x, y)
    return a


@pytest.mark.parametrize("q8", [False, True])
def test_the_same_results(count, q8):
    new, lens = [1, 40, 3], [100, 300, 50]
    make = q8_inputs if q8 else paged_inputs
    s = make(new + [0], lens + [400], 8, 2, 128, 16, seed=1, poison=False)
    pt, pl = s["bt"][3:].contiguous(), s["lens"][3:].contiguous()
    bt, ln, cu = s["bt"][:3], s["lens"][:3].contiguous(), s["cu"][:4].contiguous()
    sc = (s["ks"], s["vs"]) if q8 else ()
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(44, 2, 128, generator=g).bfloat16().to(DEV) for _ in "kv")
    w = torch.rand(128, generator=g).bfloat16().to(DEV)
    cs, pos = angles(400, 64).to(DEV), torch.arange(44, dtype=torch.int32, device=DEV)
    append = ofa.attn_paged_append_q8 if q8 else ofa.attn_paged_append
    fwd = ofa.attn_paged_fwd_q8 if q8 else ofa.attn_paged_fwd
    kw = dict(k_scales=sc[0], v_scales=sc[1]) if q8 else {}
    both(count, lambda: append(s["q"], k, v, s["kp"], s["vp"], *sc, bt, ln, cu, wq=w, wk=w, cos_sin=cs, positions=pos, eps=1e-5, interleaved=True))
    both(count, lambda: append(s["q"], k, v, s["kp"], s["vp"], *sc, bt, ln, cu, q_out=torch.empty(44, 16, 128, dtype=torch.bfloat16, device=DEV)[:, ::2]))
    both(count, lambda: fwd(s["q"], s["kp"], s["vp"], *sc, bt, ln, cu))
    both(count, lambda: fwd(s["q"], s["kp"], s["vp"], *sc, bt, ln, cu, max_q=40, causal=False, scale=0.3))
    both(count, lambda: fwd(s["q"][:42], s["kp"], s["vp"], *sc, bt, ln))
    both(count, lambda: ofa.attn_paged_prefix_fwd(s["q"], s["kp"], s["vp"], bt, ln, pt, pl, cu, max_q=40, **kw))
    if q8:
        both(count, lambda: ofa.attn_paged_read_q8(s["kp"], s["vp"], *sc, bt, ln, 44, cu))
        both(count, lambda: ofa.attn_paged_read_q8(s["kp"].view(torch.uint8), s["vp"], sc[0].view(torch.uint8), sc[1], bt, ln, 42, dtype=torch.float32))
    # given tensors come back themselves
    o, l = torch.empty_like(s["q"]), torch.empty(44, 8, device=DEV)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    r = fwd(s["q"], s["kp"], s["vp"], *sc, bt, ln, cu, workspace=ws, out=o, lse=l)
    assert r[0] is o and r[1] is l
    assert ofa.device_error_flags() == 0


def test_refusals_are_those_of_python(count):
    s = q8_inputs([1, 2], [20, 30], 4, 2, 64, 16, poison=False)
    a = [s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"]]
    wrong = [(0, s["q"].half(), TypeError), (0, s["q"][0], ValueError), (0, s["q"].cpu(), ValueError), (1, s["kp"].view(torch.int8), ValueError),
             (1, s["kp"][..., :32], ValueError), (2, s["vp"][:2], ValueError), (3, s["ks"].cpu(), ValueError), (5, s["bt"].long(), ValueError),
             (5, s["bt"][0], ValueError), (6, s["lens"][:1], ValueError), (7, s["cu"][:2], ValueError), (2, s["vp"].transpose(1, 3), ValueError)]
    for i, bad, kind in wrong:
        for slow in (False, True):
            count["slow"](slow)
            with pytest.raises(kind):
                ofa.attn_paged_fwd_q8(*a[:i], bad, *a[i + 1:])
    for kw in (dict(out=torch.empty(3, 4, 64, device=DEV)), dict(lse=torch.empty(4, 3, device=DEV).T), dict(workspace=torch.empty(8, 8, device=DEV).T)):
        for slow in (False, True):
            count["slow"](slow)
            with pytest.raises(ValueError):
                ofa.attn_paged_fwd_q8(*a, **kw)
    for slow in (False, True):
        count["slow"](slow)
        with pytest.raises(ofa.AttnError) as e:
            ofa.attn_paged_fwd_q8(*a, scale=-1.0)
        assert e.value.status == ofa.Status.UNSUPPORTED and "scale" in str(e.value)
    assert ofa.device_error_flags() == 0


def test_a_decode_loop_keeps_nothing():
    """Outputs and workspaces of the quick calls belong to the caller: memory does not grow, references are let go."""
    s = q8_inputs([1] * 8, [700] * 8, 8, 2, 128, 16, poison=False)
    f = lambda: ofa.attn_paged_fwd_q8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"])  # noqa: E731
    f()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(300):
        f()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
    import sys
    n = sys.getrefcount(s["q"]), sys.getrefcount(s["kp"])
    o, lse = f()
    assert (sys.getrefcount(s["q"]), sys.getrefcount(s["kp"])) == n and sys.getrefcount(o) == sys.getrefcount(lse) == 2


def test_streams_of_the_quick_calls():
    s = q8_inputs([1] * 4, [400] * 4, 8, 2, 64, 16, poison=False)
    a = (s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"])
    want = ofa.attn_paged_fwd_q8(*a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    q = torch.zeros_like(s["q"])
    with torch.cuda.stream(st):  # the copy and the call, both on st
        torch.cuda._sleep(2_000_000)
        q.copy_(s["q"])
        got = ofa.attn_paged_fwd_q8(q, *a[1:])
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert math.isfinite(float(want[1].sum()))

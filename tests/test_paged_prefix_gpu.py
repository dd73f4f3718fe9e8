"""Attention behind shared prefixes against the 64-bit attention over the prefix's keys followed by the own
ones (paged_q8_helpers.attention_ref), over bf16 caches and caches in 8 bits."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_helpers import angles, paged_inputs
from paged_q8_helpers import E4M3, E8M0, attention_ref, check_attention, q8_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def inputs(new, lens, plens, cuts, Hq, Hkv, d, page, q8, seed=0, spread=0.5):
    """Prefixes are made as sequences without tokens, behind the others; cuts: packed tokens where the groups begin and end."""
    every, toks = list(lens) + list(plens), list(new) + [0] * len(plens)
    make = (lambda **k: q8_inputs(toks, every, Hq, Hkv, d, page, seed=seed, spread=spread, **k)) if q8 else (
        lambda **k: paged_inputs(toks, every, Hq, Hkv, d, page, seed=seed, **k))
    s = make()
    B = len(lens)
    s["pt"], s["plens"] = s["bt"][B:].contiguous(), s["lens"][B:].contiguous()
    s["bt"], s["lens"], s["cu"] = s["bt"][:B].contiguous(), s["lens"][:B].contiguous(), s["cu"][:B + 1].contiguous()
    s["pcu"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    T = sum(new)
    t = torch.arange(T)
    c = torch.tensor(cuts)
    groups = torch.searchsorted(c, t, right=True) - 1
    groups[(groups >= len(plens)) | (groups < 0)] = -1
    return s, groups


def run(s, causal=True, scale=None, **kw):
    return ofa.attn_paged_prefix_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"], causal=causal,
                                     scale=scale, k_scales=s.get("ks"), v_scales=s.get("vs"), **kw)


CASES = [  # new, lens, prefix lengths, cuts, Hq, Hkv, d, page, causal
    ([1], [1], [1], [0, 1], 1, 1, 64, 16, True),
    ([1, 1], [40, 3], [300], [0, 2], 8, 2, 64, 16, True),
    ([1] * 9, [129, 128, 0, 64, 63, 1, 1000, 2, 0], [700], [0, 9], 32, 8, 128, 64, True),   # idle places see the prefix
    ([1] * 6, [20, 30, 40, 50, 60, 70], [100, 257, 0], [0, 2, 5, 6], 4, 4, 128, 16, True),  # a prefix without keys
    ([4, 4, 4], [4, 700, 33], [500], [4, 12], 4, 4, 64, 16, True),                          # a sequence without a prefix
    ([4, 2, 0, 8], [3, 1, 50, 0], [90, 33], [0, 6, 14], 6, 2, 128, 32, True),               # rows that see no own key
    ([4, 2, 0, 8], [3, 1, 50, 0], [0, 0], [0, 6, 14], 6, 2, 128, 32, True),                 # and no prefix
    ([7, 7], [129, 256], [1000], [0, 14], 7, 1, 128, 32, False),
    ([100, 1, 17], [350, 1025, 17], [900, 31], [0, 101, 118], 28, 4, 128, 32, True),
    ([129], [400], [129], [0, 129], 4, 4, 64, 64, False),
    ([300, 2], [300, 900], [2000], [0, 302], 8, 8, 128, 128, True),
    ([255, 0, 257], [255, 0, 700], [600], [10, 500], 3, 1, 64, 16, True),                   # cuts inside sequences
    ([1] * 70, [5] * 70, [4000], [0, 70], 4, 1, 128, 16, True),
    ([2] * 40, list(range(2, 42)), [64] * 40, list(range(0, 81, 2)), 2, 1, 64, 16, True),   # many prefixes
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("hint", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_prefix(case, hint, q8):
    new, lens, plens, cuts, Hq, Hkv, d, page, causal = case
    s, groups = inputs(new, lens, plens, cuts, Hq, Hkv, d, page, q8, seed=len(new))
    ofa.device_error_flags()
    o, lse = run(s, causal, max_q=max(new) if hint else None)
    assert ofa.device_error_flags() == 0
    check_attention(o, lse, s, new, lens, causal, 1 / math.sqrt(d), groups, plens)
    o2, lse2 = run(s, causal, max_q=max(new) if hint else None)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


@pytest.mark.parametrize("seed", range(12))
def test_prefix_random(seed):
    g = torch.Generator().manual_seed(300 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    B, Hkv, G, P = r(1, 9), r(1, 3), r(1, 9), r(1, 3)
    d, page, causal, q8 = (64, 128)[r(0, 1)], (16, 32, 64, 128)[r(0, 3)], r(0, 4) > 0, bool(seed % 2)
    big = r(0, 2)
    new = [1 if big == 0 else r(0, (0, 12, 120)[big]) for _ in range(B)]
    lens = [r(0, (900, 300, 300)[big]) for _ in range(B)]
    T = sum(new)
    if T == 0:
        return
    cuts = sorted(r(0, T) for _ in range(P + 1))
    plens = [r(0, 1500) for _ in range(P)]
    s, groups = inputs(new, lens, plens, cuts, Hkv * G, Hkv, d, page, q8, seed=seed, spread=(0.0, 2.0)[r(0, 1)])
    o, lse = run(s, causal, max_q=r(0, 1) * max(new), scale=0.2)
    assert ofa.device_error_flags() == 0
    check_attention(o, lse, s, new, lens, causal, 0.2, groups, plens, what=f"seed {seed}")


def test_one_prefix_of_all_needs_no_cuts():
    new = [1] * 6
    s, groups = inputs(new, [5] * 6, [100, 60], [0, 3, 6], 4, 2, 64, 16, False)
    a = run(s)
    b = ofa.attn_paged_prefix_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("q8", [False, True])
def test_rows_outside_stay_whatever_the_workspace_holds(q8):
    new, lens = [2, 30], [40, 50]
    s, _ = inputs(new, lens, [200], [0, 32], 4, 2, 64, 16, q8)
    o0, l0 = run(s, max_q=30)
    pad = torch.randn(5, 4, 64, device=DEV).bfloat16()
    p = dict(s, q=torch.cat([pad, s["q"], pad]), cu=s["cu"] + 5, pcu=s["pcu"] + 5)
    args = (p["q"], p["kp"], p["vp"], p["bt"], p["lens"], p["pt"], p["plens"], p["cu"], p["pcu"])
    n = ofa.paged_prefix_fwd_workspace_bytes(*args, max_q=30, k_scales=s.get("ks"), v_scales=s.get("vs"))
    assert n >= 42 * 4 * (64 + 2) * 4
    for fill in (0, 255, 127):
        out, lse = torch.full_like(p["q"], 3.0), torch.full((42, 4), 5.0, device=DEV)
        run(p, max_q=30, out=out, lse=lse, workspace=torch.full((n,), fill, dtype=torch.uint8, device=DEV))
        assert torch.equal(out[5:-5], o0) and torch.equal(lse[5:-5], l0)
        assert bool((out[:5] == 3).all()) and bool((out[-5:] == 3).all()) and bool((lse[:5] == 5).all()) and bool((lse[-5:] == 5).all())
    assert ofa.device_error_flags() == 0
    # tokens of a prefix that no sequence has, and the other way about
    p["pcu"] = torch.tensor([0, 42], dtype=torch.int32, device=DEV)
    o1, l1 = run(p, max_q=30)
    assert torch.equal(o1[5:-5], o0) and torch.equal(l1[5:-5], l0)
    p["pcu"] = torch.tensor([7, 30], dtype=torch.int32, device=DEV)
    o2, l2 = run(p, max_q=30, workspace=torch.full((n,), 255, dtype=torch.uint8, device=DEV))
    groups = torch.full((42,), -1)
    groups[7:30] = 0
    check_attention(o2[5:-5], l2[5:-5], s, new, lens, True, 1 / 8, groups[5:-5], [200])


def test_a_nan_in_the_prefix_reaches_those_that_see_it():
    new = [1] * 8 + [40]
    lens = [30] * 8 + [64]
    for q8 in (False, True):
        s, groups = inputs(new, lens, [300, 200], [0, 4, 48], 4, 2, 128, 16, q8, seed=4)
        want, wl = run(s)
        page = int(s["pt"][1, 3])
        if q8:
            s["kp"].view(torch.uint8)[page, 5, 0, 7] = 0x7F
        else:
            s["kp"][page, 5, 0, 7] = math.nan
        o, lse = run(s)
        hit = (groups == 1).to(DEV)
        assert bool(o[hit][:, :2].isnan().all()) and bool(lse[hit][:, :2].isnan().all())
        assert torch.equal(o[:, 2:], want[:, 2:]) and torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])


def test_an_infinite_value_of_the_own_keys_leaves_rows_that_see_none():
    """0 * inf of a tile's weights may reach rows that see its keys; a sequence's rows before its keys begin have a state
    without weight, and take the prefix's alone."""
    new, lens = [20, 20], [10, 20]  # the first ten rows see no own key
    s, groups = inputs(new, lens, [100], [0, 40], 2, 1, 128, 16, False, seed=6)
    want, wl = run(s, max_q=20)
    s["vp"][int(s["bt"][0, 0]), 9, 0, 3] = math.inf
    o, lse = run(s, max_q=20)
    assert torch.equal(o[:10], want[:10]) and torch.equal(lse, wl) and torch.equal(o[20:], want[20:])


@pytest.mark.parametrize("cu", [[0, 4, 2], [0, 9, 9], [-5, 2, 6], [6, 4, 2], [2, 2, 2]])
def test_malformed_cuts_fault_nothing(cu):
    for q8 in (False, True):
        s, _ = inputs([2, 2, 2], [20, 30, 17], [40, 50], [0, 2, 6], 2, 1, 64, 16, q8)
        s["pcu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        ofa.device_error_flags()
        run(s)
        assert ofa.device_error_flags() in ((0,) if cu == [2, 2, 2] else (4,))
        s["pcu"][:] = torch.tensor([0, 2, 6], dtype=torch.int32)
        s["pt"][0, 1], s["plens"][1] = -3, 10 ** 6
        run(s)
        assert ofa.device_error_flags() == 6


@pytest.mark.parametrize("q8", [False, True])
def test_malformed_cuts_after_others_in_one_workspace(q8):
    """Rows that no prefix's attention has reached find what an earlier call left there, entries of cut rows among it."""
    new, lens, plens, cuts = [300, 200, 150], [300, 400, 900], [5000, 3000], [0, 420, 650]
    s, groups = inputs(new, lens, plens, cuts, 8, 2, 64, 16, q8, seed=8)
    n = ofa.paged_prefix_fwd_workspace_bytes(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"], 300,
                                             k_scales=s.get("ks"), v_scales=s.get("vs"))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    ofa.device_error_flags()
    for bad in ([0, 700, 650], [0, 0, 650], [400, 100, 650], [-9, 90, 20]):
        s["pcu"] = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        o, lse = run(s, max_q=300, workspace=ws)
        assert ofa.device_error_flags() == 0
        check_attention(o, lse, s, new, lens, True, 1 / 8, groups, plens, what=str(bad))
        s["pcu"] = torch.tensor(bad, dtype=torch.int32, device=DEV)
        run(s, max_q=300, workspace=ws)
        assert (ofa.device_error_flags() != 0) == (bad != [0, 0, 650])


@pytest.mark.parametrize("q8", [False, True])
def test_a_serving_run(q8):
    """A prompt appended once, eight answers that go on from it in pages of their own, step by step: what each step
    gives is the attention over the prompt and the answer, and equals attn_paged_fwd's over one table of both within
    the two calls' bounds."""
    Hq, Hkv, d, page, P, B = 8, 2, 128, 16, 230, 8
    g = torch.Generator().manual_seed(3)
    rnd = lambda *x: torch.randn(*x, generator=g).bfloat16().to(DEV)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pages = 15 + 2 * B + 1
    perm = torch.randperm(pages, generator=g).int().to(DEV)
    pt, bt = perm[:15][None], perm[15:15 + 2 * B].view(B, 2)
    w, cs = (1 + 0.2 * rnd(d).float()).bfloat16(), angles(400, d).to(DEV)
    if q8:
        cache = [torch.zeros(pages, page, Hkv, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in "kv"]
        cache += [torch.zeros(pages, Hkv, page, dtype=torch.uint8, device=DEV).view(E8M0) for _ in "kv"]
        append, names = ofa.attn_paged_append_q8, ("kp", "vp", "ks", "vs")
    else:
        cache = [torch.zeros(pages, page, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
        append, names = ofa.attn_paged_append, ("kp", "vp")
    append(rnd(P, Hq, d), rnd(P, Hkv, d), rnd(P, Hkv, d), *cache, pt, i32([P]), wq=w, wk=w, cos_sin=cs)
    lens = [0] * B
    for new in ([5, 1, 9, 3, 17, 1, 2, 8], [1] * B, [1] * B):
        lens = [a + b for a, b in zip(lens, new)]
        T = sum(new)
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        pos = torch.cat([torch.arange(P + n - c, P + n) for n, c in zip(lens, new)]).int().to(DEV)
        q = append(rnd(T, Hq, d), rnd(T, Hkv, d), rnd(T, Hkv, d), *cache, bt, i32(lens), cu, wq=w, wk=w, cos_sin=cs, positions=pos)
        s = dict(zip(names, cache), q=q, bt=bt, lens=i32(lens), cu=cu, pt=pt, plens=i32([P]), pcu=i32([0, T]))
        o, lse = run(s, max_q=max(new))
        check_attention(o, lse, s, new, lens, True, 1 / math.sqrt(d), torch.zeros(T, dtype=torch.long), [P], what=str(lens))
    assert ofa.device_error_flags() == 0


def test_captured_with_a_workspace_shared_by_two_graphs():
    new, lens = [1] * 20, [30 + i for i in range(20)]
    s, groups = inputs(new, lens, [800], [0, 20], 8, 2, 128, 16, False, seed=2)
    t, tg = inputs(new, lens, [500], [0, 20], 8, 2, 128, 16, False, seed=3)
    want = [run(x) for x in (s, t)]
    n = max(ofa.paged_prefix_fwd_workspace_bytes(x["q"], x["kp"], x["vp"], x["bt"], x["lens"], x["pt"], x["plens"], x["cu"], x["pcu"]) for x in (s, t))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x in (s, t):
        out, lse = torch.zeros_like(x["q"]), torch.zeros(20, 8, device=DEV)
        with torch.cuda.stream(side):
            run(x, workspace=ws, out=out, lse=lse)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(x, workspace=ws, out=out, lse=lse)
        outs.append((out, lse))
    for _ in range(3):
        for gr, (out, lse), w in zip(graphs, outs, want):
            out.zero_()
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_python_refusals():
    s, _ = inputs([1, 1], [20, 20], [40], [0, 2], 2, 1, 64, 16, True)
    a = [s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"]]
    with pytest.raises(ValueError):
        ofa.attn_paged_prefix_fwd(*a, k_scales=s["ks"])
    with pytest.raises(ValueError):
        ofa.attn_paged_prefix_fwd(*a)  # codes without scales
    with pytest.raises(ValueError):
        ofa.attn_paged_prefix_fwd(*a[:5], s["pt"].long(), *a[6:], k_scales=s["ks"], v_scales=s["vs"])
    with pytest.raises(ValueError):
        ofa.attn_paged_prefix_fwd(*a[:8], s["pcu"][:1], k_scales=s["ks"], v_scales=s["vs"])
    with pytest.raises(ofa.AttnError) as e:
        ofa.attn_paged_prefix_fwd(*a, k_scales=s["ks"], v_scales=s["vs"], workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == ofa.Status.WORKSPACE


BESIDE = [  # decode steps: the own keys' attention beside the prefixes'; new, lens, prefix lengths, cuts, Hq, Hkv, d, page
    ([1] * 40, [30 + 5 * i for i in range(40)], [3000, 10, 0, 700], [3, 13, 20, 30, 38], 8, 2, 128, 16),   # finished and cut prefixes, tokens with none
    ([1] * 70, [1 + 40 * i % 900 for i in range(70)], [5000], [0, 70], 32, 8, 128, 64),
    ([2] * 12, [2] * 12, [129] * 3, [0, 8, 16, 24], 16, 2, 64, 32),
    ([3, 0, 4, 1] * 8, [900, 0, 4, 0] * 8, [2500, 2500], [0, 33, 64], 4, 2, 64, 128),
    ([1] * 300, [17] * 300, [6000], [0, 300], 4, 1, 128, 16),                                             # more rows than two tiles
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", BESIDE)
def test_decode_steps_behind_prefixes(case, q8):
    new, lens, plens, cuts, Hq, Hkv, d, page = case
    s, groups = inputs(new, lens, plens, cuts, Hq, Hkv, d, page, q8, seed=5)
    want = None
    n = ofa.paged_prefix_fwd_workspace_bytes(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"], max(new),
                                             k_scales=s.get("ks"), v_scales=s.get("vs"))
    ofa.device_error_flags()
    for fill in (0, 255, 191):  # (191: -1.5 in every word, 255: NaN)
        o, lse = run(s, max_q=max(new), workspace=torch.full((n,), fill, dtype=torch.uint8, device=DEV))
        assert ofa.device_error_flags() == 0
        if want is None:
            check_attention(o, lse, s, new, lens, True, 1 / math.sqrt(d), groups, plens, what=f"fill {fill}")
            want = o, lse
        assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), want[1].view(torch.int32))


SHORT = [  # prefixes too short to be cut; more sequences than a warp looks at at once, and than 32 times as many
    ([1] * 24, [10 + 30 * i for i in range(24)], [600], [0, 24], 8, 2, 128, 16),
    ([1] * 40, [0, 3] * 20, [128, 0, 513], [2, 20, 21, 40], 16, 4, 64, 64),
    ([1, 0, 2] * 400, [7 * i % 50 for i in range(1200)], [13 * i % 600 for i in range(50)], [24 * i for i in range(51)], 4, 1, 64, 16),
    ([1] * 20, [5 + 40 * i for i in range(20)], [4000], [0, 20], 64, 64, 128, 64),   # and long prefixes of many heads
    ([1] * 1100, [i % 40 for i in range(1100)], [3000, 5, 640], [0, 500, 520, 1090], 2, 1, 64, 16),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", SHORT)
def test_short_prefixes_and_many_sequences(case, q8):
    new, lens, plens, cuts, Hq, Hkv, d, page = case
    s, groups = inputs(new, lens, plens, cuts, Hq, Hkv, d, page, q8, seed=6)
    ofa.device_error_flags()
    for fill in (255, 191):
        n = ofa.paged_prefix_fwd_workspace_bytes(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"],
                                                 max(new), k_scales=s.get("ks"), v_scales=s.get("vs"))
        o, lse = run(s, max_q=max(new), workspace=torch.full((n,), fill, dtype=torch.uint8, device=DEV))
        assert ofa.device_error_flags() == 0
    check_attention(o, lse, s, new, lens, True, 1 / math.sqrt(d), groups, plens)


@pytest.mark.parametrize("q8", [False, True])
def test_decode_steps_captured_one_after_the_other(q8):
    """Steps of two batches in one graph over one workspace, replayed with other lengths in the same tensors."""
    new = [1] * 24
    steps = [inputs(new, [40 + i for i in range(24)], [1500], [0, 24], 8, 2, 128, 16, q8, seed=k) for k in (6, 7)]
    ws = torch.zeros(max(ofa.paged_prefix_fwd_workspace_bytes(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"], 1,
                                                              k_scales=s.get("ks"), v_scales=s.get("vs")) for s, _ in steps), dtype=torch.uint8, device=DEV)
    outs = [(torch.zeros_like(s["q"]), torch.zeros(24, 8, device=DEV)) for s, _ in steps]

    def go():
        for (s, _), (o, lse) in zip(steps, outs):
            run(s, max_q=1, workspace=ws, out=o, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
        go()
    for lens, plen in (([40 + i for i in range(24)], 1500), ([1 + 2 * i for i in range(24)], 700), ([0] * 24, 3)):
        for s, _ in steps:
            s["lens"].copy_(torch.tensor(lens))
            s["plens"].fill_(plen)
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        for (s, groups), (o, lse) in zip(steps, outs):
            check_attention(o, lse, s, new, lens, True, 1 / math.sqrt(128), groups, [plen], what=str(plen))
    assert ofa.device_error_flags() == 0


def test_calls_on_two_streams_at_once():
    data = [inputs([1] * 30, [100 + i for i in range(30)], [2000], [0, 30], 16, 4, 128, 16, q8, seed=8)[0] for q8 in (False, True)]
    data.append(inputs([60, 1, 30], [200, 300, 30], [900], [0, 91], 8, 2, 64, 32, False, seed=9)[0])
    want = [run(s) for s in data]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in data], [[] for _ in data]
    for _ in range(6):
        for i, s in enumerate(data):
            got[i].append(run(s, stream=streams[i]))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o, lse in outs:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_steps_back_to_back_read_what_the_append_before_wrote():
    """Appends and prefix attention queued without a pause: each attention starts early beside the work before it, and still
    sees its tokens, lengths and keys."""
    Hq, Hkv, d, page, P, B, steps = 8, 2, 128, 16, 900, 40, 6
    g = torch.Generator().manual_seed(5)
    rnd = lambda *x: torch.randn(*x, generator=g).bfloat16().to(DEV)  # noqa: E731
    pages = 57 + B + 1
    perm = torch.randperm(pages, generator=g).int().to(DEV)
    pt, bt = perm[:57][None], perm[57:57 + B].view(B, 1)
    plens = torch.tensor([P], dtype=torch.int32, device=DEV)
    base = [rnd(pages, page, Hkv, d) for _ in "kv"]
    qkv = [(rnd(B, Hq, d), rnd(B, Hkv, d), rnd(B, Hkv, d)) for _ in range(steps)]

    def go(sync):
        cache = [t.clone() for t in base]
        lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        got = []
        torch.cuda.synchronize()
        for q, k, v in qkv:
            lens += 1
            qr = ofa.attn_paged_append(q, k, v, *cache, bt, lens)
            got.append(ofa.attn_paged_prefix_fwd(qr, *cache, bt, lens, pt, plens))
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got

    want = go(True)
    for _ in range(5):
        for (o, lse), (wo, wl) in zip(go(False), want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)

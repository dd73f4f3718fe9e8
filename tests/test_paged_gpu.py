"""Attention over a paged cache against a plain form in 64 bits (paged_helpers), and runs of the
operators together."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from online_softmax_fa2_gb300 import paged
from paged_helpers import angles, check_paged, paged_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(s, causal=True, scale=None, **kw):
    return ofa.attn_paged_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], causal=causal, scale=scale, **kw)


CASES = [  # new, lens, Hq, Hkv, d, page, causal
    ([1], [1], 1, 1, 64, 16, True),
    ([1], [300], 8, 2, 64, 16, True),
    ([1], [5000], 4, 1, 128, 128, True),
    ([1, 1, 1, 1], [1, 16, 17, 0], 8, 8, 128, 16, True),
    ([1] * 9, [129, 128, 127, 64, 63, 65, 1000, 2, 0], 32, 8, 128, 64, True),
    ([4, 4, 4], [4, 700, 33], 4, 4, 64, 16, True),
    ([4, 2, 0, 8], [3, 1, 50, 0], 6, 2, 128, 32, True),      # rows that see no key
    ([7, 7], [129, 256], 7, 1, 128, 32, False),
    ([33], [33], 5, 1, 128, 16, True),
    ([100, 1, 17], [350, 1025, 17], 28, 4, 128, 32, True),
    ([129], [400], 4, 4, 64, 64, False),
    ([300, 2], [300, 900], 8, 8, 128, 128, True),
    ([255, 0, 257], [255, 0, 700], 3, 1, 64, 16, True),
    ([64], [64], 64, 1, 128, 16, True),
    ([150, 20], [149, 10], 2, 1, 128, 16, True),             # more queries than keys
    ([513], [1100], 12, 4, 64, 256, True),
]


@pytest.mark.parametrize("hint", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_paged_fwd(case, hint):
    new, lens, Hq, Hkv, d, page, causal = case
    s = paged_inputs(new, lens, Hq, Hkv, d, page, seed=len(new), heads_first=page == 32)
    ofa.device_error_flags()
    o, lse = run(s, causal, max_q=max(new) if hint else None)
    assert ofa.device_error_flags() == 0
    check_paged(o, lse, s, new, lens, causal, 1 / math.sqrt(d))
    o2, lse2 = run(s, causal, max_q=max(new) if hint else None)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


@pytest.mark.parametrize("seed", range(16))
def test_paged_fwd_random(seed):
    g = torch.Generator().manual_seed(100 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    B, Hkv, G = r(1, 7), r(1, 3), r(1, 9)
    d, page, causal = (64, 128)[r(0, 1)], (16, 32, 64, 128)[r(0, 3)], r(0, 4) > 0
    big = r(0, 2)
    new = [1 if big == 0 else r(0, (0, 12, 200)[big]) for _ in range(B)]
    lens = [r(0, (2000, 300, 600)[big]) for _ in range(B)]
    s = paged_inputs(new, lens, Hkv * G, Hkv, d, page, seed=seed, heads_first=bool(r(0, 1)))
    if sum(new) == 0:
        return
    o, lse = run(s, causal, max_q=r(0, 1) * max(new), scale=0.2)
    assert ofa.device_error_flags() == 0
    check_paged(o, lse, s, new, lens, causal, 0.2, f"seed {seed}")


def test_large_logits_and_growing_maxima():
    # each page's keys are larger than the last one's: the maximum moves at every tile
    new, lens = [3, 200], [900, 700]
    s = paged_inputs(new, lens, 4, 2, 128, 64, seed=5)
    for b in range(2):
        for j in range(-(-lens[b] // 64)):
            s["kp"][s["bt"][b, j].long()] *= 1 + j
    o, lse = run(s)
    check_paged(o, lse, s, new, lens, True, 1 / math.sqrt(128))


def test_rows_outside_the_sequences_stay():
    new, lens = [2, 30], [40, 50]
    s = paged_inputs(new, lens, 4, 2, 64, 16)
    o0, l0 = run(s, max_q=30)  # the same hint in both calls: the same kernel, so the same bits
    pad = torch.randn(5, 4, 64, device=DEV).bfloat16()
    q = torch.cat([pad, s["q"], pad])
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 5.0, device=DEV)
    ofa.attn_paged_fwd(q, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"] + 5, out=out, lse=lse,
                       max_q=30)
    assert torch.equal(out[5:-5], o0) and torch.equal(lse[5:-5], l0)
    for t in (out[:5], out[-5:]):
        assert bool((t == 3.0).all())
    assert bool((lse[:5] == 5.0).all()) and bool((lse[-5:] == 5.0).all())
    assert ofa.device_error_flags() == 0


def test_strided_queries_and_outputs_no_lse():
    new, lens = [1, 20], [100, 70]
    s = paged_inputs(new, lens, 6, 2, 128, 32)
    want, _ = run(s)
    wide = torch.zeros(21, 10, 2, 128, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 2:8, 1]
    q.copy_(s["q"])
    out = torch.zeros(6, 21, 256, dtype=torch.bfloat16, device=DEV).permute(1, 0, 2)[..., :128]
    ofa.attn_paged_fwd(q, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], out=out)
    assert torch.equal(out, want)


def test_uniform_batch_needs_no_cu():
    s = paged_inputs([3] * 4, [50, 3, 200, 1], 4, 2, 128, 16)
    a = run(s)
    b = ofa.attn_paged_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_pages_and_lengths_are_reported():
    s = paged_inputs([1, 1], [100, 40], 2, 1, 64, 16)
    want, _ = run(s)
    s["bt"][0, 3] = -7
    s["bt"][0, 4] = 1 << 30
    ofa.device_error_flags()
    o, _ = run(s)
    assert ofa.device_error_flags() == 4
    assert torch.equal(o[1], want[1])
    s = paged_inputs([1, 40], [112, 40], 2, 1, 64, 16, width=7)
    want, _ = run(s)
    s["lens"][0] = 5000  # the table holds 112
    o, _ = run(s)
    assert ofa.device_error_flags() == 2 and torch.equal(o, want)


@pytest.mark.parametrize("cu", [[0, 4, 2, 6], [0, 9, 9, 9], [-5, 2, 3, 6], [6, 4, 2, 0], [2, 3, 4, 5]])
def test_a_malformed_cu_faults_nothing(cu):
    s = paged_inputs([2, 2, 2], [20, 30, 17], 2, 1, 64, 16)
    for mq in (0, 2, 64):
        ofa.attn_paged_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"],
                           torch.tensor(cu, dtype=torch.int32, device=DEV), max_q=mq)
    torch.cuda.synchronize()
    ofa.device_error_flags()


def test_a_cache_past_two_gib_of_elements():
    # pages at offsets beyond 2^31 elements (and 2^32 bytes) in both caches
    page, Hkv, d = 128, 8, 128
    pages = (1 << 31) // (page * Hkv * d) + 40
    kp = torch.zeros(pages, page, Hkv, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    s = paged_inputs([1, 40], [900, 700], 16, 8, d, page, poison=False)
    n = s["kp"].shape[0]
    kp[-n:], vp[-n:] = s["kp"], s["vp"]
    a = run(s, max_q=40)
    bt = torch.where(s["bt"] < n, s["bt"] + (pages - n), s["bt"])
    b = ofa.attn_paged_fwd(s["q"], kp, vp, bt, s["lens"], s["cu"], max_q=40)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    k, v = (torch.randn(41, 8, d, device=DEV).bfloat16() for _ in range(2))
    ofa.attn_paged_append(s["q"], k, v, kp, vp, bt, s["lens"], s["cu"])
    assert torch.equal(kp[bt[0, 7].long(), 899 % 128], k[0]) and torch.equal(vp[bt[1, 5].long(), 699 % 128], v[40])


def step(s, k, v, w, cs):
    q = ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], wq=w, wk=w, cos_sin=cs)
    return ofa.attn_paged_fwd(q, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], max_q=1)


def test_prompt_in_chunks_then_tokens_equals_the_whole_at_once():
    """A prompt appended in chunks of many sizes and then token by token gives the rows that the
    prefill over the same normed and rotated tensors gives, and the cache it leaves holds them."""
    N, Hq, Hkv, d, page = 333, 8, 2, 128, 16
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, N, h, d, generator=g).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv))
    w = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16().to(DEV)
    cs = angles(N, d).to(DEV)
    q2, k2 = ofa.attn_qk_norm_rope(q, k, w, w, cs)
    rep = lambda t: t.repeat_interleave(Hq // Hkv, 2)  # noqa: E731
    want, wl = ofa.attn_fwd(q2, rep(k2), rep(v), causal=True)
    pages = -(-N // page)
    kp = torch.full((pages + 2, page, Hkv, d), math.nan, dtype=torch.bfloat16, device=DEV)
    vp = kp.clone()
    bt = torch.randperm(pages + 2, generator=g)[:pages].int().to(DEV)[None]
    at = 0
    for c in [100, 1, 64, 130, 5] + [1] * 33:
        sl = slice(at, at + c)
        at += c
        lens = torch.tensor([at], dtype=torch.int32, device=DEV)
        cu = torch.tensor([0, c], dtype=torch.int32, device=DEV)
        qr = ofa.attn_paged_append(q[0, sl], k[0, sl], v[0, sl], kp, vp, bt, lens, cu, wq=w, wk=w, cos_sin=cs)
        assert torch.equal(qr, q2[0, sl])
        o, lse = ofa.attn_paged_fwd(qr, kp, vp, bt, lens, cu, max_q=c)
        # both round weights and outputs to bf16: a step of 2^-8 each of values below 4
        assert float((o.float() - want[0, sl].float()).abs().max()) <= 4 * 2 * 2.0 ** -8
        assert float((lse - wl[0, :, sl].T).abs().max()) <= 1e-4
    assert at == N and ofa.device_error_flags() == 0
    assert torch.equal(kp[bt[0].long()].flatten(0, 1)[:N], k2[0])


def test_training_run_norm_rope_attention_and_back():
    """attn_qk_norm_rope -> attn_fwd -> attn_bwd -> attn_qk_norm_rope_bwd against the same chain in
    64 bits differentiated by torch, on the relative norm of each gradient."""
    B, N, H, d = 2, 130, 2, 64
    g = torch.Generator().manual_seed(4)
    q, k, v, do = (torch.randn(B, N, H, d, generator=g).bfloat16().to(DEV) for _ in range(4))
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).bfloat16().to(DEV) for _ in range(2))
    cs = angles(N, d).to(DEV)
    q2, k2 = ofa.attn_qk_norm_rope(q, k, wq, wk, cs)
    o, lse = ofa.attn_fwd(q2, k2, v, causal=True)
    dq2, dk2, dv = ofa.attn_bwd(q2, k2, v, o, lse, do, causal=True)
    dq, dk, dwq, dwk = ofa.attn_qk_norm_rope_bwd(q, k, dq2, dk2, wq, wk, cs)

    leaves = [t.cpu().double().requires_grad_() for t in (q, k, v, wq, wk)]
    c = cs.cpu().double()[None, :, None]

    def nr(x, w):
        t = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        a, b = t[..., :d // 2], t[..., d // 2:]
        co, si = c[..., :d // 2], c[..., d // 2:]
        return torch.cat([a * co - b * si, a * si + b * co], -1)

    Q, K = nr(leaves[0], leaves[3]), nr(leaves[1], leaves[4])
    X = torch.einsum("bihd,bjhd->bhij", Q, K) / math.sqrt(d)
    X = X.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -math.inf)
    O = torch.einsum("bhij,bjhd->bihd", X.softmax(-1), leaves[2])
    refs = torch.autograd.grad(O, leaves, do.cpu().double())
    # bf16 roundings on the way: q', k', o, the weights, dS, dq', dk', and the result: eight half
    # steps of 2^-8 that do not all point one way (their root sum of squares is 0.011)
    for got, ref, n in zip((dq, dk, dv, dwq, dwk), refs, "dq dk dv dwq dwk".split()):
        rel = float((got.cpu().double() - ref).norm() / ref.norm())
        assert rel <= 8 * 2.0 ** -8, (n, rel)


def test_captured_step_replays_with_new_values():
    new, lens = [1] * 5, [300, 20, 1, 64, 1000]
    s = paged_inputs(new, lens, 8, 2, 128, 16, seed=2, poison=False)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    cs = angles(1024, 128).to(DEV)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(5, 2, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(s, k, v, w, cs)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step(s, k, v, w, cs)
    for i in range(3):
        s["lens"].copy_(torch.tensor([300 - i, 20, 1 + i, 64, 1000], dtype=torch.int32))
        s["q"].copy_(torch.randn(s["q"].shape, generator=g).bfloat16())
        k.copy_(torch.randn(k.shape, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        a, b = o.clone(), lse.clone()
        eo, el = step(s, k, v, w, cs)
        assert torch.equal(a, eo) and torch.equal(b, el), i
    assert ofa.device_error_flags() == 0


def test_two_streams_at_once():
    jobs = []
    for i in range(4):
        new, lens = ([1] * 6, [500 + 100 * i] * 6) if i % 2 else ([90, 3], [400, 800])
        s = paged_inputs(new, lens, 8, 2, 128, 32, seed=i)
        jobs.append((s, run(s)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(5):
        for (s, _), st, into in zip(jobs, streams, got):
            into.append(run(s, stream=st))
    torch.cuda.synchronize()
    for (s, want), into in zip(jobs, got):
        for o, lse in into:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("new,lens,Hq,Hkv,d,page", [
    ([1], [200001], 2, 1, 64, 64),         # hundreds of shares of one row block: merged in two levels
    ([3, 1], [90000, 5], 4, 1, 128, 128),
    ([40], [60011], 2, 1, 64, 32),         # the same on the 128-row tiles
    ([5, 150], [40000, 30000], 7, 1, 128, 64),
])
def test_one_long_cache_over_the_whole_gpu(new, lens, Hq, Hkv, d, page):
    s = paged_inputs(new, lens, Hq, Hkv, d, page, seed=11)
    o, lse = run(s, max_q=max(new))
    check_paged(o, lse, s, new, lens, True, 1 / math.sqrt(d))
    o2, lse2 = run(s, max_q=max(new))
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and ofa.device_error_flags() == 0


def test_a_workspace_of_any_contents_shared_by_calls_of_many_shapes():
    """The counters are found in whatever state another call (or other data) left the workspace."""
    jobs = []
    for i, (new, lens) in enumerate([([1] * 3, [3000, 10, 500]), ([200], [900]), ([1], [20000]), ([33, 1], [5000, 4000])]):
        s = paged_inputs(new, lens, 4, 2, 64, 16, seed=i)
        jobs.append((s, max(new), run(s, max_q=max(new))))
    n = max(ofa.paged_fwd_workspace_bytes(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], max_q=mq) for s, mq, _ in jobs)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    for fill in range(3):
        ws.random_(0, 256, generator=g)
        for s, mq, (o, lse) in jobs + jobs[::-1]:
            a, b = run(s, max_q=mq, workspace=ws)
            assert torch.equal(a, o) and torch.equal(b, lse)
    assert ofa.device_error_flags() == 0


@pytest.mark.parametrize("new,lens,Hq,Hkv,d,page,mq", [
    ([1 + b % 3 for b in range(200)], [(37 * b) % 400 for b in range(200)], 4, 2, 64, 16, 3),     # many chunks of 32 sequences
    ([(b * 13) % 70 for b in range(130)], [(91 * b) % 500 for b in range(130)], 2, 1, 64, 32, 69),
    ([9, 40], [300, 41], 33, 1, 128, 16, 40),          # head groups that leave rows of a tile unused
    ([3, 100], [700, 120], 48, 1, 64, 64, 100),
    ([1, 70], [5000, 4100], 4, 2, 128, 4096, 70),      # pages longer than a tile
    ([1] * 3, [5000, 4096, 1], 4, 2, 128, 4096, 1),
])
def test_many_sequences_odd_groups_long_pages(new, lens, Hq, Hkv, d, page, mq):
    s = paged_inputs(new, lens, Hq, Hkv, d, page, seed=21)
    o, lse = run(s, max_q=mq)
    check_paged(o, lse, s, new, lens, True, 1 / math.sqrt(d))
    assert ofa.device_error_flags() == 0


@pytest.mark.parametrize("mq", [1, 64])
def test_no_pages_no_keys(mq):
    q = torch.randn(6, 4, 64, device=DEV).bfloat16()
    kp = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device=DEV)
    for bt in (torch.zeros(6, 3, dtype=torch.int32, device=DEV), torch.zeros(6, 0, dtype=torch.int32, device=DEV)):
        o, lse = ofa.attn_paged_fwd(q, kp, kp.clone(), bt, torch.zeros(6, dtype=torch.int32, device=DEV), max_q=mq)
        assert bool((o.view(torch.int16) == 0).all()) and bool((lse == -math.inf).all())
        assert ofa.device_error_flags() == 0


def test_captured_chunk_and_training_gradients_replay_beside_another_graph():
    """Two graphs over one workspace, replayed in turn with other lengths, and the gradients of the
    head norms in a graph while the eager call's tensors live."""
    s = paged_inputs([200, 40], [1500, 900], 8, 2, 128, 16, seed=2, poison=False)
    one = paged_inputs([1] * 3, [4000, 100, 900], 8, 2, 128, 16, seed=3, poison=False)
    n = max(ofa.paged_fwd_workspace_bytes(x["q"], x["kp"], x["vp"], x["bt"], x["lens"], x["cu"], max_q=m)
            for x, m in ((s, 200), (one, 1)))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    q, k = torch.randn(2, 33, 4, 128, device=DEV).bfloat16(), torch.randn(2, 33, 2, 128, device=DEV).bfloat16()
    w, cs = torch.rand(128, device=DEV).bfloat16(), angles(33, 128).to(DEV)
    eager = ofa.attn_qk_norm_rope_bwd(q, k, q * 2, k * 3, w, w, cs)
    calls = [lambda: run(s, max_q=200, workspace=ws), lambda: run(one, max_q=1, workspace=ws),
             lambda: ofa.attn_qk_norm_rope_bwd(q, k, q * 2, k * 3, w, w, cs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for lens in ([1500, 900], [200, 41], [777, 900]):
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        one["lens"].copy_(torch.tensor([lens[0], 1, lens[1]], dtype=torch.int32))
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        for c, o in zip(calls, got):
            for a, b in zip(c(), o):
                assert torch.equal(a, b)
    for a, b in zip(eager, outs[2]):
        assert torch.equal(a, b)
    assert ofa.device_error_flags() == 0


def test_a_stream_given_owns_what_the_call_allocates():
    s = paged_inputs([1] * 4, [900, 30, 2000, 1], 8, 2, 64, 16, seed=2)
    want = run(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = run(s, stream=st)
    k = torch.randn(4, 2, 64, device=DEV).bfloat16()
    st.wait_stream(torch.cuda.current_stream())
    q2 = ofa.attn_paged_append(s["q"], k, k, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(q2, s["q"])


@pytest.mark.parametrize("new,lens,Hq,Hkv,mq", [
    ([1] * 1500, [(37 * b) % 61 for b in range(1500)], 2, 2, 1),
    ([(b * 7) % 4 for b in range(1100)], [(29 * b) % 90 for b in range(1099)] + [9000], 4, 1, 3),
    ([(b * 7) % 3 for b in range(1089)] + [300], [(29 * b) % 50 for b in range(1089)] + [2000], 2, 2, 300),
])
def test_thousands_of_sequences(new, lens, Hq, Hkv, mq):
    # more than 32 x 32: the line's parts are found in two steps
    s = paged_inputs(new, lens, Hq, Hkv, 64, 16, seed=31)
    o, lse = run(s, max_q=mq)
    check_paged(o, lse, s, new, lens, True, 1 / math.sqrt(64))
    assert ofa.device_error_flags() == 0


def test_a_cu_that_goes_back_and_forth_past_every_length_is_reported():
    # every other sequence claims all tokens over 65536 keys: 2 heads x 512 sequences x 2048 blocks of
    # 1028 tiles, more than 2^31, though T tokens alone are far below it.  Nothing is computed.
    T, B, page = 1 << 15, 1024, 1024
    q = torch.randn(T, 2, 64, device=DEV).bfloat16()
    kp = torch.randn(64, page, 2, 64, device=DEV).bfloat16()
    bt = torch.arange(64, dtype=torch.int32, device=DEV).repeat(B, 1)
    lens = torch.full((B,), 64 * page, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32, device=DEV)
    out, lse = torch.full_like(q, 3.0), torch.full((T, 2), 5.0, device=DEV)
    ofa.device_error_flags()
    ofa.attn_paged_fwd(q, kp, kp, bt, lens, cu, max_q=1, causal=False, out=out, lse=lse)
    assert ofa.device_error_flags() == 4
    assert bool((out == 3.0).all()) and bool((lse == 5.0).all())


@pytest.mark.parametrize("Hq,Hkv,d,page", [(1, 1, 128, 16), (10, 2, 64, 64), (16, 2, 128, 32), (33, 1, 64, 16), (64, 1, 128, 128)])
def test_every_hint_takes_a_kernel_that_is_right(Hq, Hkv, d, page):
    # blocks of 16 rows, one tile of 64 or 128 rows, two tiles, whatever the tokens; items cut or whole
    new, lens = [3, 70, 1, 0, 9, 2], [900, 2500, 6000, 3, 9, 0]
    s = paged_inputs(new, lens, Hq, Hkv, d, page, seed=41)
    G = Hq // Hkv
    for rows in (1, 17, 40, 64, 65, 100, 128, 129, 1000):
        if rows * 2 <= G:
            continue
        for causal in (True, False):
            o, lse = run(s, causal, max_q=-(-rows // G))
            check_paged(o, lse, s, new, lens, causal, 1 / math.sqrt(d), f"{rows} rows, causal {causal}")
    assert ofa.device_error_flags() == 0


@pytest.mark.parametrize("mq", [1, 8, 16, 40])
def test_a_hidden_key_or_value_of_any_content_reaches_no_row(mq):
    # NaN and infinities past the lengths, inside the last page and in pages of other sequences' tails, and
    # the type's lowest value in keys that are seen: rows stay finite, hidden ones do not count
    new, lens = [1, 8, 40], [33, 65, 140]
    s = paged_inputs(new, lens, 8, 1, 128, 64, seed=43)
    want = run(s, max_q=mq)
    bad = torch.isnan(s["kp"])
    for fill in (math.inf, -math.inf, torch.finfo(torch.bfloat16).min):
        s["kp"][bad] = fill
        s["vp"][bad] = fill
        got = run(s, max_q=mq)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_paged(*want, s, new, lens, True, 1 / math.sqrt(128))


def test_a_chunk_kernel_captured_with_one_tile_replays_over_a_shared_workspace():
    a = paged_inputs([8, 3, 5], [3000, 200, 900], 16, 2, 128, 16, seed=51, poison=False)
    b = paged_inputs([16], [20000], 8, 1, 64, 32, seed=52, poison=False)
    n = max(ofa.paged_fwd_workspace_bytes(x["q"], x["kp"], x["vp"], x["bt"], x["lens"], x["cu"], max_q=m)
            for x, m in ((a, 8), (b, 16)))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    calls = [lambda: run(a, max_q=8, workspace=ws), lambda: run(b, max_q=16, workspace=ws)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c())
        graphs.append(g)
    for la, lb in (([3000, 200, 900], 20000), ([9, 200, 1], 17), ([2999, 0, 640], 12345)):
        a["lens"].copy_(torch.tensor(la, dtype=torch.int32))
        b["lens"].fill_(lb)
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        for c, o in zip(calls, got):
            for x, y in zip(c(), o):
                assert torch.equal(x, y)
    assert ofa.device_error_flags() == 0


def test_tile_kernels_of_both_kinds_beside_each_other_and_a_prefill():
    # one-tile blocks (two CTAs an SM, half the tensor memory each), two-tile blocks and attn_fwd on
    # three streams at once
    a = paged_inputs([8, 5, 8], [3000, 700, 2000], 16, 2, 64, 16, seed=61, poison=False)
    b = paged_inputs([200, 60], [1500, 2900], 8, 2, 128, 32, seed=62, poison=False)
    q = torch.randn(2, 1024, 8, 128, device=DEV).bfloat16()
    jobs = [lambda: run(a, max_q=8), lambda: run(b, max_q=200), lambda: ofa.attn_fwd(q, q, q, causal=True)]
    want = [j() for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for st, j, g in zip(streams, jobs, got):
            with torch.cuda.stream(st):
                g.append(j())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x in g:
            assert torch.equal(x[0], w[0]) and torch.equal(x[1], w[1])
    assert ofa.device_error_flags() == 0


@pytest.mark.parametrize("cu,ok", [([0, 4, 2, 6], False), ([0, 9, 9, 9], False), ([-5, 2, 3, 6], False), ([6, 4, 2, 0], False),
                                   ([0, 2, 4, 7], False), ([2, 3, 4, 5], True)])
def test_a_malformed_cu_is_reported_and_clamped(cu, ok):
    lens, T = [20, 30, 17], 6
    s = paged_inputs([2, 2, 2], lens, 2, 1, 64, 16)
    c = [min(max(x, 0), T) for x in cu]
    claims = [(b, t) for b in range(3) for t in range(c[b], max(c[b + 1], c[b]))]
    for mq in (0, 2, 64):
        out, lse = torch.full_like(s["q"], 3.0), torch.full((T, 2), 5.0, device=DEV)
        ofa.device_error_flags()
        ofa.attn_paged_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], torch.tensor(cu, dtype=torch.int32, device=DEV),
                           max_q=mq, out=out, lse=lse)
        assert ofa.device_error_flags() == (0 if ok else 4)
        for t in range(T):
            of = [b for b, u in claims if u == t]
            if not of:
                assert bool((out[t] == 3.0).all()) and bool((lse[t] == 5.0).all())
            if len(of) == 1:  # the row of a batch of that sequence's clamped tokens alone
                b = of[0]
                sub = dict(s, q=s["q"][c[b]:c[b + 1]], bt=s["bt"][b:b + 1], lens=s["lens"][b:b + 1],
                           cu=torch.tensor([0, c[b + 1] - c[b]], dtype=torch.int32, device=DEV))
                o1, l1 = run(sub, max_q=mq)
                check_paged(o1, l1, sub, [c[b + 1] - c[b]], [lens[b]], True, 1 / 8)
                assert torch.equal(out[t], o1[t - c[b]]) and torch.equal(lse[t], l1[t - c[b]])


@pytest.mark.parametrize("mq", [1, 12, 30, 150])  # the warp-level kernel, one tile of 64 or 128 rows, two tiles
@pytest.mark.parametrize("d,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_a_nan_reaches_the_rows_that_see_it_and_no_others(mq, d, page, causal):
    # sequences whose blocks are cut into parts (9000 keys) and one whose block is whole (100)
    new, lens, Hq, Hkv = [2, 150, 1, 3], [700, 900, 9000, 100], 8, 2
    G, starts = Hq // Hkv, [0, 2, 152, 153]
    s = paged_inputs(new, lens, Hq, Hkv, d, page, seed=71)
    for j in range(-(-100 // page)):
        s["kp"][s["bt"][3, j].long(), :, 0, 0] = 1.0  # (sequence 3, key head 0: -inf logits for a query that starts with -inf)
    clean = run(s, causal, max_q=mq)
    check_paged(*clean, s, new, lens, causal, 1 / math.sqrt(d))
    nan = torch.zeros(sum(new), Hq, dtype=torch.bool)
    q, kp = s["q"].clone(), s["kp"].clone()
    for t, h, at, v in ((1, 3, 5, math.nan), (60, 7, 0, math.nan), (100, 2, d - 1, math.inf), (152, 6, 17, math.nan),
                        (154, 4, 3, math.nan)):
        q[t, h, at] = v
        nan[t, h] = True
    for b, j, hk, v in ((0, 333, 0, math.nan), (1, 820, 1, math.nan), (2, 8999, 0, math.inf), (3, 98, 1, -math.inf),
                        (3, 99, 1, math.nan)):
        kp[s["bt"][b, j // page].long(), j % page, hk, 9] = v
        for i in range(new[b]):
            if not causal or j <= i + lens[b] - new[b]:
                rows = slice(hk * G, (hk + 1) * G)
                if v == v:  # an infinite key: logits of +inf where the query's element has its sign
                    nan[starts[b] + i, rows] |= (q[starts[b] + i, rows, 9].cpu() * v) > 0
                else:
                    nan[starts[b] + i, rows] = True
    q[153, 1, 0] = -math.inf
    for kind in ("queries", "keys", "both"):
        x = dict(s, q=s["q"] if kind == "keys" else q, kp=s["kp"] if kind == "queries" else kp)
        o, lse = run(x, causal, max_q=mq)
        assert ofa.device_error_flags() == 0
        if kind == "both":
            hit = torch.isnan(lse).cpu()
            assert torch.equal(hit, nan) and torch.equal(torch.isnan(o).all(-1).cpu(), nan)
            assert torch.equal(torch.isnan(o).any(-1).cpu(), nan)
            assert bool((o[153, 1].view(torch.int16) == 0).all()) and float(lse[153, 1]) == -math.inf
        else:
            hit = torch.isnan(lse).cpu()
            assert bool(hit.any()) and not bool((hit & ~nan).any()) and torch.equal(hit, torch.isnan(o).any(-1).cpu())
        same = ~nan.clone()
        same[153, 1] = False
        if kind != "queries":
            # an infinite key whose logit is -inf leaves a row with one key less
            for b, j, hk in ((2, 8999, 0), (3, 98, 1)):
                for i in range(new[b]):
                    same[starts[b] + i, hk * G:(hk + 1) * G] = False
        assert torch.equal(o.cpu()[same], clean[0].cpu()[same]) and torch.equal(lse.cpu()[same], clean[1].cpu()[same])


@pytest.mark.parametrize("nq", [1, 20])  # the warp-level kernel and the tiles
def test_the_longest_table(nq):
    # 2^31 - 261 keys in a table of 2^31 - 256: 8 pages of 256 keys, each a million times
    d, page, width, pages = 64, 256, (1 << 23) - 1, 8
    n = width * page - 5
    g = torch.Generator().manual_seed(81)
    q = torch.randn(nq, 1, d, generator=g).bfloat16()
    kp, vp = (torch.randn(pages, page, 1, d, generator=g).bfloat16() for _ in range(2))
    vp += 2.0  # (outputs near 2, so that a relative bound says something)
    bt = torch.arange(width, dtype=torch.int32) % pages
    count = bt.bincount(minlength=pages).double()[:, None].expand(pages, page).clone()
    count[bt[-1], -5:] -= 1
    o, lse = ofa.attn_paged_fwd(q.to(DEV), kp.to(DEV), vp.to(DEV), bt[None].to(DEV),
                                torch.tensor([n], dtype=torch.int32, device=DEV), causal=False)
    assert ofa.device_error_flags() == 0
    X = q[:, 0].double() @ kp.reshape(-1, d).double().T / 8 + count.reshape(-1).log()
    L = torch.logsumexp(X, -1)
    V = vp.reshape(-1, d).double()
    P = torch.exp(X - L[:, None])
    # A CTA's share is at most 2^31 / 152 keys, in tiles of 64 or 128: its row sums are chains of as many
    # fp32 additions of half a step of 2^-24 as it has tiles (and 20 in a tile), its accumulator's of one
    # a 16 keys, which a tensor core may cut off instead of rounding (a whole step, 2^-23).
    tiles, steps = 2 ** 31 / 152 / 64 + 20, 2 ** 31 / 152 / 16
    assert float((lse[:, 0].cpu().double() - L).abs().max()) <= tiles * 2.0 ** -24 + 2.0 ** -18 * (1 + float(L.max()))
    err = (o[:, 0].cpu().double() - P @ V).abs()
    assert bool((err <= (2 * 2.0 ** -8 + tiles * 2.0 ** -24 + steps * 2.0 ** -23) * (P @ V.abs())).all())


@pytest.mark.parametrize("mq", [1, 12, 30, 150])
def test_without_lse_the_outputs_are_the_same(mq):
    # the C entry takes a null lse: whole items, cut ones and rows that see no key
    new, lens = [2, 150, 1, 3], [700, 900, 9000, 2]
    s = paged_inputs(new, lens, 8, 2, 128, 16, seed=91)
    want, _ = run(s, max_q=mq)
    o = torch.full_like(want, 7.0)
    p = paged._paged_fwd_params(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], mq, True, None, o, None)
    n = ofa.paged_fwd_workspace_bytes(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], max_q=mq)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert paged._load().attn_paged_fwd(p, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(o, want) and ofa.device_error_flags() == 0

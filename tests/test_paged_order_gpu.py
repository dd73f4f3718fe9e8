"""Attention behind prefixes that begins beside the work queued before it: steps without a pause give what steps with one
between them give, whatever that work writes (tokens, lengths, tables, cuts, keys)."""
import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_q8_helpers import E4M3, E8M0

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("new", [[1] * 40, [4, 1] * 10, [60, 1, 130, 33], [200, 250]])
def test_steps_back_to_back(new, q8):
    """Decode steps, drafted tokens, chunks of one tile and of two; every step overwrites the tensors of the last one."""
    Hq, Hkv, d, page, P, B, steps = 8, 2, 128, 16, 700, len(new), 5
    g = torch.Generator().manual_seed(11)
    rnd = lambda *x: torch.randn(*x, generator=g).bfloat16().to(DEV)  # noqa: E731
    T, width, ppages = sum(new), -(-max(new) * steps // page), -(-P // page)
    pages = ppages + 2 * B * width
    perm = torch.randperm(pages, generator=g).int()
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pt = i32(perm[:ppages][None])
    tables = [i32(perm[ppages + k * B * width:ppages + (k + 1) * B * width].view(B, width)) for k in (0, 1)]
    order = [torch.randperm(B, generator=g).tolist() for _ in range(steps)]
    if q8:
        base = [torch.randint(0, 0x7E, (pages, page, Hkv, d), generator=g, dtype=torch.uint8).to(DEV).view(E4M3) for _ in "kv"]
        base += [torch.randint(116, 122, (pages, Hkv, page), generator=g, dtype=torch.uint8).to(DEV).view(E8M0) for _ in "kv"]
    else:
        base = [rnd(pages, page, Hkv, d) for _ in "kv"]
    data = []
    for k in range(steps):
        n = [new[j] for j in order[k]]
        data.append(dict(q=rnd(T, Hq, d), k=rnd(T, Hkv, d), v=rnd(T, Hkv, d), bt=tables[k % 2], plens=i32([P - 40 * k]),
                         lens=i32([x + 3 * k if x < 8 else x for x in n]), cu=i32([0] + torch.tensor(n).cumsum(0).tolist()),
                         pcu=i32([k, T - k])))

    def go(sync):
        cache = [t.clone() for t in base]
        live = {n: torch.zeros_like(t) for n, t in data[0].items()}
        ws, got = None, []
        append = ofa.attn_paged_append_q8 if q8 else ofa.attn_paged_append
        for s in data:
            for n, t in s.items():
                live[n].copy_(t)
            q = append(live["q"], live["k"], live["v"], *cache, live["bt"], live["lens"], live["cu"])
            a = (q, *cache[:2], live["bt"], live["lens"], pt, live["plens"], live["cu"], live["pcu"])
            kw = dict(k_scales=cache[2], v_scales=cache[3]) if q8 else {}
            if ws is None:
                ws = torch.randint(0, 256, (ofa.paged_prefix_fwd_workspace_bytes(*a, max(new), **kw),), dtype=torch.uint8, device=DEV)
            got.append(ofa.attn_paged_prefix_fwd(*a, max_q=max(new), workspace=ws, **kw))
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got

    ofa.device_error_flags()
    want = go(True)
    for _ in range(4):
        for (o, lse), (wo, wl) in zip(go(False), want):
            assert torch.equal(o.view(torch.int16), wo.view(torch.int16)) and torch.equal(lse.view(torch.int32), wl.view(torch.int32))
    assert ofa.device_error_flags() == 0


@pytest.mark.parametrize("q8", [False, True])
def test_one_graph_replayed_over_a_workspace_that_keeps_its_words(q8):
    """A captured append and attention, replayed without a pause and without anything between that touches the workspace:
    each replay's tag is the last one's, and is not found before the replay's own first attention has begun."""
    Hq, Hkv, d, page, P, B = 8, 2, 128, 16, 700, 40
    g = torch.Generator().manual_seed(12)
    rnd = lambda *x: torch.randn(*x, generator=g).bfloat16().to(DEV)  # noqa: E731
    ppages = -(-P // page)
    perm = torch.randperm(ppages + B, generator=g).int().to(DEV)
    pt, bt = perm[:ppages][None], perm[ppages:].view(B, 1)
    plens = torch.tensor([P], dtype=torch.int32, device=DEV)
    if q8:
        cache = [torch.randint(0, 0x7E, (ppages + B, page, Hkv, d), generator=g, dtype=torch.uint8).to(DEV).view(E4M3) for _ in "kv"]
        cache += [torch.randint(116, 122, (ppages + B, Hkv, page), generator=g, dtype=torch.uint8).to(DEV).view(E8M0) for _ in "kv"]
    else:
        cache = [rnd(ppages + B, page, Hkv, d) for _ in "kv"]
    kw = dict(k_scales=cache[2], v_scales=cache[3]) if q8 else {}
    steps = 8
    toks = rnd(steps, B, Hq + 2 * Hkv, d)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    outs = torch.zeros(steps, B, Hq, d, dtype=torch.bfloat16, device=DEV)
    now = torch.zeros(B, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    out = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device=DEV)
    append = ofa.attn_paged_append_q8 if q8 else ofa.attn_paged_append

    def step():
        lens.add_(1)
        q = append(now[:, :Hq], now[:, Hq:Hq + Hkv], now[:, Hq + Hkv:], *cache, bt, lens)
        ofa.attn_paged_prefix_fwd(q, *cache[:2], bt, lens, pt, plens, workspace=ws, out=out, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def go(sync):
        lens.zero_()
        for i in range(steps):
            now.copy_(toks[i])
            graph.replay()
            outs[i].copy_(out)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs.clone()

    want = go(True)
    for _ in range(4):
        assert torch.equal(go(False), want)
    assert ofa.device_error_flags() == 0

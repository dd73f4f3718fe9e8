"""Head norms with rotation, their gradients, and the append to a paged cache against a plain form
in 64 bits (paged_helpers), within bounds that count the roundings."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_helpers import U, angles, check, norm_rope, norm_rope_bwd, paged_inputs, pair_index

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def draw(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def table_for(cs, pos):
    """cs rows of positions [B, N] broadcast over heads, on the CPU."""
    return cs.cpu()[pos.cpu().long()][:, :, None, :]


CASES = [  # B, N, Hq, Hkv, d, rot, inter, weights
    (1, 1, 1, 1, 64, 64, False, "qk"),
    (2, 37, 3, 1, 64, 32, True, "qk"),
    (1, 5, 7, 7, 16, 16, False, "qk"),
    (3, 129, 16, 4, 128, 128, False, "qk"),
    (2, 65, 5, 5, 128, 64, True, "q"),
    (1, 300, 8, 2, 192, 192, False, "k"),
    (2, 33, 40, 8, 256, 128, True, "qk"),
    (1, 17, 2, 1, 112, 48, False, "qk"),
    (2, 9, 4, 4, 128, 0, False, "qk"),
    (4, 8, 6, 3, 96, 96, True, ""),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_norm_rope_and_its_gradients(case, dtype):
    B, N, Hq, Hkv, d, rot, inter, weights = case
    q, k = draw(1, B, N, Hq, d, dtype=dtype), draw(2, B, N, Hkv, d, dtype=dtype, scale=3.0)
    q[0, 0, 0] = 0  # a row of zeros: the norm leaves it zero
    wq = (1 + 0.3 * draw(3, d, dtype=torch.float32)).to(dtype) if "q" in weights else None
    wk = (1 + 0.3 * draw(4, d, dtype=torch.float32)).to(dtype) if "k" in weights else None
    cs = angles(N, rot).to(DEV) if rot else None
    q2, k2 = ofa.attn_qk_norm_rope(q, k, wq, wk, cs, eps=EPS, interleaved=inter)
    tab = table_for(cs, torch.arange(N).expand(B, N)) if rot else None
    for x, y, w, n in ((q, q2, wq, "q"), (k, k2, wk, "k")):
        ref, lim = norm_rope(x.cpu(), None if w is None else w.cpu(), tab, inter, EPS)
        check(y, ref, lim, n)
    dq2, dk2 = draw(5, B, N, Hq, d, dtype=dtype), draw(6, B, N, Hkv, d, dtype=dtype)
    dq, dk, dwq, dwk = ofa.attn_qk_norm_rope_bwd(q, k, dq2, dk2, wq, wk, cs, eps=EPS, interleaved=inter)
    for x, dy, w, dx, dw, H, n in ((q, dq2, wq, dq, dwq, Hq, "dq"), (k, dk2, wk, dk, dwk, Hkv, "dk")):
        rx, rw, lim, size = norm_rope_bwd(x.cpu(), dy.cpu(), None if w is None else w.cpu(), tab, inter, EPS)
        check(dx, rx, lim, n)
        if w is None:
            assert dw is None
        else:  # terms good to 32 U, summed in chains of at most 64 + rows / 32
            check(dw, rw, (96 + B * N * H / 32) * U * size, n + " weight")
    again = ofa.attn_qk_norm_rope_bwd(q, k, dq2, dk2, wq, wk, cs, eps=EPS, interleaved=inter)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert (a is None) == (b is None) and (a is None or torch.equal(a, b))
    assert ofa.device_error_flags() == 0


def test_long_rows_sum_in_a_fixed_order_and_match():
    B, N, Hq, Hkv, d = 2, 4099, 6, 2, 64
    q, k = draw(1, B, N, Hq, d), draw(2, B, N, Hkv, d)
    dq2, dk2 = draw(5, B, N, Hq, d), draw(6, B, N, Hkv, d)
    w = (1 + 0.3 * draw(3, d, dtype=torch.float32)).bfloat16()
    cs = angles(N, d).to(DEV)
    dq, dk, dwq, dwk = ofa.attn_qk_norm_rope_bwd(q, k, dq2, dk2, w, w, cs, eps=EPS)
    tab = table_for(cs, torch.arange(N).expand(B, N))
    for x, dy, dx, dw, H in ((q, dq2, dq, dwq, Hq), (k, dk2, dk, dwk, Hkv)):
        rx, rw, lim, size = norm_rope_bwd(x.cpu(), dy.cpu(), w.cpu(), tab, False, EPS)
        check(dx, rx, lim, "dx")
        check(dw, rw, (96 + B * N * H / 32) * U * size, "dw")


def test_positions_strides_and_in_place():
    B, N, Hq, Hkv, d, P = 2, 50, 4, 2, 128, 5000
    big = draw(1, B, N, 3, Hq + Hkv, d)  # q and k as slices of one projection
    q, k = big[:, :, 1, :Hq], big[:, :, 1, Hq:]
    w = (1 + 0.3 * draw(3, d, dtype=torch.float32)).bfloat16()
    cs_wide = torch.zeros(P, d + 4, device=DEV)
    cs_wide[:, :d] = angles(P, d).to(DEV)
    cs = cs_wide[:, :d]
    pos = torch.randint(0, P, (N, B), generator=torch.Generator().manual_seed(9)).int().to(DEV).T  # strided
    ref_q, lim_q = norm_rope(q.cpu(), w.cpu(), table_for(cs, pos), False, EPS)
    ref_k, lim_k = norm_rope(k.cpu(), None, table_for(cs, pos), False, EPS)
    rest = big.clone()
    q2, k2 = ofa.attn_qk_norm_rope(q, k, w, None, cs, positions=pos, eps=EPS, q_out=q, k_out=k)
    assert q2.data_ptr() == q.data_ptr()
    check(q2, ref_q, lim_q, "q")
    check(k2, ref_k, lim_k, "k")
    assert torch.equal(big[:, :, 0], rest[:, :, 0]) and torch.equal(big[:, :, 2], rest[:, :, 2])
    one = torch.tensor([4999], dtype=torch.int32, device=DEV)  # broadcast position
    a, _ = ofa.attn_qk_norm_rope(q.contiguous(), k.contiguous(), None, None, cs, positions=one[:, None])
    ref, lim = norm_rope(q.contiguous().cpu(), None, table_for(cs, one.expand(B, N)), False, EPS)
    check(a, ref, lim, "broadcast position")
    # gradients written over the incoming ones
    g = draw(7, B, N, Hq, d)
    gk = draw(8, B, N, Hkv, d)
    want = ofa.attn_qk_norm_rope_bwd(q, k, g, gk, w, None, cs, positions=pos)
    got = ofa.attn_qk_norm_rope_bwd(q, k, g, gk, w, None, cs, positions=pos, dq=g, dk=gk)
    assert all((x is None and y is None) or torch.equal(x, y) for x, y in zip(want, got))
    assert ofa.device_error_flags() == 0


def test_a_position_outside_the_table_is_clamped_and_reported():
    q, k = draw(1, 1, 3, 2, 64), draw(2, 1, 3, 2, 64)
    cs = angles(4, 64).to(DEV)
    ofa.device_error_flags()
    pos = torch.tensor([[0, 7, -2]], dtype=torch.int32, device=DEV)
    a, _ = ofa.attn_qk_norm_rope(q, k, None, None, cs, positions=pos)
    assert ofa.device_error_flags() == 4
    b, _ = ofa.attn_qk_norm_rope(q, k, None, None, cs, positions=pos.clamp(0, 3))
    assert torch.equal(a, b) and ofa.device_error_flags() == 0


def test_empty_batch():
    q, k = draw(1, 0, 5, 2, 64), draw(2, 0, 5, 2, 64)
    w = draw(3, 64)
    cs = angles(8, 64).to(DEV)
    q2, k2 = ofa.attn_qk_norm_rope(q, k, w, w, cs)
    assert q2.shape == q.shape and k2.shape == k.shape
    dq, dk, dwq, dwk = ofa.attn_qk_norm_rope_bwd(q, k, q, k, w, w, cs)
    assert float(dwq.abs().sum()) == 0 and float(dwk.abs().sum()) == 0


APPEND = [  # new, lens, Hq, Hkv, d, rot, page, inter
    ([1], [1], 1, 1, 64, 64, 16, False),
    ([1, 1, 1], [300, 17, 16], 8, 2, 128, 128, 16, False),
    ([5, 0, 40, 1], [5, 9, 64, 33], 6, 3, 64, 32, 32, True),
    ([100, 3], [260, 3], 4, 4, 256, 256, 7, False),
    ([2, 1, 1], [0, 0, 5], 4, 2, 128, 64, 64, True),   # places without a sequence
    ([3] * 70, [3 + b for b in range(70)], 2, 1, 64, 64, 16, False),
    ([1] * 1500, [1 + b % 9 for b in range(1500)], 2, 1, 64, 64, 16, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", APPEND)
def test_append(case, dtype):
    new, lens, Hq, Hkv, d, rot, page, inter = case
    s = paged_inputs(new, lens, Hq, Hkv, d, page, dtype=dtype, heads_first=d == 64)
    T = sum(new)
    q, k, v = s["q"], draw(2, T, Hkv, d, dtype=dtype), draw(3, T, Hkv, d, dtype=dtype)
    wq = (1 + 0.3 * draw(4, d, dtype=torch.float32)).to(dtype)
    cs = angles(max(lens) + 1, rot).to(DEV)
    kp0, vp0 = s["kp"].clone(), s["vp"].clone()
    tail = 3  # rows behind the last sequence
    qpad = torch.cat([q, draw(8, tail, Hq, d, dtype=dtype)])
    kpad, vpad = (torch.cat([t, draw(9, tail, Hkv, d, dtype=dtype)]) for t in (k, v))
    out = torch.full_like(qpad, 7.0)
    ofa.device_error_flags()
    got = ofa.attn_paged_append(qpad, kpad, vpad, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], wq=wq, wk=None,
                                cos_sin=cs, eps=EPS, interleaved=inter, q_out=out)
    assert got is out and ofa.device_error_flags() == 0
    assert bool((out[T:] == 7.0).all())
    at = torch.cat([torch.arange(n - m, n) for m, n in zip(new, lens)]) if T else torch.zeros(0)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    tab = cs.cpu()[at.clamp(min=0).long()][:, None, :]
    ref, lim = norm_rope(q.cpu(), wq.cpu(), tab, inter, EPS)
    check(out[:T], ref, lim, "q")
    rk, lk = norm_rope(k.cpu(), None, tab, inter, EPS)
    kp, vp, bt = s["kp"].cpu(), s["vp"].cpu(), s["bt"].cpu()
    has = at >= 0
    pg = bt[seq[has], at[has].long() // page].long()
    sl = at[has].long() % page
    check(kp[pg, sl], rk[has], lk[has], "k pages")
    assert torch.equal(vp[pg, sl], v.cpu()[has])
    # nothing else was touched
    ek, ev = kp0.cpu(), vp0.cpu()
    ek[pg, sl], ev[pg, sl] = kp[pg, sl], vp[pg, sl]
    assert torch.equal(ek.nan_to_num(9e9), kp.nan_to_num(9e9)) and torch.equal(ev.nan_to_num(9e9), vp.nan_to_num(9e9))


def test_append_uniform_positions_and_plain_copy():
    new, lens = [4, 4, 4], [10, 4, 40]
    s = paged_inputs(new, lens, 4, 2, 128, 16)
    k, v = draw(2, 12, 2, 128), draw(3, 12, 2, 128)
    pos = torch.arange(12, dtype=torch.int32, device=DEV) * 3
    cs = angles(64, 128).to(DEV)
    a = ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], cos_sin=cs, positions=pos)
    kp, vp = s["kp"].clone(), s["vp"].clone()
    b = ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], cos_sin=cs, positions=pos)
    assert torch.equal(a, b) and torch.equal(kp.nan_to_num(9e9), s["kp"].nan_to_num(9e9))
    ref, lim = norm_rope(s["q"].cpu(), None, cs.cpu()[pos.cpu().long()][:, None], False, EPS)
    check(a, ref, lim, "q")
    # neither norms nor angles: keys and queries go as they are
    c = ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"])
    assert torch.equal(c, s["q"])
    assert torch.equal(s["kp"][s["bt"][1, 0].long(), :4], k[4:8])


def test_append_reports_bad_pages_and_lengths():
    new, lens = [1, 1], [20, 20]
    s = paged_inputs(new, lens, 2, 1, 64, 16)
    k, v = draw(2, 2, 1, 64), draw(3, 2, 1, 64)
    kp0, vp0 = s["kp"].clone(), s["vp"].clone()
    s["bt"][0, 1] = s["kp"].shape[0]  # sequence 0's last page does not exist
    ofa.device_error_flags()
    ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"])
    assert ofa.device_error_flags() == 4
    changed = (s["kp"].nan_to_num(9e9) != kp0.nan_to_num(9e9)).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(s["bt"][1, 1])]
    s["bt"][0, 1] = -1
    s["lens"][1] = 1000  # more than the table holds: clamped to its last slot
    ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"])
    assert ofa.device_error_flags() == 6
    assert torch.equal(s["kp"][s["bt"][1, 1].long(), 15], k[1])


@pytest.mark.parametrize("cu", [[0, 4, 2, 6], [0, 9, 9, 9], [-5, 2, 3, 6], [6, 4, 2, 0], [2, 3, 4, 5]])
def test_append_survives_a_malformed_cu(cu):
    s = paged_inputs([2, 2, 2], [20, 30, 17], 2, 1, 64, 16)
    k, v = draw(2, 6, 1, 64), draw(3, 6, 1, 64)
    ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], torch.tensor(cu, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    ofa.device_error_flags()


@pytest.mark.parametrize("cu,places", [  # places: (sequence, token, place) of the tokens that one sequence has
    ([0, 9, 9, 9], [(0, t, 14 + t) for t in range(6)]),
    ([-5, 2, 3, 6], [(0, 0, 18), (0, 1, 19), (1, 2, 29), (2, 3, 14), (2, 4, 15), (2, 5, 16)]),
    ([0, 4, 2, 6], [(0, 0, 16), (0, 1, 17), (2, 4, 15), (2, 5, 16)]),
    ([6, 4, 2, 0], []),
    ([3, 1, 6, 6], [(1, t, 24 + t) for t in range(1, 6)]),
    ([0, 2, 4, 7], [(0, 0, 18), (0, 1, 19), (1, 2, 28), (1, 3, 29), (2, 4, 15), (2, 5, 16)]),
    ([2, 3, 4, 5], [(0, 2, 19), (1, 3, 29), (2, 4, 16)]),
])
def test_append_places_tokens_of_a_malformed_cu_as_the_attention_does_and_reports_it(cu, places):
    T, lens = 6, [20, 30, 17]
    s = paged_inputs([2, 2, 2], lens, 2, 1, 64, 16, poison=False)
    k, v = draw(2, T, 1, 64), draw(3, T, 1, 64)
    kp, vp, bt = s["kp"].clone(), s["vp"].clone(), s["bt"].cpu()
    for b, t, at in places:
        kp[bt[b, at // 16], at % 16], vp[bt[b, at // 16], at % 16] = k[t], v[t]
    out = torch.full_like(s["q"], 7.0)
    ofa.device_error_flags()
    ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"],
                          torch.tensor(cu, dtype=torch.int32, device=DEV), q_out=out)
    assert ofa.device_error_flags() == (0 if cu == [2, 3, 4, 5] else 4)
    # what the attention's sequences (c0 = cu[b], c1 = max(cu[b + 1], c0), in [0, T]) do not hold stays
    c = [min(max(x, 0), T) for x in cu]
    owned, claimed = set(), set()
    for b in range(3):
        nq = max(c[b + 1], c[b]) - c[b]
        claimed |= set(range(c[b], c[b] + nq))
        owned |= {(int(bt[b, p // 16]), p % 16) for p in range(max(lens[b] - nq, 0), lens[b])}
    sure = {(int(bt[b, at // 16]), at % 16) for b, _, at in places}
    for page in range(kp.shape[0]):
        for slot in range(16):
            if (page, slot) in sure or (page, slot) not in owned:
                assert torch.equal(s["kp"][page, slot], kp[page, slot]) and torch.equal(s["vp"][page, slot], vp[page, slot])
    for _, t, _ in places:
        assert torch.equal(out[t], s["q"][t])
    for t in range(T):
        if t not in claimed:
            assert bool((out[t] == 7.0).all())


@pytest.mark.parametrize("B,at", [(3, 1), (40, 39), (5000, 4097)])
def test_append_reports_a_bad_cu_entry_wherever_it_stands(B, at):
    # one token in the first sequence, the others empty; one entry behind it out of range, negative or falling back
    s = paged_inputs([1], [5], 2, 1, 64, 16, poison=False)
    k = draw(2, 1, 1, 64)
    bt, lens = s["bt"].repeat(B, 1), s["lens"].repeat(B)
    cu = torch.ones(B + 1, dtype=torch.int32)
    cu[0] = 0
    for bad in (None, 2, -1, 0, 2 ** 31 - 1, -2 ** 31):
        c = cu.clone()
        if bad is not None:
            c[at + 1] = bad
        ofa.attn_paged_append(s["q"], k, k, s["kp"], s["vp"], bt, lens, c.to(DEV))
        assert ofa.device_error_flags() == (0 if bad is None else 4), bad


def bits(t):
    return t.view(torch.int16 if t.dtype is torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter", [(64, 32, False), (128, 64, True), (192, 64, False), (112, 16, True), (256, 0, False)])
def test_what_is_not_rotated_reaches_no_other_element(d, rot, inter, dtype):
    # infinities, NaN and negative zeros in the dimensions behind the rotated ones
    B, N, H = 2, 19, 3
    x = draw(1, B, N, H, d, dtype=dtype)
    cs = angles(N, rot).to(DEV) if rot else None
    want, _ = ofa.attn_qk_norm_rope(x, x, None, None, cs, interleaved=inter)
    assert torch.equal(bits(want[..., rot:]), bits(x[..., rot:]))
    g = torch.Generator().manual_seed(7)
    bad = torch.rand(B, N, H, d, generator=g) < 0.1
    bad[..., :rot] = False
    bad = bad.to(DEV)
    for v in (math.inf, -math.inf, math.nan, -0.0):
        y = x.masked_fill(bad, v)
        for got in ofa.attn_qk_norm_rope(y, y, None, None, cs, interleaved=inter):
            assert torch.equal(bits(got[~bad]), bits(want[~bad])), v
            assert bool(torch.isnan(got[bad]).all()) if v != v else torch.equal(bits(got[bad]), bits(y[bad])), v
        back = ofa.attn_qk_norm_rope_bwd(x, x, y, y, None, None, cs, interleaved=inter)[1]
        clean = ofa.attn_qk_norm_rope_bwd(x, x, x, x, None, None, cs, interleaved=inter)[1]
        assert torch.equal(bits(back[~bad]), bits(clean[~bad])), v
        assert bool(torch.isnan(back[bad]).all()) if v != v else torch.equal(bits(back[bad]), bits(y[bad])), v
    # with a norm the root of an infinite mean is 0: 0 for every finite element, NaN for the infinite one alone
    w = (1 + 0.3 * draw(3, d, dtype=torch.float32)).to(dtype)
    y = x.clone()
    y[0, 4, 1, d - 3] = math.inf
    got, _ = ofa.attn_qk_norm_rope(y, y, w, w, cs, eps=EPS, interleaved=inter)
    hit = torch.zeros_like(bad)
    hit[0, 4, 1, d - 3] = True
    assert torch.equal(torch.isnan(got), hit)
    row = got[0, 4, 1]
    assert bool((row[~hit[0, 4, 1]] == 0).all())


def test_append_without_norms_or_angles_copies_every_element():
    s = paged_inputs([3, 5], [20, 9], 4, 2, 64, 16, poison=False)
    k, v = draw(2, 8, 2, 64), draw(3, 8, 2, 64)
    for t, at, x in ((k, 5, math.inf), (k, 40, -0.0), (v, 7, math.inf), (s["q"], 9, -math.inf), (s["q"], 41, -0.0)):
        t[:, :, at] = x
    q2 = ofa.attn_paged_append(s["q"], k, v, s["kp"], s["vp"], s["bt"], s["lens"], s["cu"])
    assert torch.equal(bits(q2), bits(s["q"]))
    for b, t, at in [(0, i, 17 + i) for i in range(3)] + [(1, 3 + i, 4 + i) for i in range(5)]:
        page = s["bt"][b, at // 16].long()
        assert torch.equal(bits(s["kp"][page, at % 16]), bits(k[t])) and torch.equal(bits(s["vp"][page, at % 16]), bits(v[t]))


def weight_chain(rows, H, other, d, dtype):
    """Additions that a term of a weight gradient goes through at most: a group of lanes takes two heads of a
    token at a time; its sum over all of them, the groups of a warp (3), the 4 warps of a block, every
    32nd block's partial, and 32 of those."""
    blocks = 4 * torch.cuda.get_device_properties(0).multi_processor_count
    per, per_other = -(-H // 2), -(-other // 2)
    groups = 32 // ((4 if dtype is torch.bfloat16 else 8) * (1 if d <= 64 else 2 if d <= 128 else 4))
    mine = max(blocks * per // (per + per_other), 1)  # (the queries' share is rounded down, the keys' up)
    mine = min(mine, -(-rows * per // (4 * groups)))
    return 2 * -(-rows * per // (mine * 4 * groups)) + 3 + 4 + -(-blocks // 32) + 32


@pytest.mark.parametrize("dtype,B,N,Hq,Hkv,d,rot,inter", [
    (torch.bfloat16, 2, 4099, 5, 3, 64, 64, True),
    (torch.bfloat16, 1, 5003, 7, 2, 128, 64, False),
    (torch.bfloat16, 3, 1501, 3, 1, 256, 256, True),
    (torch.float32, 2, 2999, 5, 3, 64, 32, False),
    (torch.float32, 1, 4001, 3, 5, 128, 128, True),
    (torch.float32, 2, 1009, 4, 3, 192, 64, True),
    (torch.float32, 1, 2503, 1, 2, 256, 256, False),
])
def test_weight_gradients_leave_no_row_out(dtype, B, N, Hq, Hkv, d, rot, inter):
    # several units a group of lanes, the last round ragged; a bound that one row more or less breaks
    q, k = draw(1, B, N, Hq, d, dtype=dtype), draw(2, B, N, Hkv, d, dtype=dtype)
    dq2, dk2 = draw(5, B, N, Hq, d, dtype=dtype), draw(6, B, N, Hkv, d, dtype=dtype)
    wq, wk = ((1 + 0.3 * draw(i, d, dtype=torch.float32)).to(dtype) for i in (3, 4))
    cs = angles(N, rot).to(DEV)
    dq, dk, dwq, dwk = ofa.attn_qk_norm_rope_bwd(q, k, dq2, dk2, wq, wk, cs, eps=EPS, interleaved=inter)
    tab = table_for(cs, torch.arange(N).expand(B, N))
    a, b = pair_index(d, rot, inter)
    for x, dy, w, dx, dw, H, other in ((q, dq2, wq, dq, dwq, Hq, Hkv), (k, dk2, wk, dk, dwk, Hkv, Hq)):
        rx, rw, lim, _ = norm_rope_bwd(x.cpu(), dy.cpu(), w.cpu(), tab, inter, EPS)
        check(dx, rx, lim, "dx")
        f, t = x.cpu().double(), dy.cpu().double().abs()
        n = f / (f.square().mean(-1, keepdim=True) + EPS).sqrt()
        turned, co, si = t.clone(), tab[..., :rot // 2].double().abs(), tab[..., rot // 2:].double().abs()
        turned[..., a], turned[..., b] = t[..., a] * co + t[..., b] * si, t[..., b] * co + t[..., a] * si
        # terms good to 32 U of what they are made of (the turn's three roundings, the norm's, two products)
        bound = (32 + weight_chain(B * N, H, other, d, dtype)) * U * (turned * n.abs()).sum((0, 1, 2))
        check(dw, rw, bound, "dw")
        for at in (0, B * N - 1, B * N // 2):  # the sum without one token's last head is out of it
            y = dy.cpu().clone()
            y.view(B * N, H, d)[at, H - 1] = 0
            less = norm_rope_bwd(x.cpu(), y, w.cpu(), tab, inter, EPS)[1]
            assert bool(((less - rw).abs() > 2 * bound).any())

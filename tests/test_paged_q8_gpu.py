"""The 8-bit paged cache on the GPU against plain 64-bit forms (paged_q8_helpers): what the append
writes, what is read back, attention over it, and runs of the three together."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_helpers import U, angles, norm_rope, paged_inputs
from paged_q8_helpers import CODE_HALF, E4M3, E8M0, check_attention, dequantise, pow2, q8_inputs, quantise, scale_bytes

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu()


def empty_cache(pages, page, Hkv, d, fill=0x7F):
    """Pages and scales in the places-first order, every byte `fill`."""
    kp, vp = (torch.full((pages, page, Hkv, d), fill, dtype=torch.uint8, device=DEV).view(E4M3) for _ in "kv")
    ks, vs = (torch.full((pages, Hkv, page), fill, dtype=torch.uint8, device=DEV).view(E8M0) for _ in "kv")
    return kp, vp, ks, vs


def batch(new, lens, page, seed=0):
    s = paged_inputs(new, lens, 1, 1, 16, page, seed=seed, poison=False)
    return s["bt"], s["lens"], s["cu"], s["kp"].shape[0]


def slots(bt, lens, new, page):
    """(page, slot) of every packed token that has one, and which do."""
    pg, sl, on = [], [], []
    for b, (nq, n) in enumerate(zip(new, lens)):
        for i in range(nq):
            at = n - nq + i
            on.append(at >= 0)
            pg.append(int(bt[b, at // page]) if at >= 0 else 0)
            sl.append(at % page if at >= 0 else 0)
    return torch.tensor(pg), torch.tensor(sl), torch.tensor(on)


# ------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,Hkv,page", [(16, 1, 1), (64, 2, 16), (128, 8, 7), (192, 3, 16), (256, 1, 64)])
def test_rows_as_they_are(d, Hkv, page, dtype):
    """Without norm and rotation what is written is decided to the bit: codes and scales of every row, special rows
    among them; nothing else is written."""
    new, lens = [1, 40, 0, 3], [9, 40, 5, 2]
    bt, ln, cu, pages = batch(new, lens, page)
    g = torch.Generator().manual_seed(d)
    T = sum(new)
    k, v = (torch.randn(T, Hkv, d, generator=g) * torch.exp2(torch.randint(-20, 20, (T, Hkv, 1), generator=g).float()) for _ in "kv")
    k[0], v[0] = 0.0, -0.0
    k[1], v[1] = 448.0, 448.0 * 2.0 ** -3                 # a power of two exactly
    k[2, :, 0], v[2, :, 0] = 449.0, 1.7501 * 2.0 ** 10    # just past one
    k[3, :, 1], v[3, :, 2] = math.nan, math.nan
    k[4, :, 1], v[4, :, 2] = math.inf, -math.inf
    k[5], v[5] = math.nan, math.inf
    k[6], v[6] = 3e38, -1e-38
    v[7] = 1e-42
    k[8] = torch.linspace(-1, 1, d)
    k, v = k.to(dtype).to(DEV), v.to(dtype).to(DEV)
    q = torch.randn(T, 2 * Hkv, d, generator=g).to(dtype).to(DEV)
    kp, vp, ks, vs = empty_cache(pages, page, Hkv, d)
    ofa.device_error_flags()
    qo = ofa.attn_paged_append_q8(q, k, v, kp, vp, ks, vs, bt, ln, cu)
    assert ofa.device_error_flags() == 0 and torch.equal(qo, q)
    pg, sl, on = slots(bt.cpu(), lens, new, page)
    assert not bool(on.all())  # the last sequence has a token without a place
    for x, codes, scales in ((k, kp, ks), (v, vp, vs)):
        want_c, want_s = (torch.full(t.shape, 0x7F, dtype=torch.uint8) for t in (codes, scales))
        c, e = quantise(x.cpu())
        want_c[pg[on], sl[on]] = c.view(torch.uint8)[on]
        want_s[pg[on], :, sl[on]] = e.view(torch.uint8)[on]
        got = bytes_of(codes)
        nan = (want_c & 0x7F) == 0x7F  # a NaN's sign is not promised
        assert torch.equal(nan, (got & 0x7F) == 0x7F) and torch.equal(got[~nan], want_c[~nan])
        assert torch.equal(bytes_of(scales), want_s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,rot", [(4, 2, 64, 64), (16, 8, 128, 128), (7, 1, 128, 64), (5, 5, 256, 32), (2, 2, 48, 16)])
def test_keys_after_norm_and_rotation(Hq, Hkv, d, rot, inter, dtype):
    """Against 64 bits: a scale is the least that holds the row (within the fp32 error of its largest element), a
    code is off by half a step and that error; the queries are attn_paged_append's bit for bit."""
    new, lens, page = [1, 33, 5], [100, 33, 64], 16
    bt, ln, cu, pages = batch(new, lens, page, seed=3)
    g = torch.Generator().manual_seed(4)
    T = sum(new)
    q, k, v = (torch.randn(T, h, d, generator=g).to(dtype).to(DEV) for h in (Hq, Hkv, Hkv))
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).to(DEV)
    cs = angles(100, rot).to(DEV)
    kp, vp, ks, vs = empty_cache(pages, page, Hkv, d)
    qo = ofa.attn_paged_append_q8(q, k, v, kp, vp, ks, vs, bt, ln, cu, wq=w, wk=w, cos_sin=cs, interleaved=inter)
    kb, vb = (torch.zeros(pages, page, Hkv, d, dtype=dtype, device=DEV) for _ in "kv")
    assert torch.equal(qo, ofa.attn_paged_append(q, k, v, kb, vb, bt, ln, cu, wq=w, wk=w, cos_sin=cs, interleaved=inter))
    pg, sl, _ = slots(bt.cpu(), lens, new, page)
    pos = torch.cat([torch.arange(n - c, n) for n, c in zip(lens, new)])
    y, _ = norm_rope(k.cpu(), w.cpu(), cs.cpu()[pos][:, None], inter, 1e-6)
    t = k.cpu().double()
    t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.cpu().double()
    err = 32 * U * 1.5 * t.abs().amax(-1, keepdim=True)  # of y in fp32, as norm_rope derives it
    e = ks.cpu().view(torch.uint8)[pg, :, sl]
    amax, room = y.abs().amax(-1), 448 * pow2(e)
    assert bool((amax - err[..., 0] <= room).all()) and bool(((amax + err[..., 0] > room / 2) | (e == 0)).all())
    got = dequantise(kp.cpu().view(torch.uint8)[pg, sl], e)
    step = pow2(e)[..., None] * 2.0 ** -10  # half the step of the smallest codes
    assert bool(((got - y).abs() <= torch.maximum(CODE_HALF * y.abs(), step) + 2 * err).all())
    c, ev = quantise(v.cpu())
    assert torch.equal(vp.cpu().view(torch.uint8)[pg, sl], c.view(torch.uint8)) and torch.equal(vs.cpu().view(torch.uint8)[pg, :, sl], ev.view(torch.uint8))


def test_append_reports_and_leaves():
    new, lens, page, Hkv, d = [2, 2], [20, 17], 16, 2, 64
    bt, ln, cu, pages = batch(new, lens, page)
    bt[0, 1] = 10 ** 6  # positions 18 and 19 have no page
    x = torch.ones(8, Hkv, d, dtype=torch.bfloat16, device=DEV)
    kp, vp, ks, vs = empty_cache(pages, page, Hkv, d, 0x11)
    qo = torch.full((8, Hkv, d), 5.0, dtype=torch.bfloat16, device=DEV)
    ofa.device_error_flags()
    ofa.attn_paged_append_q8(x, x, x, kp, vp, ks, vs, bt, ln, cu + 2, q_out=qo)
    assert ofa.device_error_flags() == 4
    assert bool((qo[:2] == 5).all()) and bool((qo[6:] == 5).all()) and bool((qo[2:6] == 1).all())
    touched = (bytes_of(kp) != 0x11).any(-1).any(-1).nonzero().tolist()
    assert sorted(touched) == sorted([[int(bt[1, 0]), 15], [int(bt[1, 1]), 0]])
    assert int((bytes_of(ks) != 0x11).sum()) == int((bytes_of(vs) != 0x11).sum()) == 2 * Hkv


# -------------------------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,Hkv,page,hf", [(16, 1, 1, False), (64, 3, 16, True), (128, 8, 64, True), (256, 5, 7, False), (48, 40, 16, False)])
def test_read_gives_the_numbers(d, Hkv, page, hf, dtype):
    """Every code and scale byte as the number that it stands for, rounded to nearest."""
    lens, rows = [70, 1, 0, 33], [70, 1, 0, 20]
    bt, ln, _, pages = batch(lens, lens, page)
    g = torch.Generator().manual_seed(d)
    kp, vp = (torch.randint(0, 256, (pages, page, Hkv, d), generator=g, dtype=torch.uint8) for _ in "kv")
    ks, vs = (torch.randint(0, 256, (pages, Hkv, page), generator=g, dtype=torch.uint8) for _ in "kv")
    dk, dv = (p.permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3) if hf else p.to(DEV) for p in (kp, vp))
    cu = torch.tensor([0, 70, 71, 71, 91], dtype=torch.int32, device=DEV) + 1
    T = sum(rows) + 3
    out = [torch.full((T, Hkv, d), 9.0, dtype=dtype, device=DEV) for _ in "kv"]
    ofa.device_error_flags()
    got = ofa.attn_paged_read_q8(dk.view(E4M3), dv.view(E4M3), ks.to(DEV).view(E8M0), vs.to(DEV), bt, ln, T, cu, dtype=dtype,
                                 k_out=out[0], v_out=out[1])
    assert ofa.device_error_flags() == 0
    b = bt.cpu()
    place = [(int(b[s, at // page]), at % page) for s, (n, r) in enumerate(zip(lens, rows)) for at in range(n - r, n)]
    pg, sl = (torch.tensor(x) for x in zip(*place))
    for o, c, e in zip(got, (kp, vp), (ks, vs)):
        o = o.cpu()
        assert bool((o[0] == 9).all()) and bool((o[-2:] == 9).all())
        want = dequantise(c[pg, sl], e[pg, :, sl])
        have, exact = o[1:-2], want.to(dtype)
        same = (have == exact) | (have.isnan() & exact.isnan())
        assert bool(same.all())


def test_read_of_uniform_rows_and_bad_pages():
    lens = [32, 48]
    s = q8_inputs([1, 1], lens, 1, 2, 64, 16, poison=False)
    ofa.device_error_flags()
    k, v = ofa.attn_paged_read_q8(s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], 64)
    b = s["bt"].cpu().long()
    for o, n in ((k, "k"), (v, "v")):
        want = torch.cat([dequantise(s[n + "p"].cpu().view(torch.uint8)[b[i, :-(-x // 16)]].flatten(0, 1)[x - 32:x],
                                     s[n + "s"].cpu().view(torch.uint8)[b[i, :-(-x // 16)]].transpose(1, 2).flatten(0, 1)[x - 32:x]) for i, x in enumerate(lens)])
        assert torch.equal(o.cpu().double(), want)
    s["bt"][0, 1] = -1
    out = torch.full((64, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    k2, _ = ofa.attn_paged_read_q8(s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], 64, k_out=out)
    assert ofa.device_error_flags() == 4
    assert bool((k2[16:32] == 3).all()) and torch.equal(k2[:16], k[:16]) and torch.equal(k2[32:], k[32:])


# --------------------------------------------------------------------------------- attention

def run(s, causal=True, scale=None, **kw):
    return ofa.attn_paged_fwd_q8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"], causal=causal, scale=scale, **kw)


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
def test_paged_fwd_q8(case, hint):
    new, lens, Hq, Hkv, d, page, causal = case
    s = q8_inputs(new, lens, Hq, Hkv, d, page, seed=len(new), heads_first=page != 32)
    ofa.device_error_flags()
    o, lse = run(s, causal, max_q=max(new) if hint else None)
    assert ofa.device_error_flags() == 0
    check_attention(o, lse, s, new, lens, causal, 1 / math.sqrt(d))
    o2, lse2 = run(s, causal, max_q=max(new) if hint else None)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


@pytest.mark.parametrize("seed", range(16))
def test_paged_fwd_q8_random(seed):
    g = torch.Generator().manual_seed(200 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    B, Hkv, G = r(1, 7), r(1, 3), r(1, 9)
    d, page, causal = (64, 128)[r(0, 1)], (16, 32, 64, 128)[r(0, 3)], r(0, 4) > 0
    big = r(0, 2)
    new = [1 if big == 0 else r(0, (0, 12, 200)[big]) for _ in range(B)]
    lens = [r(0, (2000, 300, 600)[big]) for _ in range(B)]
    s = q8_inputs(new, lens, Hkv * G, Hkv, d, page, seed=seed, heads_first=bool(r(0, 1)), spread=(0.0, 0.5, 2.0)[r(0, 2)])
    if sum(new) == 0:
        return
    o, lse = run(s, causal, max_q=r(0, 1) * max(new), scale=0.2)
    assert ofa.device_error_flags() == 0
    check_attention(o, lse, s, new, lens, causal, 0.2, what=f"seed {seed}")


@pytest.mark.parametrize("max_q", [1, 40, 300])
@pytest.mark.parametrize("order", [1, -1, 0])
def test_scales_far_apart(order, max_q):
    """Value scales that grow, fall or jump along the sequence by 2^24 in all, key scales by 2^10."""
    new, lens = [1, 40], [700, 900]
    s = q8_inputs(new, lens, 4, 2, 128, 64, seed=5)
    g = torch.Generator().manual_seed(6)
    for b in range(2):
        at = torch.arange(lens[b], dtype=torch.float64) / lens[b]
        if order == 0:
            at = torch.rand(lens[b], generator=g).double()
        at = at if order >= 0 else 1 - at
        pg, sl = s["bt"][b].cpu().long()[torch.arange(lens[b]) // 64], torch.arange(lens[b]) % 64
        s["vs"].view(torch.uint8)[pg.to(DEV), :, sl.to(DEV)] = (127 - 12 + (24 * at).int()).to(torch.uint8)[:, None].to(DEV).expand(-1, 2)
        s["ks"].view(torch.uint8)[pg.to(DEV), :, sl.to(DEV)] = (127 - 16 + (10 * at).int()).to(torch.uint8)[:, None].to(DEV).expand(-1, 2)
    o, lse = run(s, max_q=max_q)
    check_attention(o, lse, s, new, lens, True, 1 / math.sqrt(128))


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -30, 2.0 ** 18, 2.0 ** 100])
@pytest.mark.parametrize("max_q", [1, 40])
def test_queries_of_any_size(size, max_q):
    """Queries far outside fp16's range, the scale taking it back."""
    new, lens = [1, 40], [200, 300]
    s = q8_inputs(new, lens, 4, 2, 64, 16, seed=7)
    s["q"] = (s["q"].float() * size).bfloat16()
    o, lse = run(s, scale=0.1 / size, max_q=max_q)
    check_attention(o, lse, s, new, lens, True, 0.1 / size)


@pytest.mark.parametrize("max_q", [1, 30])
def test_a_nan_reaches_the_rows_that_see_it(max_q):
    new, lens, d = [1, 30], [100, 130], 128
    s = q8_inputs(new, lens, 4, 2, d, 16, seed=8)
    want, wl = run(s, max_q=max_q)
    pg = lambda b, at: (int(s["bt"][b, at // 16]), at % 16)  # noqa: E731
    p, i = pg(1, 115)
    s["kp"].view(torch.uint8)[p, i, 0, 3] = 0x7F   # key 115 of sequence 1, head 0
    p, i = pg(1, 120)
    s["ks"].view(torch.uint8)[p, 1, i] = 255       # key 120, head 1
    o, lse = run(s, max_q=max_q)
    sees = torch.arange(130 - 30, 130)
    for h, at in ((0, 115), (1, 115), (2, 120), (3, 120)):
        nan = torch.cat([torch.tensor([False]), sees >= at]).to(DEV)
        assert torch.equal(o[:, h].isnan().all(-1), nan) and torch.equal(lse[:, h].isnan(), nan)
        assert torch.equal(o[~nan, h], want[~nan, h]) and torch.equal(lse[~nan, h], wl[~nan, h])
    s["q"][0, 1, 5] = math.nan
    o, lse = run(s, max_q=max_q)
    assert bool(o[0, 1].isnan().all()) and bool(lse[0, 1].isnan()) and torch.equal(o[0, 0], want[0, 0]) and torch.equal(o[0, 2:], want[0, 2:])


def test_rows_outside_the_sequences_stay_and_strides():
    new, lens = [2, 30], [40, 50]
    s = q8_inputs(new, lens, 4, 2, 64, 16)
    o0, l0 = run(s, max_q=30)
    wide = torch.zeros(42, 10, 2, 64, dtype=torch.bfloat16, device=DEV)
    q = wide[:, 2:6, 1]
    q[5:-5] = s["q"]
    out, lse = torch.full((4, 42, 128), 3.0, dtype=torch.bfloat16, device=DEV).permute(1, 0, 2)[..., :64], torch.full((42, 4), 5.0, device=DEV)
    # a cache inside a wider one
    big = {n: torch.zeros(s[n + "p"].shape[0], 16, 5, 64, dtype=torch.uint8, device=DEV).view(E4M3) for n in "kv"}
    sc = {n: torch.zeros(s[n + "p"].shape[0], 5, 32, dtype=torch.uint8, device=DEV).view(E8M0) for n in "kv"}
    for n in "kv":
        big[n].view(torch.uint8)[:, :, 1:3] = s[n + "p"].view(torch.uint8)
        sc[n].view(torch.uint8)[:, 2:4, 16:] = s[n + "s"].view(torch.uint8)
    ofa.attn_paged_fwd_q8(q, big["k"][:, :, 1:3], big["v"][:, :, 1:3], sc["k"][:, 2:4, 16:], sc["v"][:, 2:4, 16:], s["bt"], s["lens"],
                          s["cu"] + 5, out=out, lse=lse, max_q=30)
    assert torch.equal(out[5:-5], o0) and torch.equal(lse[5:-5], l0)
    assert bool((out[:5] == 3).all()) and bool((out[-5:] == 3).all()) and bool((lse[:5] == 5).all()) and bool((lse[-5:] == 5).all())
    assert ofa.device_error_flags() == 0


def test_bad_pages_and_lengths_are_reported():
    for mq in (1, 40):
        s = q8_inputs([1, 1], [100, 40], 2, 1, 64, 16)
        want, _ = run(s, max_q=mq)
        s["bt"][0, 3] = -7
        s["bt"][0, 4] = 1 << 30
        ofa.device_error_flags()
        o, _ = run(s, max_q=mq)
        assert ofa.device_error_flags() == 4 and torch.equal(o[1], want[1])
        s = q8_inputs([1, 40], [112, 40], 2, 1, 64, 16, width=7)
        want, _ = run(s, max_q=mq)
        s["lens"][0] = 5000  # the table holds 112
        o, _ = run(s, max_q=mq)
        assert ofa.device_error_flags() == 2 and torch.equal(o, want)


@pytest.mark.parametrize("cu", [[0, 4, 2, 6], [0, 9, 9, 9], [-5, 2, 3, 6], [6, 4, 2, 0], [2, 3, 4, 5]])
def test_a_malformed_cu_faults_nothing(cu):
    s = q8_inputs([2, 2, 2], [20, 30, 17], 2, 1, 64, 16)
    bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
    for mq in (0, 2, 64):
        ofa.attn_paged_fwd_q8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], bad, max_q=mq)
    ofa.attn_paged_read_q8(s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], 6, bad)
    torch.cuda.synchronize()
    ofa.device_error_flags()


def test_a_cache_past_four_gib():
    # codes beyond 2^32 bytes of both caches
    page, Hkv, d = 128, 8, 128
    pages = (1 << 32) // (page * Hkv * d) + 40
    s = q8_inputs([1, 40], [900, 700], 16, 8, d, page, poison=False, heads_first=False)
    n = s["kp"].shape[0]
    big = dict(s)
    for x in "kv":
        big[x + "p"] = torch.zeros(pages, page, Hkv, d, dtype=torch.uint8, device=DEV)
        big[x + "s"] = torch.zeros(pages, Hkv, page, dtype=torch.uint8, device=DEV)
        big[x + "p"][-n:] = s[x + "p"].view(torch.uint8)
        big[x + "s"][-n:] = s[x + "s"].view(torch.uint8)
    big["bt"] = torch.where(s["bt"] < n, s["bt"] + (pages - n), s["bt"])
    for mq in (1, 40):
        a, b = run(s, max_q=mq), run(big, max_q=mq)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    args = lambda t: (t["kp"], t["vp"], t["ks"], t["vs"], t["bt"], t["lens"], 41, t["cu"])  # noqa: E731
    for x, y in zip(ofa.attn_paged_read_q8(*args(s)), ofa.attn_paged_read_q8(*args(big))):
        assert torch.equal(x, y)
    k, v = (torch.randn(41, 8, d, device=DEV).bfloat16() for _ in "kv")
    for t in (s, big):
        ofa.attn_paged_append_q8(s["q"], k, v, t["kp"], t["vp"], t["ks"], t["vs"], t["bt"], t["lens"], t["cu"])
    for x, y in zip(ofa.attn_paged_read_q8(*args(s)), ofa.attn_paged_read_q8(*args(big))):
        assert torch.equal(x, y)


# ------------------------------------------------------------------------------ all together

def test_a_prompt_in_chunks_then_tokens():
    """Appended in chunks of many sizes and token by token, attended over, read back: every step's rows are those of
    the 64-bit attention over what the cache holds, and the cache holds what one append of all would leave."""
    N, Hq, Hkv, d, page = 333, 8, 2, 128, 16
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(N, h, d, generator=g).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv))
    w = (1 + 0.2 * torch.randn(d, generator=g)).bfloat16().to(DEV)
    cs = angles(N, d).to(DEV)
    pages = -(-N // page) + 2
    bt = torch.randperm(pages, generator=g)[:pages - 2].int().to(DEV)[None]
    whole, parts = empty_cache(pages, page, Hkv, d), empty_cache(pages, page, Hkv, d)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    qa = ofa.attn_paged_append_q8(q, k, v, *whole, bt, i32(N), None, wq=w, wk=w, cos_sin=cs)
    at = 0
    for c in [100, 1, 64, 130, 5] + [1] * 33:
        sl = slice(at, at + c)
        at += c
        qr = ofa.attn_paged_append_q8(q[sl], k[sl], v[sl], *parts, bt, i32(at), i32(0, c), wq=w, wk=w, cos_sin=cs)
        assert torch.equal(qr, qa[sl])
        o, lse = ofa.attn_paged_fwd_q8(qr, *parts, bt, i32(at), i32(0, c), max_q=c)
        s = dict(q=qr, kp=parts[0], vp=parts[1], ks=parts[2], vs=parts[3], bt=bt)
        check_attention(o, lse, s, [c], [at], True, 1 / math.sqrt(d), what=f"to {at}")
    assert at == N and ofa.device_error_flags() == 0
    for a, b in zip(whole, parts):
        assert torch.equal(bytes_of(a), bytes_of(b))
    # the numbers read back, in a bf16 cache: the same attention but for the rounding of the weights
    kb, vb = ofa.attn_paged_read_q8(*parts, bt, i32(N), N)
    full = [torch.zeros(pages, page, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    for f, x in zip(full, (kb, vb)):
        f[bt[0].long()] = torch.cat([x, x.new_zeros((pages - 2) * page - N, Hkv, d)]).view(-1, page, Hkv, d)
    o8, l8 = ofa.attn_paged_fwd_q8(qa, *parts, bt, i32(N))
    o16, l16 = ofa.attn_paged_fwd(qa, *full, bt, i32(N))
    s = dict(q=qa, kp=parts[0], vp=parts[1], ks=parts[2], vs=parts[3], bt=bt)
    check_attention(o8, l8, s, [N], [N], True, 1 / math.sqrt(d))
    assert float((o8.float() - o16.float()).norm() / o16.float().norm()) <= 2 * 2.0 ** -8  # two roundings to bf16, and one of the weights
    assert float((l8 - l16).abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("max_q", [1, 4])
def test_captured_and_replayed(max_q):
    """Append and attention in one graph, replayed with new tokens and lengths in the same tensors, the workspace full
    of anything."""
    Hq, Hkv, d, page, B = 16, 2, 128, 16, 5
    lens = [700, 3, 0, 129, 1400]
    new = [1] * B
    s = q8_inputs(new, [n + 2 for n in lens], Hq, Hkv, d, page, seed=9)
    g = torch.Generator().manual_seed(10)
    q, k, v = (torch.randn(2, B, h, d, generator=g).bfloat16().to(DEV) for h in (Hq, Hkv, Hkv))
    ln = torch.zeros(B, dtype=torch.int32, device=DEV)
    sq, sk, sv = (torch.zeros_like(t[0]) for t in (q, k, v))
    cache = (s["kp"], s["vp"], s["ks"], s["vs"])
    n = ofa.paged_fwd_q8_workspace_bytes(sq, *cache, s["bt"], ln, s["cu"], max_q)
    assert n > 0
    ws = torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros_like(sq), torch.zeros(B, Hq, device=DEV)

    def step():
        qr = ofa.attn_paged_append_q8(sq, sk, sv, *cache, s["bt"], ln, s["cu"])
        ofa.attn_paged_fwd_q8(qr, *cache, s["bt"], ln, s["cu"], max_q=max_q, workspace=ws, out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(2):
        for dst, src in ((sq, q[i]), (sk, k[i]), (sv, v[i])):
            dst.copy_(src)
        ln.copy_(torch.tensor([x + i + 1 for x in lens]))
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out, lse, dict(s, q=q[i]), new, [x + i + 1 for x in lens], True, 1 / math.sqrt(d), what=f"replay {i}")
    assert ofa.device_error_flags() == 0


def test_calls_on_two_streams_at_once():
    cases = [([1] * 20, [1500 + 7 * i for i in range(20)], 1), ([300, 1], [900, 2000], 300)]
    data = [q8_inputs(new, lens, 8, 2, 128, 16, seed=i) for i, (new, lens, _) in enumerate(cases)]
    want = [run(s, max_q=c[2]) for s, c in zip(data, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(5):
        for i, (s, c) in enumerate(zip(data, cases)):
            got[i].append(run(s, max_q=c[2], stream=streams[i]))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o, lse in outs:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_python_refusals():
    s = q8_inputs([1], [20], 2, 1, 64, 16)
    args = [s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"]]
    for i, bad in ((1, s["kp"].view(torch.int8)), (2, s["vp"].to(torch.bfloat16)), (3, s["ks"].view(torch.uint8).float()), (4, s["vs"].cpu()),
                   (3, s["ks"][:, :, :8]), (4, s["vs"].transpose(1, 2))):
        with pytest.raises(ValueError):
            ofa.attn_paged_fwd_q8(*args[:i], bad, *args[i + 1:])
    with pytest.raises(TypeError):
        ofa.attn_paged_read_q8(*args[1:7], 4, dtype=torch.float16)
    with pytest.raises(ofa.AttnError) as e:  # fp32 queries
        ofa.attn_paged_fwd_q8(s["q"].float(), *args[1:])
    assert e.value.status == ofa.Status.UNSUPPORTED
    with pytest.raises(ofa.AttnError) as e:  # scales that do not begin on 16 bytes
        sc = torch.zeros(s["kp"].shape[0], 1, 40, dtype=torch.uint8, device=DEV)
        ofa.attn_paged_fwd_q8(args[0], args[1], args[2], sc[..., 4:20], *args[4:])
    assert e.value.status == ofa.Status.MISALIGNED


def test_no_tokens():
    s = q8_inputs([1], [20], 2, 1, 64, 16)
    o, lse = ofa.attn_paged_fwd_q8(s["q"][:0], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"] * 0)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    k, v = ofa.attn_paged_read_q8(s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], 0, s["cu"] * 0)
    assert k.shape == v.shape == (0, 1, 64)

"""NaN and infinities behind shared prefixes: what one of the two attentions makes NaN stays NaN whatever the other one's
weight, on every path that joins two states (rows finished and cut, side by side and one after the other)."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from test_paged_prefix_gpu import inputs, run

pytestmark = pytest.mark.gpu
DEV = "cuda"

PATHS = [  # new, own lens, prefix lengths, cuts
    ([1] * 3, [30, 1, 17], [40, 30], [0, 2, 3]),                        # few rows either way
    ([1] * 40, [20 + i for i in range(40)], [120, 90], [0, 20, 40]),    # side by side, prefixes too short to be cut
    ([1] * 40, [20 + i for i in range(40)], [3000, 90], [0, 20, 40]),   # side by side, a cut one
    ([70, 50], [70, 90], [100, 60], [0, 70, 120]),                      # one after the other
    ([70, 50], [70, 90], [3000, 60], [0, 70, 120]),                     # and a cut prefix
]


def make(path, q8, d=128):
    new, lens, plens, cuts = path
    s, groups = inputs(new, lens, plens, cuts, 16, 2, d, 16, q8, seed=21)
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    return s, groups.to(DEV), seq.to(DEV)


def key_rows(s, table, at):
    """(page, slot) index tensors of the positions `at` of a table row."""
    at = torch.as_tensor(at)
    return table.cpu().long()[at // 16].to(DEV), (at % 16).to(DEV)


def set_key(s, n, table, at, head, value):
    p, i = key_rows(s, table, at)
    if n + "s" in s:
        s[n + "p"].view(torch.uint8)[p, i, head] = 0x7F if math.isnan(value) else 0x38  # (1)
        s[n + "s"].view(torch.uint8)[p, head, i] = 127 if math.isnan(value) else 127 + int(math.log2(value))
    else:
        s[n + "p"][p, i, head] = value


def check_nan(got, want, hit):
    (o, lse), (wo, wl) = got, want
    assert torch.equal(o.isnan().all(-1), hit) and torch.equal(o.isnan().any(-1), hit) and torch.equal(lse.isnan(), hit)
    assert torch.equal(o[~hit], wo[~hit]) and torch.equal(lse[~hit], wl[~hit])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("path", PATHS)
def test_a_prefix_of_nan_keys(path, q8):
    """Every logit over prefix 0 is NaN: the state has no maximum, and its sum is NaN."""
    s, groups, _ = make(path, q8)
    mq = max(path[0])
    want = run(s, max_q=mq)
    set_key(s, "k", s["pt"][0], torch.arange(path[2][0]), 0, math.nan)
    hit = (groups == 0)[:, None] & (torch.arange(16, device=DEV) < 8)
    check_nan(run(s, max_q=mq), want, hit)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("path", PATHS)
def test_a_nan_query(path, q8):
    """Of a token with own keys and of one without."""
    new, lens, plens, cuts = path
    lens = [0 if new[0] == 1 else lens[0]] + list(lens[1:])
    s, _, _ = make((new, lens, plens, cuts), q8)
    want = run(s, max_q=max(new))
    hit = torch.zeros(len(s["q"]), 16, dtype=torch.bool, device=DEV)
    for t, h in ((0, 3), (len(s["q"]) - 1, 9)):
        s["q"][t, h, 5] = math.nan
        hit[t, h] = True
    check_nan(run(s, max_q=max(new)), want, hit)


@pytest.mark.parametrize("nan_in", ["k", "v"])
@pytest.mark.parametrize("heavy", ["own", "prefix"])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("path", PATHS)
def test_a_nan_in_the_lighter_part(path, q8, heavy, nan_in):
    """One NaN key, or value, among those of the part whose weight beside the other's is 0 in fp32 (logits 512 apart)."""
    s, groups, seq = make(path, q8)
    mq = max(path[0])
    s["q"] = torch.ones_like(s["q"])  # a logit is the sum of a key's elements, times the scale
    scale = 16 / math.sqrt(128)       # 724 for a key of 4 in every element; 16 times a normal number or two for the others
    if heavy == "own":
        for b in range(len(path[0])):
            set_key(s, "k", s["bt"][b], [0], 0, 4.0)
        where, table = groups == 0, s["pt"][0]
    else:
        for p in (0, 1):
            set_key(s, "k", s["pt"][p], [0], 0, 4.0)
        where, table = seq == 0, s["bt"][0]
    want = run(s, max_q=mq, scale=scale)
    # position 0 of a sequence's own keys is seen by its first token where there are as many keys as tokens, and by the later ones
    at = 7 if heavy == "own" else 0
    set_key(s, nan_in, table, [at], 0, math.nan)
    hit = where[:, None] & (torch.arange(16, device=DEV) < 8)
    got = run(s, max_q=mq, scale=scale)
    if nan_in == "k":
        check_nan(got, want, hit)
    else:  # lse knows nothing of values
        assert torch.equal(got[0].isnan().all(-1), hit) and torch.equal(got[0].isnan().any(-1), hit) and torch.equal(got[1], want[1])
        assert torch.equal(got[0][~hit], want[0][~hit])

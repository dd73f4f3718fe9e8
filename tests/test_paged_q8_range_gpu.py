"""Attention over codes whose scales lie far apart: what a row does not see, or gives no weight, does not touch it, and what it
does see is not lost beside it (paged_range_helpers.visible_ref)."""
import math

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_q8_helpers import q8_inputs
from paged_range_helpers import check_visible
from test_paged_prefix_gpu import inputs, run as run_prefix
from test_paged_q8_gpu import run

pytestmark = pytest.mark.gpu
DEV = "cuda"

SHAPES = [  # new, lens, Hq, Hkv, d
    ([4, 1], [70, 40], 4, 2, 128),          # up to 8 rows a key head
    ([8, 3], [150, 200], 4, 2, 64),         # up to 16
    ([1, 2], [900, 300], 4, 2, 128),        # few rows, cut
    ([30, 12], [140, 300], 4, 2, 128),      # one tile
    ([30, 12], [140, 2300], 4, 2, 64),      # one tile, cut
    ([150, 70], [200, 300], 4, 2, 128),     # two tiles
]


def places(s, b, at, page=16):
    at = torch.as_tensor(at)
    return s["bt"][b].cpu().long()[at // page].to(DEV), (at % page).to(DEV)


def bytes_at(s, n, b, at):
    """The scale bytes of positions `at` of sequence b, [keys, Hkv], to read and to write back."""
    p, i = places(s, b, at)
    return s[n + "s"].view(torch.uint8)[p, :, i]


def set_bytes(s, n, b, at, v):
    p, i = places(s, b, at)
    s[n + "s"].view(torch.uint8)[p, :, i] = v.to(torch.uint8).to(DEV)


def set_codes(s, n, b, at, x):
    """x [keys, d] floats that are codes."""
    p, i = places(s, b, at)
    s[n + "p"].view(torch.uint8)[p, i] = x.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)[:, None].expand(-1, s["kp"].shape[2], -1)


def go(s, new, lens, scale, **kw):
    ofa.device_error_flags()
    o, lse = run(s, scale=scale, max_q=max(new))
    assert ofa.device_error_flags() == 0
    check_visible(o, lse, s, new, lens, True, scale, **kw)


@pytest.mark.parametrize("up", [30, 90])
@pytest.mark.parametrize("which", ["v", "k", "kv"])
@pytest.mark.parametrize("shape", SHAPES)
def test_hidden_keys_of_large_scales(shape, which, up):
    """The later tokens' keys and values lie 2^30 and more above the others: the tokens before them do not see them."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=31)
    for b, (nq, n) in enumerate(zip(new, lens)):
        for at in {n - 1, n - nq // 2}:
            if at < n:
                for x in which:
                    set_bytes(s, x, b, [at], bytes_at(s, x, b, [at]).cpu().int() + up)
    go(s, new, lens, 0.1)


@pytest.mark.parametrize("size", [4, 16])
@pytest.mark.parametrize("shape", SHAPES)
def test_keys_of_no_weight_and_large_values(shape, size):
    """A visible key whose weight is 2^-60 or less (0 in fp32), with a value 2^40 above the others'."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=32)
    g = torch.Generator().manual_seed(1)
    u = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    s["q"] = (u + 0.1 * torch.randn(s["q"].shape, generator=g)).bfloat16().to(DEV)
    for b, n in enumerate(lens):
        at = [3, n // 2]
        set_codes(s, "k", b, at, (-size * u).expand(2, -1))
        set_bytes(s, "k", b, at, torch.full((2, Hkv), 127))
        set_bytes(s, "v", b, at, bytes_at(s, "v", b, at).cpu().int() + 40)
    scale = 1.0 if d == 64 else 0.5
    go(s, new, lens, scale, fine=2.0 ** -5)


@pytest.mark.parametrize("shape", SHAPES)
def test_many_small_weights(shape):
    """The largest weight's value is zero, the others' weights are 2^-22 of it: the output is theirs alone."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=33, spread=0.0)
    g = torch.Generator().manual_seed(2)
    u = torch.where(torch.rand(d, generator=g) < 0.5, -1.0, 1.0)
    s["q"] = u.expand(s["q"].shape).bfloat16().contiguous().to(DEV)
    scale = 22 * math.log(2) / d
    for b, n in enumerate(lens):
        set_codes(s, "k", b, torch.arange(n), torch.zeros(n, d))
        set_codes(s, "k", b, [1], u[None])
        set_bytes(s, "k", b, torch.arange(n), torch.full((n, Hkv), 127))
        p, i = places(s, b, torch.arange(n))
        s["vp"].view(torch.uint8)[p, i] &= 0x7F  # of one sign
        set_codes(s, "v", b, [1], torch.zeros(1, d))
    go(s, new, lens, scale, fine=2.0 ** -4)


@pytest.mark.parametrize("low,high", [(-20, 20), (-60, 60), (-120, 100)])
@pytest.mark.parametrize("shape", SHAPES)
def test_values_of_any_scale(shape, low, high):
    """Scales of values anywhere within 2^40, 2^120 and 2^220, key by key and head by head; some rows of zeros."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=34)
    g = torch.Generator().manual_seed(3)
    for b, n in enumerate(lens):
        set_bytes(s, "v", b, torch.arange(n), torch.randint(127 + low, 128 + high, (n, Hkv), generator=g))
        zero = torch.arange(2, n, 5)
        set_codes(s, "v", b, zero, torch.zeros(len(zero), d))
        set_bytes(s, "v", b, zero, torch.zeros(len(zero), Hkv))
    go(s, new, lens, 0.1)


@pytest.mark.parametrize("step", [1, 2, -1, -2])
@pytest.mark.parametrize("shape", SHAPES)
def test_values_that_grow_as_their_weights_fall(shape, step):
    """Weights over 2^20, a key's value as much larger as its weight is smaller: every key counts alike, whichever way the
    maximum goes."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=35, spread=0.0)
    s["q"] = torch.zeros_like(s["q"])
    s["q"][..., 0] = 1.0
    for b, n in enumerate(lens):
        at = torch.arange(n)
        e = ((at - n // 2) * step / 8).clamp(-10, 10).int()  # eight keys of one weight
        x = torch.zeros(n, d)
        x[:, 0] = -e.float()
        set_codes(s, "k", b, at, x)
        set_bytes(s, "k", b, at, torch.full((n, Hkv), 127))
        set_bytes(s, "v", b, at, (120 + e)[:, None].expand(-1, Hkv))
    go(s, new, lens, math.log(2), fine=2.0 ** -3)


@pytest.mark.parametrize("shape", SHAPES)
def test_keys_of_large_scales_across_the_queries(shape):
    """Keys 2^40 above the others in dimensions that the queries leave out: the others' logits stay."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=36)
    s["q"][..., d // 2:] = 0
    g = torch.Generator().manual_seed(4)
    for b, n in enumerate(lens):
        at = torch.arange(0, n, 3)
        x = torch.randn(len(at), d, generator=g)
        x[:, :d // 2] = 0
        set_codes(s, "k", b, at, x)
        set_bytes(s, "k", b, at, torch.full((len(at), Hkv), 167))
    go(s, new, lens, 0.1, fine=2.0 ** -4)


@pytest.mark.parametrize("shape", SHAPES)
def test_a_nan_value_of_no_weight(shape):
    """A value row whose scale byte is 255 is NaN for every row that sees it, its weight 0 in fp32 or not."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=37)
    u = torch.ones(d)
    s["q"] = torch.ones_like(s["q"])
    want = run(s, scale=1.0, max_q=max(new))
    for b in range(len(new)):
        set_codes(s, "k", b, [5], -16 * u[None])
        set_bytes(s, "k", b, [5], torch.full((1, Hkv), 127))
        set_bytes(s, "v", b, [5], torch.full((1, Hkv), 255))
    o, lse = run(s, scale=1.0, max_q=max(new))
    assert bool(o.isnan().all()) and bool(lse.isfinite().all()) and bool(want[0].isfinite().all())


@pytest.mark.parametrize("shape", SHAPES)
def test_queries_near_the_largest_over_the_smallest_keys(shape):
    """Elements of 2^126 against rows of scale byte 0 and up: logits of ordinary size, whose parts do not fit fp32."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=38)
    g = torch.Generator().manual_seed(5)
    s["q"] = (torch.randn(s["q"].shape, generator=g).clamp(-2, 2).double() * 2.0 ** 126).bfloat16().to(DEV)
    for b, n in enumerate(lens):
        set_codes(s, "k", b, torch.arange(n), torch.randn(n, d, generator=g))
        set_bytes(s, "k", b, torch.arange(n), torch.randint(0, 4, (n, Hkv), generator=g))
    go(s, new, lens, 0.125)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_logits_of_minus_infinity(shape, wide):
    """Over keys so small, with queries so small but for an infinite element, that the factor of the products is under fp32: a
    row of such logits alone is empty, and a key without one is all that another row sees."""
    new, lens, Hq, Hkv, d = shape
    s = q8_inputs(new, lens, Hq, Hkv, d, 16, seed=40)
    s["q"] = torch.zeros_like(s["q"])
    s["q"][..., 0] = -math.inf
    s["q"][:, 1::2, 0] = -1e-30
    for b, n in enumerate(lens):
        x = torch.ones(n, d)
        set_codes(s, "k", b, torch.arange(n), x)
        set_bytes(s, "k", b, torch.arange(n), torch.full((n, Hkv), 60) + (20 * (torch.arange(n) % 2)[:, None] if wide else 0))
    ofa.device_error_flags()
    o, lse = run(s, scale=0.1, max_q=max(new))
    assert ofa.device_error_flags() == 0
    assert bool((lse[:, 0::2] == -math.inf).all()) and bool((o[:, 0::2].contiguous().view(torch.int16) == 0).all())
    check_visible(o[:, 1::2], lse[:, 1::2], dict(s, q=s["q"][:, 1::2].contiguous()), new, lens, True, 0.1)


@pytest.mark.parametrize("shape", [SHAPES[0], SHAPES[3], SHAPES[5]])
def test_large_hidden_keys_behind_a_prefix(shape):
    """Side by side and one after the other; a prefix's own values 2^35 above or below the own keys'."""
    new, lens, Hq, Hkv, d = shape
    for up in (35, -35):
        s, groups = inputs(new, lens, [500], [0, sum(new)], Hq, Hkv, d, 16, True, seed=39)
        pg = s["pt"][0].long()
        b = s["vs"].view(torch.uint8)[pg].int()
        s["vs"].view(torch.uint8)[pg] = torch.where(b == 255, b, b + up).to(torch.uint8)
        for i, n in enumerate(lens):
            set_bytes(s, "v", i, [n - 1], bytes_at(s, "v", i, [n - 1]).cpu().int() + 60)
        o, lse = run_prefix(s, scale=0.1, max_q=max(new))
        check_visible(o, lse, s, new, lens, True, 0.1, groups, [500], what=f"up {up}")

"""Attention over codes whose scales lie far apart: what a row does not see, or gives no weight, does not touch it, and what it
does see is not lost beside it (paged_range_helpers.visible_ref)."""
import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from paged_q8_helpers import q8_inputs
from paged_range_helpers import check_visible
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

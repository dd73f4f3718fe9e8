"""The 8-bit paged cache and the shared prefixes without a GPU: structure layouts, refusals on the host,
workspace sizes, and the plain forms that the GPU tests use."""
import ctypes
import math
import shutil

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from online_softmax_fa2_gb300 import build as ofa_build
from online_softmax_fa2_gb300 import paged
from paged_q8_helpers import E4M3, E8M0, dequantise, pow2, quantise, scale_bytes
from test_abi_layout_cpu import c_layout
from test_paged_cpu import append, arr, fill, fwd
from test_paged_cpu import test_packed_blocks_are_the_mirrors as packed_block_is_the_mirror

S = ofa.Status


@pytest.fixture(scope="module")
def lib():
    ofa_build.build()
    return paged._load()


MIRRORS = [("attn_paged_scales_t", paged.PagedScales, None),
           ("attn_paged_append_q8_params_t", paged.PagedAppendQ8Params, paged._pack_append_q8),
           ("attn_paged_read_q8_params_t", paged.PagedReadQ8Params, paged._pack_read_q8),
           ("attn_paged_fwd_q8_params_t", paged.PagedFwdQ8Params, paged._pack_fwd_q8),
           ("attn_paged_prefix_params_t", paged.PagedPrefixParams, paged._pack_prefix)]


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("struct,cls,pack", MIRRORS)
def test_ctypes_mirrors_match_the_header(tmp_path, struct, cls, pack):
    got = c_layout(tmp_path, struct, [name for name, _ in cls._fields_])
    assert got["size"] == ctypes.sizeof(cls)
    for name, _ in cls._fields_:
        assert got[name] == getattr(cls, name).offset, (struct, name)
    if pack:
        packed_block_is_the_mirror(cls, pack)


def scales(**kw):
    return fill(paged.PagedScales(0x10000, 0x20000, (32, 16), (32, 16)), **kw)


def split(kw):
    sc = {k[7:]: v for k, v in kw.items() if k.startswith("scales_")}
    return {k: v for k, v in kw.items() if not k.startswith("scales_")}, scales(**sc)


def append8(**kw):
    kw, sc = split(kw)
    return paged.PagedAppendQ8Params(append(**kw), sc)


def fwd8(**kw):
    kw, sc = split(kw)
    return paged.PagedFwdQ8Params(fwd(**kw), sc)


def read8(**kw):
    kw, sc = split(kw)
    return fill(paged.PagedReadQ8Params(append().cache, sc, 0x1000, 0x2000, (256, 128), (256, 128)), **kw)


def prefix(q8=True, **kw):
    own = {k: kw.pop(k) for k in list(kw) if k in ("P", "prefix_width", "prefix_stride", "prefix_table", "prefix_lens", "cu_prefix")}
    kw, sc = split(kw)
    p = paged.PagedPrefixParams(fwd(**kw), sc if q8 else paged.PagedScales(None, None, (0, 0), (0, 0)), 1, 4, 4, 0x3000, 0x4000, 0x5000)
    return fill(p, **own)


CACHE_BAD = [
    (dict(cache_dtype=5), S.INVALID_ARG), (dict(cache_B=-1), S.INVALID_ARG), (dict(cache_Hkv=0), S.INVALID_ARG),
    (dict(cache_kv_lens=None), S.INVALID_ARG), (dict(cache_block_table=None), S.INVALID_ARG), (dict(cache_k_pages=None), S.INVALID_ARG),
    (dict(cache_v_pages=0x2008), S.MISALIGNED), (dict(cache_k_stride=arr(4096, 264, 128)), S.MISALIGNED),
    (dict(cache_v_stride=arr(0, 256, 128)), S.INVALID_ARG), (dict(cache_k_stride=arr(-4096, 256, 128)), S.INVALID_ARG),
    (dict(cache_cu_q=None, cache_T=3), S.INVALID_ARG), (dict(scales_k=None), S.INVALID_ARG), (dict(scales_v=None), S.INVALID_ARG),
    (dict(scales_k_stride=arr(-32, 16)), S.INVALID_ARG), (dict(scales_v_stride=arr(32, 0)), S.INVALID_ARG),
]
STEPS_BAD = [(dict(scales_k=0x10008), S.MISALIGNED), (dict(scales_v_stride=arr(40, 16)), S.MISALIGNED), (dict(scales_k_stride=arr(32, 8)), S.MISALIGNED)]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(Hq=0), S.INVALID_ARG), (dict(v=None), S.INVALID_ARG), (dict(q_out_stride=arr(512, 0)), S.INVALID_ARG),
    (dict(rot=8), S.UNSUPPORTED), (dict(cache_d=24), S.UNSUPPORTED), (dict(eps=-1.0), S.INVALID_ARG)])
def test_append_refuses(lib, kw, status):
    assert lib.attn_paged_append_q8(append8(**kw), None) == status, ofa.last_error()
    assert ofa.last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(k=0x1008), S.MISALIGNED), (dict(v_stride=arr(256, 0)), S.INVALID_ARG), (dict(cache_d=24), S.UNSUPPORTED),
    (dict(cache_d=0), S.INVALID_ARG), (dict(cache_d=272), S.UNSUPPORTED)])
def test_read_refuses(lib, kw, status):
    assert lib.attn_paged_read_q8(read8(**kw), None) == status, ofa.last_error()


FWD_BAD = CACHE_BAD + STEPS_BAD + [
    (dict(cache_dtype=0), S.UNSUPPORTED), (dict(cache_d=96), S.UNSUPPORTED), (dict(cache_page_size=24), S.UNSUPPORTED),
    (dict(cache_page_size=8), S.UNSUPPORTED), (dict(Hq=3), S.INVALID_ARG), (dict(Hq=130), S.UNSUPPORTED),
    (dict(causal=2), S.INVALID_ARG), (dict(scale=0.0), S.UNSUPPORTED), (dict(max_q=-1), S.INVALID_ARG), (dict(o=None), S.INVALID_ARG)]


@pytest.mark.parametrize("kw,status", FWD_BAD)
def test_fwd_refuses(lib, kw, status):
    assert lib.attn_paged_fwd_q8(fwd8(**kw), 0x10000, 1 << 40, None) == status, ofa.last_error()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("kw,status", FWD_BAD + [
    (dict(P=0), S.INVALID_ARG), (dict(P=65536), S.INVALID_ARG), (dict(prefix_width=-1), S.INVALID_ARG),
    (dict(prefix_stride=-4), S.INVALID_ARG), (dict(prefix_width=1 << 27), S.UNSUPPORTED), (dict(prefix_table=None), S.INVALID_ARG),
    (dict(prefix_lens=None), S.INVALID_ARG), (dict(P=4, cu_prefix=None), S.INVALID_ARG)])
def test_prefix_refuses(lib, kw, status, q8):
    if not q8 and any(k.startswith("scales_") for k in kw):
        return
    if not q8 and status == S.MISALIGNED and "cache_k_stride" in kw:
        kw = dict(cache_k_stride=arr(4096, 260, 128))
    assert lib.attn_paged_prefix_fwd(prefix(q8, **kw), 0x10000, 1 << 40, None) == status, ofa.last_error()


def test_null_empty_and_workspaces(lib):
    assert lib.attn_paged_append_q8(None, None) == S.INVALID_ARG
    assert lib.attn_paged_read_q8(None, None) == S.INVALID_ARG
    assert lib.attn_paged_fwd_q8(None, None, 0, None) == S.INVALID_ARG
    assert lib.attn_paged_prefix_fwd(None, None, 0, None) == S.INVALID_ARG
    assert lib.attn_paged_fwd_q8_workspace_bytes(None) == lib.attn_paged_prefix_fwd_workspace_bytes(None) == 0
    none = dict(cache_T=0, cache_B=0)
    assert lib.attn_paged_append_q8(append8(**none), None) == S.OK
    assert lib.attn_paged_read_q8(read8(**none), None) == S.OK
    assert lib.attn_paged_read_q8(read8(k=None, v=None), None) == S.OK
    assert lib.attn_paged_fwd_q8(fwd8(**none), None, 0, None) == S.OK
    assert lib.attn_paged_prefix_fwd(prefix(**none), None, 0, None) == S.OK
    assert lib.attn_paged_fwd_q8_workspace_bytes(fwd8(cache_table_width=1024)) > 0
    for q8 in (True, False):
        need = lib.attn_paged_prefix_fwd_workspace_bytes(prefix(q8))
        assert need >= 2 * 4 * (128 + 2) * 4
        assert lib.attn_paged_prefix_fwd(prefix(q8), 0x10000, need - 1, None) == S.WORKSPACE
        assert lib.attn_paged_prefix_fwd(prefix(q8), 0x10008, need, None) == S.WORKSPACE
        # a long prefix may be cut: states of its parts too
        assert lib.attn_paged_prefix_fwd_workspace_bytes(prefix(q8, prefix_width=1024)) > need
        for kw in (dict(P=0), dict(prefix_width=1 << 62), dict(cache_d=96), dict(cache_T=0)):
            assert lib.attn_paged_prefix_fwd_workspace_bytes(prefix(q8, **kw)) == 0 and ofa.last_error() == ""


def test_python_refusals_without_a_gpu():
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    c, e = torch.zeros(1, 16, 2, 64, dtype=torch.uint8), torch.zeros(1, 2, 16, dtype=torch.uint8)
    t, n = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: ofa.attn_paged_append_q8(x, x, x, c, c, e, e, t, n), lambda: ofa.attn_paged_read_q8(c, c, e, e, t, n, 1),
                 lambda: ofa.attn_paged_fwd_q8(x, c, c, e, e, t, n), lambda: ofa.attn_paged_prefix_fwd(x, c, c, t, n, t, n)):
        with pytest.raises(ValueError):
            call()


def test_the_plain_quantiser():
    """Its scales are the least that hold a row, by trying all; its codes are the nearest of all codes, ties to even."""
    codes = torch.arange(256, dtype=torch.uint8)
    value = codes.view(E4M3).double()
    fine = value.isfinite()
    g = torch.Generator().manual_seed(0)
    x = torch.randn(300, 32, generator=g) * torch.exp2(torch.randint(-140, 120, (300, 1), generator=g).float())
    x[0], x[1], x[2] = 0.0, 448.0, 1.75 * 2.0 ** -100
    c, e = quantise(x)
    e = e.view(torch.uint8).int()
    room = 448.0 * torch.exp2(torch.arange(256).double() - 127)
    amax = x.abs().amax(-1).double()
    assert torch.equal(e, (room[None] < amax[:, None]).sum(-1).int())
    got = c.view(torch.uint8).view(E4M3).double()
    target = x.double() * torch.exp2(127 - e.double())[:, None]
    dist = (target[..., None] - value[fine]).abs()
    assert torch.equal((target - got).abs(), dist.amin(-1))
    tie = (dist == dist.amin(-1, keepdim=True)).sum(-1) > 1
    assert bool(((c.view(torch.uint8) & 1) == 0)[tie & (got != 0)].all())
    back = dequantise(c, e.to(torch.uint8).view(E8M0))
    assert bool(((back - x.double()).abs() <= torch.maximum(2.0 ** -4 * x.double().abs(), pow2(e.to(torch.uint8))[:, None] * 2.0 ** -10)).all())
    z = torch.tensor([[math.nan, 1.0], [math.inf, 2.0], [math.inf, math.nan]])
    c, e = quantise(z)
    assert c.float().isnan().tolist() == [[True, False], [True, False], [True, True]]
    assert e.view(torch.uint8).tolist() == scale_bytes(torch.tensor([1.0, 2.0, 0.0])).tolist()

"""The head norms' and the paged cache's entry points without a GPU: structure layouts, refusals on
the host, workspace sizes, and the plain gradient formula against differences."""
import ctypes
import shutil

import pytest
import torch

import online_softmax_fa2_gb300 as ofa
from online_softmax_fa2_gb300 import build as ofa_build
from online_softmax_fa2_gb300 import paged
from paged_helpers import angles, norm_rope, norm_rope_bwd
from test_abi_layout_cpu import c_layout

S = ofa.Status


@pytest.fixture(scope="module")
def lib():
    ofa_build.build()
    return paged._load()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("struct,cls", [
    ("attn_qk_norm_rope_params_t", paged.NormRopeParams), ("attn_qk_norm_rope_bwd_params_t", paged.NormRopeBwdParams),
    ("attn_paged_cache_t", paged.PagedCache), ("attn_paged_append_params_t", paged.PagedAppendParams),
    ("attn_paged_fwd_params_t", paged.PagedFwdParams)])
def test_ctypes_mirrors_match_the_header(tmp_path, struct, cls):
    fields = [name for name, _ in cls._fields_]
    got = c_layout(tmp_path, struct, fields)
    assert got["size"] == ctypes.sizeof(cls)
    for name in fields:
        assert got[name] == getattr(cls, name).offset, (struct, name)


@pytest.mark.parametrize("cls,pack", [
    (paged.NormRopeParams, paged._pack_norm_rope), (paged.NormRopeBwdParams, paged._pack_norm_rope_bwd),
    (paged.PagedAppendParams, paged._pack_append), (paged.PagedFwdParams, paged._pack_fwd)])
def test_packed_blocks_are_the_mirrors(cls, pack):
    """Every field of a block packed by position reads back from the mirror laid over it."""
    def fields(c, path=()):
        for name, t in c._fields_:
            if issubclass(t, ctypes.Structure):
                yield from fields(t, path + (name,))
            else:
                yield path + (name,), t
    values, want, n = [], [], 1
    for path, t in fields(cls):
        k = t._length_ if issubclass(t, ctypes.Array) else 1
        values += list(range(n, n + k))
        want.append((path, list(range(n, n + k))))
        n += k
    p = cls.from_buffer_copy(pack(*values))
    for path, w in want:
        v = p
        for name in path:
            v = getattr(v, name)
        assert (list(v) if isinstance(v, ctypes.Array) else [v]) == w, path


def fill(p, **kw):
    for k, v in kw.items():
        if k.startswith("cache_"):
            setattr(p.cache, k[6:], v)
        elif k.startswith("fwd_"):
            setattr(p.fwd, k[4:], v)
        else:
            setattr(p, k, v)
    return p


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def rope(**kw):
    p = paged.NormRopeParams(1, 0, 2, 3, 4, 2, 128, 64, 0x1000, 0x2000, 0x3000, 0x4000, (1536, 512, 128), (768, 256, 128),
                             (1536, 512, 128), (768, 256, 128), 0x5000, 0x6000, 0x7000, 100, 64, None, (0, 0), 1e-6)
    return fill(p, **kw)


def cache():
    return paged.PagedCache(1, 16, 2, 2, 2, 128, 0x1000, 0x2000, (4096, 256, 128), (4096, 256, 128), 10, 0x3000, 4, 4,
                            0x4000, 0x5000)


def append(**kw):
    p = paged.PagedAppendParams(cache(), 4, 64, 0x1000, 0x2000, 0x3000, 0x4000, (512, 128), (256, 128), (256, 128),
                                (512, 128), 0x5000, 0x6000, 0x7000, 100, 64, None, 1e-6, 0)
    return fill(p, **kw)


def fwd(**kw):
    return fill(paged.PagedFwdParams(cache(), 1, 0.1, 4, 1, 0x1000, 0x2000, (512, 128), (512, 128), None), **kw)


ROPE_BAD = [
    (dict(dtype=2), S.INVALID_ARG), (dict(B=-1), S.INVALID_ARG), (dict(Hq=0), S.INVALID_ARG),
    (dict(d=120), S.UNSUPPORTED), (dict(d=272), S.UNSUPPORTED), (dict(d=0), S.INVALID_ARG),
    (dict(rot=24), S.UNSUPPORTED), (dict(rot=144), S.INVALID_ARG), (dict(interleaved=2), S.INVALID_ARG),
    (dict(eps=0.0), S.INVALID_ARG), (dict(eps=float("nan")), S.INVALID_ARG), (dict(q=None), S.INVALID_ARG),
    (dict(k=0x2008), S.MISALIGNED), (dict(q_stride=arr(1536, 516, 128)), S.MISALIGNED),
    (dict(wq=0x5002), S.MISALIGNED), (dict(cos_sin_rows=0), S.INVALID_ARG), (dict(cos_sin_stride=32), S.INVALID_ARG),
    (dict(cos_sin_stride=66), S.MISALIGNED), (dict(cos_sin=0x7004), S.MISALIGNED),
    (dict(k_out_stride=arr(768, 0, 128)), S.INVALID_ARG), (dict(q_stride=arr(1536, -512, 128)), S.INVALID_ARG),
    (dict(positions=0x100, positions_stride=arr(-1, 1)), S.INVALID_ARG), (dict(B=1 << 20, N=1 << 12), S.UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", ROPE_BAD)
def test_norm_rope_refuses(lib, kw, status):
    assert lib.attn_qk_norm_rope(rope(**kw), None) == status, ofa.last_error()
    assert ofa.last_error()


def test_norm_rope_null_and_empty(lib):
    assert lib.attn_qk_norm_rope(None, None) == S.INVALID_ARG
    assert lib.attn_qk_norm_rope(rope(B=0, q=None), None) == S.OK


def bwd(**kw):
    z = ((1536, 512, 128), (768, 256, 128))
    return fill(paged.NormRopeBwdParams(rope(q_out=None, k_out=None), 0x1000, 0x2000, 0x3000, 0x4000, *z, *z, 0x100, 0x200), **kw)


@pytest.mark.parametrize("kw,status", [
    (dict(fwd_d=40), S.UNSUPPORTED), (dict(dwq=None), S.INVALID_ARG), (dict(fwd_wk=None), S.INVALID_ARG),
    (dict(dq=None), S.INVALID_ARG), (dict(dk_out=0x2004), S.MISALIGNED), (dict(dq_stride=arr(1536, 512, 0)), S.INVALID_ARG),
    (dict(), S.WORKSPACE)])
def test_norm_rope_bwd_refuses(lib, kw, status):
    assert lib.attn_qk_norm_rope_bwd(bwd(**kw), None, 0, None) == status, ofa.last_error()
    if not kw:
        need = ofa.qk_norm_rope_bwd_workspace_bytes(2, 3, 4, 2, 128)
        assert need > 0 and need % 512 == 0
        assert lib.attn_qk_norm_rope_bwd(bwd(), 0x1000, need - 4, None) == S.WORKSPACE
        assert lib.attn_qk_norm_rope_bwd(bwd(), 0x1008, need, None) == S.WORKSPACE
        assert lib.attn_qk_norm_rope_bwd(None, None, 0, None) == S.INVALID_ARG


CACHE_BAD = [
    (dict(cache_dtype=5), S.INVALID_ARG), (dict(cache_B=-1), S.INVALID_ARG), (dict(cache_T=-2), S.INVALID_ARG),
    (dict(cache_B=0), S.INVALID_ARG), (dict(cache_Hkv=0), S.INVALID_ARG), (dict(cache_page_size=0), None),
    (dict(cache_kv_lens=None), S.INVALID_ARG), (dict(cache_block_table=None), S.INVALID_ARG),
    (dict(cache_k_pages=None), S.INVALID_ARG), (dict(cache_v_pages=0x2002), S.MISALIGNED),
    (dict(cache_k_stride=arr(4096, 260, 128)), S.MISALIGNED), (dict(cache_v_stride=arr(0, 256, 128)), S.INVALID_ARG),
    (dict(cache_table_width=1 << 28), S.UNSUPPORTED), (dict(cache_cu_q=None, cache_T=3), S.INVALID_ARG),
    (dict(cache_num_pages=-1), S.INVALID_ARG), (dict(q=None), S.INVALID_ARG), (dict(q=0x1008), S.MISALIGNED),
    (dict(q_stride=arr(512, 100)), S.MISALIGNED),
]


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(Hq=0), S.INVALID_ARG), (dict(v=None), S.INVALID_ARG), (dict(q_out_stride=arr(512, 0)), S.INVALID_ARG),
    (dict(rot=8), S.UNSUPPORTED), (dict(cache_d=24), S.UNSUPPORTED), (dict(eps=-1.0), S.INVALID_ARG)])
def test_append_refuses(lib, kw, status):
    st = lib.attn_paged_append(append(**kw), None)
    assert st == (S.INVALID_ARG if status is None else status), ofa.last_error()


@pytest.mark.parametrize("kw,status", CACHE_BAD + [
    (dict(cache_dtype=0), S.UNSUPPORTED), (dict(cache_d=96), S.UNSUPPORTED), (dict(cache_page_size=24), S.UNSUPPORTED),
    (dict(cache_page_size=8), S.UNSUPPORTED), (dict(Hq=3), S.INVALID_ARG), (dict(Hq=130), S.UNSUPPORTED),
    (dict(causal=2), S.INVALID_ARG), (dict(scale=0.0), S.UNSUPPORTED), (dict(scale=float("inf")), S.INVALID_ARG),
    (dict(max_q=-1), S.INVALID_ARG), (dict(o=None), S.INVALID_ARG), (dict(o_stride=arr(0, 128)), S.INVALID_ARG)])
def test_paged_fwd_refuses(lib, kw, status):
    st = lib.attn_paged_fwd(fwd(**kw), 0x10000, 1 << 40, None)
    assert st == (S.UNSUPPORTED if status is None else status), ofa.last_error()


def test_paged_null_and_empty(lib):
    assert lib.attn_paged_append(None, None) == S.INVALID_ARG
    assert lib.attn_paged_fwd(None, None, 0, None) == S.INVALID_ARG
    assert lib.attn_paged_fwd_workspace_bytes(None) == 0
    assert lib.attn_paged_append(append(cache_T=0, cache_B=0), None) == S.OK
    assert lib.attn_paged_fwd(fwd(cache_T=0, cache_B=0), None, 0, None) == S.OK


def test_workspace_of_invalid_or_overlong_arguments_is_none(lib):
    need = lambda **kw: lib.attn_paged_fwd_workspace_bytes(fwd(**kw))  # noqa: E731
    assert need(cache_table_width=1024) > 0
    for kw in (dict(cache_table_width=-5), dict(cache_table_width=1 << 62), dict(cache_B=0), dict(cache_T=0),
               dict(cache_T=1 << 29, cache_B=1, cache_table_width=1 << 20), dict(max_q=-1), dict(cache_d=96)):
        assert need(**kw) == 0, kw
        assert ofa.last_error() == ""
    # more tokens a sequence than there are tokens: as many as there are
    assert need(max_q=2, cache_table_width=1024) == need(max_q=(1 << 63) - 1, cache_table_width=1024) > 0


@pytest.mark.parametrize("page,width,fits", [(16, (1 << 27) - 16, True), (16, (1 << 27) - 15, False), (16, (1 << 27) - 1, False),
                                             (256, (1 << 23) - 1, True), (128, (1 << 24) - 1, False), (1 << 30, 1, True)])
def test_a_table_whose_last_tile_ends_past_an_int_is_refused(lib, page, width, fits):
    # the tile that holds key 2^31 - 17 ends at 2^31
    kw = dict(cache_page_size=page, cache_table_width=width, cache_table_stride=width)
    assert (lib.attn_paged_fwd_workspace_bytes(fwd(**kw)) > 0) == fits
    if not fits:
        assert lib.attn_paged_fwd(fwd(**kw), 0x10000, 1 << 40, None) == S.UNSUPPORTED
        assert "table_width" in ofa.last_error()


def test_python_refusals_without_a_gpu():
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ofa.attn_qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        ofa.attn_paged_fwd(x[0], x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("inter", [False, True])
def test_the_plain_gradient_is_the_difference_quotient(inter):
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(3, 2, 32, generator=g).double(), torch.randn(3, 2, 32, generator=g).double()
    w = (1 + 0.2 * torch.randn(32, generator=g)).double()
    cs = angles(3, 16)[:, None]
    import paged_helpers as h
    h.HALF[torch.float64] = 0.0
    try:
        loss = lambda a, b: float((norm_rope(a, b, cs, inter, 1e-6)[0] * dy).sum())  # noqa: E731
        dx, dw, _, _ = norm_rope_bwd(x, dy, w, cs, inter, 1e-6)
        e = 1e-6
        for at in [(0, 0, 0), (1, 1, 9), (2, 0, 15), (2, 1, 31)]:
            step = torch.zeros_like(x)
            step[at] = e
            assert abs((loss(x + step, w) - loss(x - step, w)) / (2 * e) - float(dx[at])) < 1e-7
        for c in (0, 7, 20):
            step = torch.zeros_like(w)
            step[c] = e
            assert abs((loss(x, w + step) - loss(x, w - step)) / (2 * e) - float(dw[c])) < 1e-7
    finally:
        del h.HALF[torch.float64]

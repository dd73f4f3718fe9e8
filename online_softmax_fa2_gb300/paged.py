"""Head norms with the position rotation, and the paged key/value cache: binding over the C ABI.

    q2, k2 = attn_qk_norm_rope(q, k, wq, wk, cos_sin)                    # before attn_fwd
    dq, dk, dwq, dwk = attn_qk_norm_rope_bwd(q, k, dq2, dk2, wq, wk, cos_sin)
    q2 = attn_paged_append(q, k, v, k_pages, v_pages, block_table, kv_lens, cu_q, wq=..., wk=..., cos_sin=...)
    o, lse = attn_paged_fwd(q2, k_pages, v_pages, block_table, kv_lens, cu_q, max_q=...)

Shapes: q [B, N, Hq, d] and k [B, N, Hkv, d] for the first two; packed tokens q [T, Hq, d], k and
v [T, Hkv, d] for the others, with k_pages and v_pages [num_pages, page_size, Hkv, d],
block_table int32 [B, width], kv_lens int32 [B] (the new tokens included) and cu_q int32 [B + 1]
(None: T / B new tokens in every sequence).  Any strides with the last dimension contiguous.
The names' kernels and rules are those of include/attn.h.

A call runs on torch's current stream of the tensors' device, which need not be the current
device; ``stream`` is as calling under ``torch.cuda.stream(stream)``: it has to be a stream of that
device, and what the call allocates is that stream's.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

import online_softmax_fa2_gb300 as _ofa

__all__ = ["attn_qk_norm_rope", "attn_qk_norm_rope_bwd", "attn_paged_append", "attn_paged_fwd",
           "paged_fwd_workspace_bytes", "qk_norm_rope_bwd_workspace_bytes"]

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
_S2, _S3 = _i64 * 2, _i64 * 3


class NormRopeParams(ctypes.Structure):
    """Mirror of attn_qk_norm_rope_params_t (include/attn.h)."""
    _fields_ = [("dtype", _i32), ("interleaved", _i32),
                ("B", _i64), ("N", _i64), ("Hq", _i64), ("Hkv", _i64), ("d", _i64), ("rot", _i64),
                ("q", _vp), ("k", _vp), ("q_out", _vp), ("k_out", _vp),
                ("q_stride", _S3), ("k_stride", _S3), ("q_out_stride", _S3), ("k_out_stride", _S3),
                ("wq", _vp), ("wk", _vp),
                ("cos_sin", _vp), ("cos_sin_rows", _i64), ("cos_sin_stride", _i64),
                ("positions", _vp), ("positions_stride", _S2), ("eps", _f32)]


class NormRopeBwdParams(ctypes.Structure):
    """Mirror of attn_qk_norm_rope_bwd_params_t (include/attn.h)."""
    _fields_ = [("fwd", NormRopeParams),
                ("dq_out", _vp), ("dk_out", _vp), ("dq", _vp), ("dk", _vp),
                ("dq_out_stride", _S3), ("dk_out_stride", _S3), ("dq_stride", _S3), ("dk_stride", _S3),
                ("dwq", _vp), ("dwk", _vp)]


class PagedCache(ctypes.Structure):
    """Mirror of attn_paged_cache_t (include/attn.h)."""
    _fields_ = [("dtype", _i32), ("page_size", _i32),
                ("B", _i64), ("T", _i64), ("Hkv", _i64), ("d", _i64),
                ("k_pages", _vp), ("v_pages", _vp), ("k_stride", _S3), ("v_stride", _S3), ("num_pages", _i64),
                ("block_table", _vp), ("table_width", _i64), ("table_stride", _i64),
                ("kv_lens", _vp), ("cu_q", _vp)]


class PagedAppendParams(ctypes.Structure):
    """Mirror of attn_paged_append_params_t (include/attn.h)."""
    _fields_ = [("cache", PagedCache), ("Hq", _i64), ("rot", _i64),
                ("q", _vp), ("k", _vp), ("v", _vp), ("q_out", _vp),
                ("q_stride", _S2), ("k_stride", _S2), ("v_stride", _S2), ("q_out_stride", _S2),
                ("wq", _vp), ("wk", _vp),
                ("cos_sin", _vp), ("cos_sin_rows", _i64), ("cos_sin_stride", _i64),
                ("positions", _vp), ("eps", _f32), ("interleaved", _i32)]


class PagedFwdParams(ctypes.Structure):
    """Mirror of attn_paged_fwd_params_t (include/attn.h)."""
    _fields_ = [("cache", PagedCache), ("causal", _i32), ("scale", _f32), ("Hq", _i64), ("max_q", _i64),
                ("q", _vp), ("o", _vp), ("q_stride", _S2), ("o_stride", _S2), ("lse", _vp)]


def _packer(cls):
    """struct.Struct of a mirror's fields in order (nested ones in place), C alignment: filling it takes
    a third of the time that filling the mirror takes, and a small call is as long as its host side."""
    def fmt(c):
        out = ""
        for _, t in c._fields_:
            if issubclass(t, ctypes.Structure):
                out += fmt(t) + "0q"
            elif issubclass(t, ctypes.Array):
                out += "q" * t._length_
            else:
                out += {_i32: "i", _i64: "q", _vp: "P", _f32: "f"}[t]
        return out
    pack = struct.Struct("@" + fmt(cls) + "0q")
    assert pack.size == ctypes.sizeof(cls)
    return pack.pack


_pack_norm_rope, _pack_norm_rope_bwd = _packer(NormRopeParams), _packer(NormRopeBwdParams)
_pack_append, _pack_fwd = _packer(PagedAppendParams), _packer(PagedFwdParams)


class _Block:
    """Argument type of a parameter block: packed bytes, or a mirror."""
    @classmethod
    def from_param(cls, v):
        return v if v is None or isinstance(v, bytes) else ctypes.byref(v)


_lib = None


def _load():
    global _lib
    if _lib is None:
        lib = _ofa.load()
        size, params = ctypes.c_size_t, _Block
        for name, args, res in (
                ("attn_qk_norm_rope", [params, _vp], _i32),
                ("attn_qk_norm_rope_bwd_workspace_bytes", [_i64] * 5, size),
                ("attn_qk_norm_rope_bwd", [params, _vp, size, _vp], _i32),
                ("attn_paged_append", [params, _vp], _i32),
                ("attn_paged_fwd_workspace_bytes", [params], size),
                ("attn_paged_fwd", [params, _vp, size, _vp], _i32)):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, res
        _lib = lib
    return _lib


_DTYPES = {torch.float32: _ofa.F32, torch.bfloat16: _ofa.BF16}
_BAD = "{} must be {} {} on cuda:{} with the last dimension contiguous, got {} {} with strides {} on {}"


def _need(t, name, shape, dtype, dev):
    """The address and the strides of t, checked to be a tensor of that shape and dtype on device number
    dev with its last dimension contiguous."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or st[-1] != 1 and shape[-1] > 1:
        raise ValueError(_BAD.format(name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape), st, t.device))
    return t.data_ptr(), st


def _device(q, dim):
    dev = q.get_device()
    if dev < 0:
        raise ValueError("every tensor must be on a CUDA device (there is no CPU path)")
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}: use torch.float32 or torch.bfloat16")
    if q.dim() != dim:
        raise ValueError(f"q must be {dim}-D, got {tuple(q.shape)}")
    return dev


def _bytes(dev, fn, *args):
    """Workspace bytes fn(*args) for device number dev (they depend on its multiprocessors)."""
    if torch._C._cuda_getDevice() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _call(dev, fn, *args):
    """fn(*args, torch's current stream of device number dev) with that device current."""
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st:
        raise _ofa.AttnError(st, _ofa.last_error())


def _on(stream, q, fn, *args):
    """fn(*args) with stream, of q's device, as torch's current one: what it allocates belongs to it."""
    if stream.device != q.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {q.device}")
    with torch.cuda.stream(stream):
        return fn(*args)


def _weight(w, name, d, dtype, dev):
    return 0 if w is None else _need(w, name, (d,), dtype, dev)[0]


def _angles(cos_sin, dev):
    """(pointer, rows, row stride, rot) of the angle table [P, rot], or zeros."""
    if cos_sin is None:
        return 0, 0, 0, 0
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be float32 [positions, rot]")
    rows, rot = shape = cos_sin.shape
    p, st = _need(cos_sin, "cos_sin", shape, torch.float32, dev)
    return p, rows, st[0], rot


def _norm_rope_params(q, k, qo, ko, wq, wk, cos_sin, positions, eps, interleaved):
    """The values of attn_qk_norm_rope_params_t, in order."""
    dev, dt = _device(q, 4), q.dtype
    B, N, Hq, d = shape = q.shape
    Hkv = k.shape[2] if k.dim() == 4 else -1
    kshape = (B, N, Hkv, d)
    kp, (k0, k1, k2, _) = _need(k, "k", kshape, dt, dev)
    qp, (q0, q1, q2, _) = _need(q, "q", shape, dt, dev)
    qop = kop = a0 = a1 = a2 = b0 = b1 = b2 = pos = p0 = p1 = 0
    if qo is not None:
        qop, (a0, a1, a2, _) = _need(qo, "q_out", shape, dt, dev)
        kop, (b0, b1, b2, _) = _need(ko, "k_out", kshape, dt, dev)
    cs, rows, row, rot = _angles(cos_sin, dev)
    if positions is not None:
        if positions.dtype != torch.int32 or positions.get_device() != dev:
            raise ValueError(f"positions must be int32 on cuda:{dev}")
        positions = positions.expand(B, N)
        pos, (p0, p1) = positions.data_ptr(), positions.stride()
    return (_DTYPES[dt], 1 if interleaved else 0, B, N, Hq, Hkv, d, rot, qp, kp, qop, kop, q0, q1, q2, k0, k1, k2, a0, a1,
            a2, b0, b1, b2, _weight(wq, "wq", d, dt, dev), _weight(wk, "wk", d, dt, dev), cs, rows, row, pos, p0, p1, eps)


def attn_qk_norm_rope(q, k, wq=None, wk=None, cos_sin=None, positions=None, eps=1e-6, interleaved=False, q_out=None,
                      k_out=None, stream=None):
    """RMS norm of every head of q [B, N, Hq, d] and k [B, N, Hkv, d] (weights wq, wk [d]; None: no
    norm) and the rotation by the angle table cos_sin (float32 [P, rot], cos then sin; None: none)
    at positions (int32 [B, N] or broadcast; None: 0 .. N - 1).  Pairs are (c, c + rot/2), or
    (2c, 2c + 1) when interleaved.  Returns (q_out, k_out), which may be given, q and k
    themselves included.  See include/attn.h, attn_qk_norm_rope."""
    if stream is not None:
        return _on(stream, q, attn_qk_norm_rope, q, k, wq, wk, cos_sin, positions, eps, interleaved, q_out, k_out)
    lib = _load()
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    p = _pack_norm_rope(*_norm_rope_params(q, k, q_out, k_out, wq, wk, cos_sin, positions, eps, interleaved))
    _call(q.get_device(), lib.attn_qk_norm_rope, p)
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(B, N, Hq, Hkv, d) -> int:
    """Bytes of workspace attn_qk_norm_rope_bwd needs on the current device (with any weight)."""
    return int(_load().attn_qk_norm_rope_bwd_workspace_bytes(B, N, Hq, Hkv, d))


def attn_qk_norm_rope_bwd(q, k, dq_out, dk_out, wq=None, wk=None, cos_sin=None, positions=None, eps=1e-6,
                          interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of attn_qk_norm_rope: q, k are its inputs, dq_out, dk_out the gradients of its
    outputs.  Returns (dq, dk, dwq, dwk); dq and dk may be given (dq_out and dk_out themselves
    included), dwq and dwk are float32 [d], None where the weight is."""
    if stream is not None:
        return _on(stream, q, attn_qk_norm_rope_bwd, q, k, dq_out, dk_out, wq, wk, cos_sin, positions, eps, interleaved, dq,
                   dk, workspace)
    lib = _load()
    f = _norm_rope_params(q, k, None, None, wq, wk, cos_sin, positions, eps, interleaved)
    dev, dt, cuda = q.get_device(), q.dtype, q.device
    B, N, Hq, Hkv, d = f[2:7]
    if dq is None:
        dq = torch.empty(q.shape, dtype=dt, device=cuda)
    if dk is None:
        dk = torch.empty(k.shape, dtype=dt, device=cuda)
    dwq = dwk = None
    if wq is not None:
        dwq = torch.empty(d, dtype=torch.float32, device=cuda)
    if wk is not None:
        dwk = torch.empty(d, dtype=torch.float32, device=cuda)
    if workspace is None and (dwq is not None or dwk is not None):
        workspace = torch.empty(_bytes(dev, lib.attn_qk_norm_rope_bwd_workspace_bytes, B, N, Hq, Hkv, d),
                                dtype=torch.uint8, device=cuda)
    sq, sk = (B, N, Hq, d), (B, N, Hkv, d)
    dqop, (a0, a1, a2, _) = _need(dq_out, "dq_out", sq, dt, dev)
    dkop, (b0, b1, b2, _) = _need(dk_out, "dk_out", sk, dt, dev)
    dqp, (c0, c1, c2, _) = _need(dq, "dq", sq, dt, dev)
    dkp, (d0, d1, d2, _) = _need(dk, "dk", sk, dt, dev)
    p = _pack_norm_rope_bwd(*f, dqop, dkop, dqp, dkp, a0, a1, a2, b0, b1, b2, c0, c1, c2, d0, d1, d2,
                            0 if dwq is None else dwq.data_ptr(), 0 if dwk is None else dwk.data_ptr())
    wsp, wsn = _workspace(workspace, dev)
    _call(dev, lib.attn_qk_norm_rope_bwd, p, wsp, wsn)
    return dq, dk, dwq, dwk


def _workspace(t, dev):
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _cache(T, d, dt, dev, k_pages, v_pages, block_table, kv_lens, cu_q):
    """The values of attn_paged_cache_t, in order."""
    if k_pages.dim() != 4 or k_pages.shape[3] != d:
        raise ValueError(f"k_pages must be [num_pages, page_size, Hkv, {d}], got {tuple(k_pages.shape)}")
    pages, page, Hkv, _ = shape = k_pages.shape
    kp, (k0, k1, k2, _) = _need(k_pages, "k_pages", shape, dt, dev)
    vp, (v0, v1, v2, _) = _need(v_pages, "v_pages", shape, dt, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, width]")
    B, width = table = block_table.shape
    bt, (row, _) = _need(block_table, "block_table", table, torch.int32, dev)
    lens, _ = _need(kv_lens, "kv_lens", (B,), torch.int32, dev)
    cu = 0 if cu_q is None else _need(cu_q, "cu_q", (B + 1,), torch.int32, dev)[0]
    return _DTYPES[dt], page, B, T, Hkv, d, kp, vp, k0, k1, k2, v0, v1, v2, pages, bt, width, row, lens, cu


def attn_paged_append(q, k, v, k_pages, v_pages, block_table, kv_lens, cu_q=None, wq=None, wk=None, cos_sin=None,
                      positions=None, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Writes the new tokens' keys (normed and rotated as by attn_qk_norm_rope) and values to their
    slots of the paged cache, in place, and returns the normed and rotated queries.  kv_lens
    counts the new tokens; positions (int32 [T]; None: each token's place in its sequence) are
    the rotation's.  See include/attn.h, attn_paged_append."""
    if stream is not None:
        return _on(stream, q, attn_paged_append, q, k, v, k_pages, v_pages, block_table, kv_lens, cu_q, wq, wk, cos_sin,
                   positions, eps, interleaved, q_out)
    lib = _load()
    dev, dt = _device(q, 3), q.dtype
    T, Hq, d = shape = q.shape
    if q_out is None:
        q_out = torch.empty(shape, dtype=dt, device=q.device)
    c = _cache(T, d, dt, dev, k_pages, v_pages, block_table, kv_lens, cu_q)
    sk = (T, c[4], d)
    cs, rows, row, rot = _angles(cos_sin, dev)
    qp, (q0, q1, _) = _need(q, "q", shape, dt, dev)
    kp, (k0, k1, _) = _need(k, "k", sk, dt, dev)
    vp, (v0, v1, _) = _need(v, "v", sk, dt, dev)
    op, (o0, o1, _) = _need(q_out, "q_out", shape, dt, dev)
    p = _pack_append(*c, Hq, rot, qp, kp, vp, op, q0, q1, k0, k1, v0, v1, o0, o1, _weight(wq, "wq", d, dt, dev),
                     _weight(wk, "wk", d, dt, dev), cs, rows, row,
                     0 if positions is None else _need(positions, "positions", (T,), torch.int32, dev)[0], eps,
                     1 if interleaved else 0)
    _call(dev, lib.attn_paged_append, p)
    return q_out


def _paged_fwd_params(q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, causal, scale, out, lse):
    """attn_paged_fwd_params_t, packed."""
    dev, dt = _device(q, 3), q.dtype
    T, Hq, d = shape = q.shape
    c = _cache(T, d, dt, dev, k_pages, v_pages, block_table, kv_lens, cu_q)
    lp = op = o0 = o1 = 0
    if out is not None:
        op, (o0, o1, _) = _need(out, "out", shape, dt, dev)
    if lse is not None:
        lp, _ = _need(lse, "lse", (T, Hq), torch.float32, dev)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    if max_q is None:
        max_q = 0 if cu_q is not None else T // c[2] if c[2] else 0
    qp, (q0, q1, _) = _need(q, "q", shape, dt, dev)
    return _pack_fwd(*c, 1 if causal else 0, 1.0 / math.sqrt(d) if scale is None else scale, Hq, max_q,
                     qp, op, q0, q1, o0, o1, lp)


def paged_fwd_workspace_bytes(q, k_pages, v_pages, block_table, kv_lens, cu_q=None, max_q=None, causal=True) -> int:
    """Bytes of workspace attn_paged_fwd needs for these arguments (the lengths' values play no part)."""
    p = _paged_fwd_params(q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, causal, None, None, None)
    return int(_bytes(q.get_device(), _load().attn_paged_fwd_workspace_bytes, p))


def attn_paged_fwd(q, k_pages, v_pages, block_table, kv_lens, cu_q=None, max_q=None, causal=True, scale=None,
                   workspace=None, out=None, lse=None, stream=None):
    """Attention of the packed new tokens q [T, Hq, d] over the paged cache, one or many per
    sequence in one call; query head h reads key/value head h // (Hq // Hkv).  causal aligns the
    new tokens to the end of their sequences.  max_q: the largest number of new tokens of any
    sequence, where the caller knows it (it chooses the kernel; the results hold without it, but a
    long chunk among single tokens then takes about twice the time).
    Returns (o [T, Hq, d], lse [T, Hq]).  See include/attn.h, attn_paged_fwd."""
    if stream is not None:
        return _on(stream, q, attn_paged_fwd, q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, causal, scale, workspace,
                   out, lse)
    lib = _load()
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    p = _paged_fwd_params(q, k_pages, v_pages, block_table, kv_lens, cu_q, max_q, causal, scale, out, lse)
    dev = q.get_device()
    if workspace is None:
        n = _bytes(dev, lib.attn_paged_fwd_workspace_bytes, p)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    wsp, wsn = _workspace(workspace, dev)
    _call(dev, lib.attn_paged_fwd, p, wsp, wsn)
    return out, lse

"""Cases of the operators around the attention itself, each in a plain form and through the library:

  qk_norm_rope       RMS norm of every query and key head and the position rotation, one pass
  qk_norm_rope_bwd   its gradients: dq, dk and the two norm weights'
  paged_append       the same pass over the packed new tokens of a ragged batch, the keys and
                     values going to their slots of a paged cache
  paged_fwd          attention of the new tokens (one or many per sequence) over the paged cache,
                     with query heads that share key/value heads

The plain form is elementary torch arithmetic in fp32, rounded once at the end; the exact form
is written apart from it in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# --------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a training forward at the causal training shape: q and k of every token
        dict(name="qk_train_b4_n2048_h16_d128", op="norm_rope", B=4, N=2048, Hq=16, Hkv=16, d=128, rot=128,
             dtype="bf16", inter=False),
        # a small odd one in fp32: half of each head rotated in adjacent pairs, shared kv heads
        dict(name="qk_f32_b3_n517_h6_d64", op="norm_rope", B=3, N=517, Hq=6, Hkv=2, d=64, rot=32,
             dtype="f32", inter=True),
        # the backward at the training shape
        dict(name="qk_bwd_b4_n2048_h16_d128", op="norm_rope_bwd", B=4, N=2048, Hq=16, Hkv=16, d=128, rot=128,
             dtype="bf16", inter=False),
        # the backward of a long odd sequence with shared kv heads, adjacent pairs, part of the head rotated
        dict(name="qk_bwd_b2_n4095_h24_8_d128", op="norm_rope_bwd", B=2, N=4095, Hq=24, Hkv=8, d=128, rot=64,
             dtype="bf16", inter=True),
        # one decode step of 64 sequences: one new token each into the cache
        dict(name="append_b64_one", op="append", seqs=64, new_max=1, len_max=1024, Hq=32, Hkv=8, d=128, rot=128,
             page=64, dtype="bf16", inter=False, lens_seed=5),
        # a serving step with prompts of many lengths
        dict(name="append_b12_ragged", op="append", seqs=12, new_max=2048, len_max=4096, Hq=32, Hkv=8, d=128, rot=128,
             page=16, dtype="bf16", inter=False, lens_seed=6),
        # the smallest call: one token of one short sequence
        dict(name="paged_one_n300", op="paged", seqs=1, new_max=1, len_max=300, full=True, Hq=8, Hkv=2, d=64, page=16,
             causal=True, lens_seed=1),
        # decode of a full batch, ragged lengths; the batch is padded to its size with three idle places
        dict(name="paged_decode_b64_l8192", op="paged", seqs=64, new_max=1, len_max=8192, full=False, Hq=32, Hkv=8,
             d=128, page=64, causal=True, lens_seed=2, idle=3),
        # decode of one very long sequence
        dict(name="paged_decode_b1_l131072", op="paged", seqs=1, new_max=1, len_max=131072, full=True, Hq=32, Hkv=8,
             d=128, page=128, causal=True, lens_seed=3),
        # several drafted tokens a sequence checked at once, every query head with a key head of its own
        dict(name="paged_verify_b32_nq4", op="paged", seqs=32, new_max=4, len_max=4096, full=False, Hq=16, Hkv=16, d=64,
             page=16, causal=True, lens_seed=4),
        # a mixed serving step: prompt chunks beside single tokens, seven query heads a key head
        dict(name="paged_mixed_b16_l4096", op="paged", seqs=16, new_max=512, len_max=4096, full=False, Hq=28, Hkv=4,
             d=128, page=32, causal=True, lens_seed=7),
        # the next chunk of a long prompt
        dict(name="paged_chunk_2048_of_18432", op="paged", seqs=1, new_max=2048, len_max=18432, full=True, Hq=32, Hkv=8,
             d=128, page=64, causal=True, lens_seed=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "paged", "paged", "paged"])
    inter = rng.random() < 0.3
    while True:
        if op in ("norm_rope", "norm_rope_bwd"):
            d = rng.choice([64, 128, 128, 192, 256])
            Hkv = rng.choice([1, 2, 4, 5, 8, 16])
            c = dict(op=op, B=_log(rng, 1, 8), N=_log(rng, 1, 8192), Hq=Hkv * rng.choice([1, 2, 3, 4, 7, 8]), Hkv=Hkv,
                     d=d, rot=rng.choice([d, d, d // 2]), dtype=rng.choice(["bf16", "bf16", "f32"]), inter=inter)
            if c["B"] * c["N"] * (c["Hq"] + Hkv) * d * (2 if c["dtype"] == "bf16" else 4) > 4 * 2048 * 32 * 128 * 2:
                continue
        elif op == "append":
            d, Hkv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
            c = dict(op=op, seqs=_log(rng, 1, 64), new_max=_log(rng, 1, 2048), len_max=_log(rng, 16, 4096),
                     Hq=Hkv * rng.choice([1, 2, 4, 5, 7, 8]), Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]),
                     page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), inter=inter,
                     lens_seed=rng.randrange(1 << 20))
            if work(c)["bytes"] > 1.5e8 or c["seqs"] * c["len_max"] * Hkv * d > 64 * 1024 * 8 * 128:
                continue
        else:
            Hkv = rng.choice([1, 2, 3, 4, 8, 16])
            one = rng.random() < 0.4
            c = dict(op=op, seqs=_log(rng, 1, 64), new_max=1 if one else _log(rng, 2, 2048), len_max=_log(rng, 1, 32768),
                     full=rng.random() < 0.3, Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), Hkv=Hkv,
                     d=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]), causal=rng.random() < 0.85,
                     lens_seed=rng.randrange(1 << 20))
            if one and c["seqs"] > 4 and rng.random() < 0.5:
                c["idle"] = rng.randint(1, 3)
            w = work(c)
            if w["bytes"] > 1e9 or w["flops"] > 5.5e11:
                continue
            # the plain form works on sequences padded to the longest
            if c["seqs"] * c["new_max"] * c["Hq"] * c["len_max"] > 1.2e9 or c["seqs"] * c["len_max"] * Hkv * c["d"] > 6e8:
                continue
        return c


def _lens(c):
    """(new tokens, key length after them) of every sequence of a serving case."""
    r = random.Random(c["lens_seed"])
    new, lens = [], []
    for s in range(c["seqs"]):
        if c.get("full") or c["seqs"] == 1:
            n, q = c["len_max"], c["new_max"]
        else:
            n = r.randint(1, c["len_max"])
            # serving batches mix single tokens with prompt chunks
            q = 1 if c["new_max"] == 1 or r.random() < 0.4 else r.randint(1, c["new_max"])
            if s == 0:
                n, q = c["len_max"], c["new_max"]
        new.append(min(q, n))
        lens.append(n)
    for s in range(c.get("idle", 0)):  # a place without a sequence: one token, no keys
        new[1 + s], lens[1 + s] = 1, 0
    return new, lens


def work(c):
    es = 4 if c.get("dtype") == "f32" else 2
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        x = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"]
        m = 2 if c["op"] == "norm_rope" else 3
        return {"bytes": m * x * es + 4 * c["N"] * c["rot"] + 4 * c["B"] * c["N"], "flops": (8 if m == 2 else 20) * x}
    new, lens = _lens(c)
    T = sum(new)
    if c["op"] == "append":
        x = T * (c["Hq"] + 2 * c["Hkv"]) * c["d"]
        return {"bytes": 2 * x * es + 4 * T * c["rot"], "flops": 8 * x}
    pairs = 0
    for q, n in zip(new, lens):
        pairs += q * n - (q * (q - 1) // 2 if c["causal"] else 0)
    return {"bytes": sum(lens) * c["Hkv"] * 2 * c["d"] * 2 + T * c["Hq"] * (2 * c["d"] * 2 + 4),
            "flops": 4 * c["d"] * c["Hq"] * pairs}


# -------------------------------------------------------------------------------- the inputs

def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _angles(P, rot):
    """The table a model keeps: cos then sin of position times frequency, formed in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(c=c)
    d = c["d"]
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        dt = DT[c["dtype"]]
        for n, h in (("q", c["Hq"]), ("k", c["Hkv"])):
            s[n] = _randn(g, c["B"], c["N"], h, d, dtype=dt)
            s["w" + n] = (1 + 0.2 * _randn(g, d)).to(dt)
            if c["op"] == "norm_rope_bwd":
                s["d" + n] = _randn(g, c["B"], c["N"], h, d, dtype=dt)
        s["cs"] = _angles(c["N"], c["rot"])
        return s
    new, lens = _lens(c)
    T, ps, B = sum(new), c["page"], c["seqs"]
    dt = DT[c.get("dtype", "bf16")]
    width = max(-(-n // ps) for n in lens)
    used = sum(-(-n // ps) for n in lens)
    pages = used + 3  # a few that no sequence holds
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    at, rows = 0, []
    for n in lens:
        k = -(-n // ps)
        rows.append(torch.cat([perm[at:at + k], torch.full((width - k,), -1, dtype=torch.int32, device="cuda")]))
        at += k
    s["bt"] = torch.stack(rows)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([0] + list(_cumsum(new)), dtype=torch.int32, device="cuda")
    s["max_q"], s["max_n"] = max(new), max(lens)
    s["kp"] = _randn(g, pages, ps, c["Hkv"], d, dtype=dt)
    s["vp"] = _randn(g, pages, ps, c["Hkv"], d, dtype=dt)
    s["q"] = _randn(g, T, c["Hq"], d, dtype=dt)
    if c["op"] == "append":
        s["k"] = _randn(g, T, c["Hkv"], d, dtype=dt)
        s["v"] = _randn(g, T, c["Hkv"], d, dtype=dt)
        s["wq"] = (1 + 0.2 * _randn(g, d)).to(dt)
        s["wk"] = (1 + 0.2 * _randn(g, d)).to(dt)
        s["cs"] = _angles(max(lens), c["rot"])
    return s


def _cumsum(x):
    t = 0
    for v in x:
        t += v
        yield t


# ------------------------------------------------------------------------------ one pass each

def run(state):
    s, c = state, state["c"]
    if own:
        import online_softmax_fa2_gb300 as ofa
        if c["op"] == "norm_rope":
            return ofa.attn_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cs"], eps=EPS, interleaved=c["inter"])
        if c["op"] == "norm_rope_bwd":
            return ofa.attn_qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["cs"], eps=EPS,
                                             interleaved=c["inter"])
        if c["op"] == "append":
            qo = ofa.attn_paged_append(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"],
                                       wq=s["wq"], wk=s["wk"], cos_sin=s["cs"], eps=EPS, interleaved=c["inter"])
            return qo, s["kp"], s["vp"]
        return ofa.attn_paged_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["cu"], max_q=s["max_q"],
                                  causal=c["causal"])
    if c["op"] == "norm_rope":
        cs = s["cs"][None, :, None, :]
        return (_norm_rope(s["q"], s["wq"], cs, c["inter"]), _norm_rope(s["k"], s["wk"], cs, c["inter"]))
    if c["op"] == "norm_rope_bwd":
        cs = s["cs"][None, :, None, :]
        dq, dwq = _norm_rope_bwd(s["q"], s["dq"], s["wq"], cs, c["inter"])
        dk, dwk = _norm_rope_bwd(s["k"], s["dk"], s["wk"], cs, c["inter"])
        return dq, dk, dwq, dwk
    if c["op"] == "append":
        b, i, pos = _places(s)
        cs = s["cs"][pos][:, None, :]
        qo = _norm_rope(s["q"], s["wq"], cs, c["inter"])
        ps = c["page"]
        page = s["bt"][b, pos // ps].long()
        s["kp"][page, pos % ps] = _norm_rope(s["k"], s["wk"], cs, c["inter"])
        s["vp"][page, pos % ps] = s["v"]
        return qo, s["kp"], s["vp"]
    return _paged(s, c)


def _rotate(y, cs, inter, sign):
    """The first rot dimensions of y turned by sign times the angles whose cos and sin cs holds."""
    r = cs.shape[-1]
    co, si = cs[..., :r // 2], sign * cs[..., r // 2:]
    if inter:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        t = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        t = torch.cat([a * co - b * si, a * si + b * co], -1)
    return torch.cat([t, y[..., r:]], -1)


def _norm_rope(x, w, cs, inter):
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(y, cs, inter, 1.0).to(x.dtype)


def _norm_rope_bwd(x, dy, w, cs, inter):
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    t = _rotate(dy.float(), cs, inter, -1.0)
    n = f * r
    # the sum over every token and head, rows first and then the rest, so that it keeps its digits
    dw = (t * n).sum(2).sum(1).sum(0)
    gt = t * w.float()
    dx = r * (gt - n * (gt * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _places(s):
    """Sequence, index within the new tokens and position in the sequence of every packed token."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    return b, i, s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _paged(s, c):
    Hq, Hkv, d, ps, mq, mn = c["Hq"], c["Hkv"], c["d"], c["page"], s["max_q"], s["max_n"]
    G, B = Hq // Hkv, c["seqs"]
    bt = s["bt"].long().clamp(min=0)

    def gathered(p):  # [B, Hkv, keys, d]
        return p[bt].reshape(B, -1, Hkv, d)[:, :mn].permute(0, 2, 1, 3).float()

    lens, cu = s["lens"].long(), s["cu"].long()
    nq = cu[1:] - cu[:-1]
    iq = torch.arange(mq, device="cuda")
    at = (cu[:-1, None] + iq).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().reshape(B, mq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, mq * G, d)
    x = torch.matmul(q * (1.0 / math.sqrt(d)), gathered(s["kp"]).transpose(-1, -2)).view(B, Hkv, mq, G, mn)
    last = (lens[:, None] - nq[:, None] + iq) if c["causal"] else (lens[:, None] - 1).expand(B, mq)
    hidden = torch.arange(mn, device="cuda") > last.clamp(max=mn)[:, :, None]
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(m.clamp(min=-1e30)))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, mq * G, mn), gathered(s["vp"])).view(B, Hkv, mq, G, d)
    o = o / l.clamp(min=1e-30)
    lse = (m + torch.log(l)).squeeze(-1)
    b, i, _ = _places(s)
    o = o.permute(0, 2, 1, 3, 4)[b, i].reshape(-1, Hq, d).to(s["q"].dtype)
    return o, lse.permute(0, 2, 1, 3)[b, i].reshape(-1, Hq)


# --------------------------------------------------------------------------- in 64 bits, apart

def _exact_row(x, w, ang, inter):
    """ang [..., rot / 2]: the angles as complex numbers cos + i sin."""
    x, w = x.double(), w.double()
    y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    h = ang.shape[-1]
    z = torch.complex(y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if inter else torch.complex(y[..., :h], y[..., h:2 * h])
    z = torch.view_as_real(z * ang)
    z = z.flatten(-2) if inter else torch.cat([z[..., 0], z[..., 1]], -1)
    return torch.cat([z, y[..., 2 * h:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] != "paged":
        cs = s["cs"].double()
        ang = torch.complex(cs[:, :c["rot"] // 2], cs[:, c["rot"] // 2:])
    if c["op"] == "norm_rope":
        a = ang[None, :, None]
        return tuple(_exact_row(s[n], s["w" + n], a, c["inter"]) for n in "qk")
    if c["op"] == "norm_rope_bwd":
        a, got = ang[None, :, None], []
        for n in "qk":
            x, w = s[n].double().requires_grad_(), s["w" + n].double().requires_grad_()
            got.append(torch.autograd.grad(_exact_row(x, w, a, c["inter"]), [x, w], s["d" + n].double()))
        return got[0][0], got[1][0], got[0][1], got[1][1]
    new, lens = _lens(c)
    ps = c["page"]
    if c["op"] == "append":
        qs, kp, vp, at = [], s["kp"].double(), s["vp"].double(), 0
        for b, (nq, n) in enumerate(zip(new, lens)):
            pos = torch.arange(n - nq, n, device="cuda")
            a = ang[pos][:, None]
            sl = slice(at, at + nq)
            qs.append(_exact_row(s["q"][sl], s["wq"], a, c["inter"]))
            pg = s["bt"][b, pos // ps].long()
            kp[pg, pos % ps] = _exact_row(s["k"][sl], s["wk"], a, c["inter"])
            vp[pg, pos % ps] = s["v"][sl].double()
            at += nq
        return torch.cat(qs), kp, vp
    if work(c)["flops"] > 1.5e12:
        return None
    G = c["Hq"] // c["Hkv"]
    os, ls, at = [], [], 0
    for b, (nq, n) in enumerate(zip(new, lens)):
        pg = s["bt"][b, :-(-n // ps)].long()
        o = torch.empty(nq, c["Hq"], c["d"], dtype=torch.float64, device="cuda")
        l = torch.empty(nq, c["Hq"], dtype=torch.float64, device="cuda")
        see = torch.ones(nq, n, dtype=torch.bool, device="cuda")
        if c["causal"]:
            see = see.tril(n - nq)
        for h in range(c["Hkv"]):
            K = s["kp"][pg, :, h].reshape(-1, c["d"])[:n].double()
            V = s["vp"][pg, :, h].reshape(-1, c["d"])[:n].double()
            for r in range(0, nq, 1024):  # in pieces, so that the weights of a long chunk fit
                e = min(nq, r + 1024)
                Q = s["q"][at + r:at + e, h * G:(h + 1) * G].double()
                X = torch.einsum("qgd,kd->gqk", Q, K) / math.sqrt(c["d"])
                X = torch.where(see[None, r:e], X, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                L = torch.logsumexp(X, -1)
                o[r:e, h * G:(h + 1) * G] = torch.einsum("gqk,kd->qgd", torch.exp(X - L[..., None]), V)
                l[r:e, h * G:(h + 1) * G] = L.T
        os.append(o)
        ls.append(l)
        at += nq
    return torch.cat(os), torch.cat(ls)

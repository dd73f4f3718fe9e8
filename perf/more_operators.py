"""Cases of the 8-bit paged cache and of the attention that shares a prefix, each in a plain form and
through the library:

  append8   head norms and rotation of the packed new tokens, their keys and values quantised into a
            paged cache: e4m3 codes with one power-of-two scale a row
  read8     rows of that cache read back as packed bf16 or fp32
  paged8    attention of the new tokens over that cache
  prefix    attention of a batch whose sequences share a long prefix, in bf16 or 8 bits

The plain form is elementary torch arithmetic in fp32, rounded once at the end; the exact form is
written apart from it in 64 bits (of the codes that an append writes it gives the value before the
rounding to e4m3).
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


# --------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of 64 sequences: one new token each into the cache
        dict(name="append8_b64_one", op="append8", seqs=64, new_max=1, len_max=1024, Hq=32, Hkv=8, d=128, rot=128,
             page=64, hf=True, dtype="bf16", inter=False, lens_seed=5),
        # a serving step with prompts of many lengths
        dict(name="append8_b12_ragged", op="append8", seqs=12, new_max=2048, len_max=4096, Hq=32, Hkv=8, d=128, rot=128,
             page=16, hf=False, dtype="bf16", inter=False, lens_seed=6),
        # a short sequence read back, to be moved elsewhere
        dict(name="read8_one_n300", op="read8", seqs=1, len_max=300, Hkv=2, d=64, page=16, hf=False, dtype="f32", lens_seed=1),
        # a ragged batch read back whole
        dict(name="read8_b24_l8192", op="read8", seqs=24, len_max=8192, Hkv=8, d=128, page=64, hf=True, dtype="bf16",
             lens_seed=9),
        # the smallest attention: one token of one short sequence
        dict(name="paged8_one_n300", op="paged8", seqs=1, new_max=1, len_max=300, full=True, Hq=8, Hkv=2, d=64, page=16,
             hf=False, causal=True, lens_seed=1),
        # decode of a full batch, ragged lengths, three idle places
        dict(name="paged8_decode_b64_l8192", op="paged8", seqs=64, new_max=1, len_max=8192, full=False, Hq=32, Hkv=8,
             d=128, page=64, hf=True, causal=True, lens_seed=2, idle=3),
        # a mixed serving step: prompt chunks beside single tokens, seven query heads a key head
        dict(name="paged8_mixed_b16_l4096", op="paged8", seqs=16, new_max=512, len_max=4096, full=False, Hq=28, Hkv=4,
             d=128, page=32, hf=False, causal=True, lens_seed=7),
        # the next chunk of a long prompt
        dict(name="paged8_chunk_2048_of_18432", op="paged8", seqs=1, new_max=2048, len_max=18432, full=True, Hq=32, Hkv=8,
             d=128, page=64, hf=True, causal=True, lens_seed=8),
        # two answers to one short prompt
        dict(name="prefix_b2_p300", op="prefix", q8=False, seqs=2, groups=1, prefix_max=300, new_max=1, len_max=40, Hq=8,
             Hkv=2, d=64, page=16, hf=False, causal=True, lens_seed=3),
        # decode of a full batch behind one system prompt
        dict(name="prefix_decode_b64_p8192", op="prefix", q8=False, seqs=64, groups=1, prefix_max=8192, new_max=1,
             len_max=1024, Hq=32, Hkv=8, d=128, page=64, hf=False, causal=True, lens_seed=4),
        # drafted tokens behind two prompts, 8-bit cache
        dict(name="prefix8_b32_2x4096_nq4", op="prefix", q8=True, seqs=32, groups=2, prefix_max=4096, new_max=4, len_max=1024,
             Hq=16, Hkv=4, d=128, page=32, hf=True, causal=True, lens_seed=10),
        # questions of many lengths about one document
        dict(name="prefix_chunks_b8_p4096", op="prefix", q8=False, seqs=8, groups=1, prefix_max=4096, new_max=512,
             len_max=768, Hq=28, Hkv=4, d=128, page=64, hf=False, causal=True, lens_seed=11),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append8", "read8", "paged8", "paged8", "prefix", "prefix"])
    page, hf, seed = rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.randrange(1 << 20)
    while True:
        if op == "append8":
            d, Hkv = rng.choice([64, 128, 128, 192, 256]), rng.choice([1, 2, 4, 8])
            c = dict(op=op, seqs=_log(rng, 1, 64), new_max=_log(rng, 1, 2048), len_max=_log(rng, 16, 4096),
                     Hq=Hkv * rng.choice([1, 2, 4, 5, 7, 8]), Hkv=Hkv, d=d, rot=rng.choice([d, d, d // 2]), page=page, hf=hf,
                     dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), inter=rng.random() < 0.3, lens_seed=seed)
            if work(c)["bytes"] > 1.5e8 or c["seqs"] * c["len_max"] * Hkv * d > 64 * 1024 * 8 * 128:
                continue
        elif op == "read8":
            c = dict(op=op, seqs=_log(rng, 1, 64), len_max=_log(rng, 1, 16384), Hkv=rng.choice([1, 2, 3, 4, 8, 16]),
                     d=rng.choice([64, 128, 128, 192, 256]), page=page, hf=hf, dtype=rng.choice(["bf16", "bf16", "f32"]),
                     lens_seed=seed)
            if work(c)["bytes"] > 6e8:
                continue
        else:
            Hkv = rng.choice([1, 2, 3, 4, 8, 16])
            one = rng.random() < 0.4
            c = dict(op=op, seqs=_log(rng, 1, 64), new_max=1 if one else _log(rng, 2, 2048), len_max=_log(rng, 1, 32768),
                     full=rng.random() < 0.3, Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8]), Hkv=Hkv,
                     d=rng.choice([64, 128, 128]), page=page, hf=hf, causal=rng.random() < 0.85, lens_seed=seed)
            if op == "prefix":
                c.update(q8=rng.random() < 0.4, groups=rng.choice([1, 1, 2, 3]), prefix_max=_log(rng, 64, 16384))
                c["len_max"] = min(c["len_max"], 4096)
                c["groups"] = min(c["groups"], c["seqs"])
            if one and c["seqs"] > 4 and rng.random() < 0.5:
                c["idle"] = rng.randint(1, 3)
            w, keys = work(c), c["len_max"] + c.get("prefix_max", 0)
            if w["bytes"] > 1e9 or w["flops"] > 5.5e11:
                continue
            # the plain form works on sequences padded to the longest
            if c["seqs"] * c["new_max"] * c["Hq"] * keys > 1.2e9 or c["seqs"] * keys * Hkv * c["d"] > 6e8:
                continue
        return c


def _lens(c):
    """(new tokens, own keys after them) of every sequence."""
    r = random.Random(c["lens_seed"])
    most = c.get("new_max", c["len_max"])
    new, lens = [], []
    for s in range(c["seqs"]):
        if c.get("full") or c["seqs"] == 1:
            n, q = c["len_max"], most
        else:
            n = r.randint(1, c["len_max"])
            # serving batches mix single tokens with prompt chunks
            q = 1 if most == 1 or r.random() < 0.4 else r.randint(1, most)
            if s == 0:
                n, q = c["len_max"], most
        new.append(n if c["op"] == "read8" else min(q, n))
        lens.append(n)
    for s in range(c.get("idle", 0)):  # a place without a sequence: one token, no keys of its own
        new[1 + s], lens[1 + s] = 1, 0
    return new, lens


def _groups(c):
    """(prefix lengths, first sequence of each group and the number of sequences)."""
    r = random.Random(c["lens_seed"] + 1)
    P, B = c["groups"], c["seqs"]
    cuts = sorted(r.sample(range(1, B), P - 1))
    return [c["prefix_max"]] + [r.randint(c["prefix_max"] // 2, c["prefix_max"]) for _ in range(P - 1)], [0] + cuts + [B]


def work(c):
    es = 4 if c.get("dtype") == "f32" else 2
    new, lens = _lens(c)
    T, d, Hkv = sum(new), c["d"], c["Hkv"]
    if c["op"] == "read8":
        return {"bytes": 2 * T * Hkv * (d + 1 + d * es), "flops": 2 * T * Hkv * d}
    if c["op"] == "append8":
        return {"bytes": T * (2 * c["Hq"] * d * es + 2 * Hkv * (d * es + d + 1)) + 4 * T * c["rot"],
                "flops": 8 * T * (c["Hq"] + 2 * Hkv) * d}
    pairs, keys = 0, sum(lens)
    for q, n in zip(new, lens):
        pairs += q * n - (q * (q - 1) // 2 if c["causal"] else 0)
    if c["op"] == "prefix":
        plen, cut = _groups(c)
        keys += sum(plen)
        for p, n in enumerate(plen):
            pairs += n * sum(new[cut[p]:cut[p + 1]])
    row = d + 1 if c["op"] == "paged8" or c["q8"] else 2 * d
    return {"bytes": keys * Hkv * 2 * row + T * c["Hq"] * (2 * d * 2 + 4), "flops": 4 * d * c["Hq"] * pairs}


# -------------------------------------------------------------------------------- the inputs

def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _angles(P, rot):
    """The table a model keeps: cos then sin of position times frequency, formed in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _cumsum(x):
    t = 0
    for v in x:
        t += v
        yield t


def _table(lens, perm, ps):
    width, at, rows = max(1, max(-(-n // ps) for n in lens)), 0, []
    for n in lens:
        k = -(-n // ps)
        rows.append(torch.cat([perm[at:at + k], torch.full((width - k,), -1, dtype=torch.int32, device="cuda")]))
        at += k
    return torch.stack(rows)


def _ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(c=c)
    d, Hkv, ps = c["d"], c["Hkv"], c["page"]
    new, lens = _lens(c)
    T = sum(new)
    plen, cut = _groups(c) if c["op"] == "prefix" else ([], [])
    pages = sum(-(-n // ps) for n in lens + plen) + 3  # a few that no sequence holds
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["bt"] = _table(lens, perm, ps)
    s["lens"] = _ints(lens)
    s["cu"] = _ints([0] + list(_cumsum(new)))
    s["T"], s["max_q"], s["max_n"] = T, max(new), max(lens)
    if plen:
        s["pt"] = _table(plen, perm[sum(-(-n // ps) for n in lens):], ps)
        s["plens"], s["max_p"] = _ints(plen), max(plen)
        s["pcu"] = _ints([0] + list(_cumsum(sum(new[a:b]) for a, b in zip(cut, cut[1:]))))
    for n in "kv":
        # rows of one size before the norm, and of many after it
        x = _randn(g, pages, Hkv, ps, d) * torch.exp(0.5 * _randn(g, pages, Hkv, ps, 1))
        if c["op"] != "prefix" or c["q8"]:
            x, e = _quantise(x)
            s[n + "s"] = e
        else:
            x = x.to(torch.bfloat16)
        s[n + "p"] = x.permute(0, 2, 1, 3) if c["hf"] else x.permute(0, 2, 1, 3).contiguous()
    if c["op"] == "read8":
        return s
    dt = DT[c.get("dtype", "bf16")]
    s["q"] = _randn(g, T, c["Hq"], d, dtype=dt)
    if c["op"] == "append8":
        s["k"] = _randn(g, T, Hkv, d, dtype=dt)
        s["v"] = (_randn(g, T, Hkv, d) * torch.exp(0.5 * _randn(g, T, Hkv, 1))).to(dt)
        s["wq"] = (1 + 0.2 * _randn(g, d)).to(dt)
        s["wk"] = (1 + 0.2 * _randn(g, d)).to(dt)
        s["cs"] = _angles(max(lens), c["rot"])
    return s


# ------------------------------------------------------------------------------ one pass each

def run(state):
    s, c = state, state["c"]
    if own:
        import online_softmax_fa2_gb300 as ofa
        if c["op"] == "append8":
            qo = ofa.attn_paged_append_q8(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"],
                                          s["cu"], wq=s["wq"], wk=s["wk"], cos_sin=s["cs"], eps=EPS, interleaved=c["inter"])
            return qo, s["kp"], s["vp"], s["ks"], s["vs"]
        if c["op"] == "read8":
            return ofa.attn_paged_read_q8(s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["T"], s["cu"],
                                          dtype=DT[c["dtype"]])
        if c["op"] == "paged8":
            return ofa.attn_paged_fwd_q8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["bt"], s["lens"], s["cu"],
                                         max_q=s["max_q"], causal=c["causal"])
        return ofa.attn_paged_prefix_fwd(s["q"], s["kp"], s["vp"], s["bt"], s["lens"], s["pt"], s["plens"], s["cu"], s["pcu"],
                                         max_q=s["max_q"], causal=c["causal"], k_scales=s.get("ks"), v_scales=s.get("vs"))
    if c["op"] == "append8":
        b, i, pos = _places(s)
        cs = s["cs"][pos][:, None, :]
        qo = _norm_rope(s["q"], s["wq"], cs, c["inter"]).to(s["q"].dtype)
        ps = c["page"]
        page, slot = s["bt"][b, pos // ps].long(), pos % ps
        for n, x in (("k", _norm_rope(s["k"], s["wk"], cs, c["inter"])), ("v", s["v"].float())):
            code, e = _quantise(x)
            s[n + "p"].view(torch.uint8)[page, slot] = code.view(torch.uint8)
            s[n + "s"].view(torch.uint8)[page, :, slot] = e.view(torch.uint8)
        return qo, s["kp"], s["vp"], s["ks"], s["vs"]
    if c["op"] == "read8":
        b, i, pos = _places(s)
        page, slot = s["bt"][b, pos // c["page"]].long(), pos % c["page"]
        return tuple((s[n + "p"].view(torch.uint8)[page, slot].view(E4M3).float()
                      * _pow2(s[n + "s"].view(torch.uint8)[page, :, slot])[..., None]).to(DT[c["dtype"]]) for n in "kv")
    return _attention(s, c)


def _pow2(e):
    """2 to the power of the bytes e less 127."""
    return torch.ldexp(torch.ones((), device=e.device), e.int() - 127)


def _quantise(x):
    """(codes, scales) of the rows of x, fp32: the smallest power of two that brings a row within 448."""
    a = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(a > 0, (e - 9 + (m > 0.875).int()).clamp(min=-127), -127)
    return torch.ldexp(x, -e[..., None]).to(E4M3), (e + 127).to(torch.uint8).view(E8M0)


def _rotate(y, cs, inter):
    """The first rot dimensions of y turned by the angles whose cos and sin cs holds."""
    r = cs.shape[-1]
    co, si = cs[..., :r // 2], cs[..., r // 2:]
    if inter:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        t = torch.stack([a * co - b * si, a * si + b * co], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        t = torch.cat([a * co - b * si, a * si + b * co], -1)
    return torch.cat([t, y[..., r:]], -1)


def _norm_rope(x, w, cs, inter):
    f = x.float()
    return _rotate(f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w.float(), cs, inter)


def _places(s):
    """Sequence, index within the new tokens and position in the sequence of every packed token."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    return b, i, s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _attention(s, c):
    """Every sequence over the prefix of its group (if any) and its own keys, padded to the longest."""
    Hq, Hkv, d, mq, mn = c["Hq"], c["Hkv"], c["d"], s["max_q"], s["max_n"]
    G, B = Hq // Hkv, c["seqs"]

    def rows(n, table, most):  # [sequences, Hkv, keys, d]
        t = table.long().clamp(min=0)
        x = s[n + "p"]
        if n + "s" in s:
            x = x.view(torch.uint8)[t].view(E4M3).float() * _pow2(s[n + "s"].view(torch.uint8)[t]).transpose(2, 3)[..., None]
        else:
            x = x[t].float()
        return x.reshape(t.shape[0], -1, Hkv, d)[:, :most].permute(0, 2, 1, 3)

    lens, cu = s["lens"].long(), s["cu"].long()
    nq = cu[1:] - cu[:-1]
    iq = torch.arange(mq, device="cuda")
    at = (cu[:-1, None] + iq).clamp(max=s["T"] - 1)
    last = (lens[:, None] - nq[:, None] + iq) if c["causal"] else (lens[:, None] - 1).expand(B, mq)
    hidden = torch.arange(mn, device="cuda") > last.clamp(max=mn)[:, :, None]
    K, V = rows("k", s["bt"], mn), rows("v", s["bt"], mn)
    if "pt" in s:
        group = torch.searchsorted(s["pcu"].long(), cu[:-1], right=True) - 1
        K = torch.cat([rows("k", s["pt"], s["max_p"])[group], K], 2)
        V = torch.cat([rows("v", s["pt"], s["max_p"])[group], V], 2)
        far = torch.arange(s["max_p"], device="cuda") >= s["plens"].long()[group][:, None]
        hidden = torch.cat([far[:, None].expand(B, mq, -1), hidden], 2)
    n = K.shape[2]
    q = s["q"][at].float().reshape(B, mq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, mq * G, d)
    x = torch.matmul(q * (1.0 / math.sqrt(d)), K.transpose(-1, -2)).view(B, Hkv, mq, G, n)
    x.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(m.clamp(min=-1e30)))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, mq * G, n), V).view(B, Hkv, mq, G, d) / l.clamp(min=1e-30)
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


def _keys(s, n, table, length):
    """The first keys or values of one row of a table, [length, Hkv, d] in 64 bits."""
    ps = s["c"]["page"]
    pg = table[:-(-length // ps)].long()
    if n + "s" not in s:
        return s[n + "p"][pg].double().flatten(0, 1)[:length]
    code = s[n + "p"].view(torch.uint8)[pg].view(E4M3).double()
    e = s[n + "s"].view(torch.uint8)[pg].view(E8M0).double().transpose(1, 2)
    return (code * e[..., None]).flatten(0, 1)[:length]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    new, lens = _lens(c)
    ps = c["page"]
    if c["op"] == "read8":
        return tuple(torch.cat([_keys(s, n, s["bt"][b], lens[b]) for b in range(c["seqs"])]) for n in "kv")
    if c["op"] == "append8":
        cs = s["cs"].double()
        ang = torch.complex(cs[:, :c["rot"] // 2], cs[:, c["rot"] // 2:])
        qs, at = [], 0
        got = {n: s[n].double().contiguous() for n in ("kp", "vp", "ks", "vs")}
        for b, (nq, n) in enumerate(zip(new, lens)):
            pos = torch.arange(n - nq, n, device="cuda")
            a = ang[pos][:, None]
            sl = slice(at, at + nq)
            qs.append(_exact_row(s["q"][sl], s["wq"], a, c["inter"]))
            pg = s["bt"][b, pos // ps].long()
            for t, x in (("k", _exact_row(s["k"][sl], s["wk"], a, c["inter"])), ("v", s["v"][sl].double())):
                m, e = torch.frexp(x.abs().amax(-1) / 448)  # in [0.5, 1): a power of two is its own, what lies above takes the next
                e = torch.where(m == 0.5, e - 1, e).double().clamp(min=-127)
                got[t + "p"][pg, pos % ps] = x * torch.exp2(-e)[..., None]
                got[t + "s"][pg, :, pos % ps] = torch.exp2(e)
            at += nq
        return torch.cat(qs), got["kp"], got["vp"], got["ks"], got["vs"]
    if work(c)["flops"] > 1.5e12:
        return None
    G = c["Hq"] // c["Hkv"]
    plen, cut = _groups(c) if c["op"] == "prefix" else ([0], [0, c["seqs"]])
    os, ls, at = [], [], 0
    for p, np in enumerate(plen):
        PK, PV = ((_keys(s, n, s["pt"][p], np) if np else s[n + "p"][:0, 0].double()) for n in "kv")
        for b in range(cut[p], cut[p + 1]):
            nq, n = new[b], lens[b]
            K, V = (torch.cat([P, _keys(s, t, s["bt"][b], n)]) for P, t in ((PK, "k"), (PV, "v")))
            o = torch.empty(nq, c["Hq"], c["d"], dtype=torch.float64, device="cuda")
            l = torch.empty(nq, c["Hq"], dtype=torch.float64, device="cuda")
            see = torch.ones(nq, np + n, dtype=torch.bool, device="cuda")
            if c["causal"]:
                see = see.tril(np + n - nq)
            see[:, :np] = True
            for h in range(c["Hkv"]):
                for r in range(0, nq, 1024):  # in pieces, so that the weights of a long chunk fit
                    e = min(nq, r + 1024)
                    Q = s["q"][at + r:at + e, h * G:(h + 1) * G].double()
                    X = torch.einsum("qgd,kd->gqk", Q, K[:, h]) / math.sqrt(c["d"])
                    X = torch.where(see[None, r:e], X, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                    L = torch.logsumexp(X, -1)
                    W = torch.exp(X - torch.where(L.isinf(), 0.0, L)[..., None])
                    o[r:e, h * G:(h + 1) * G] = torch.einsum("gqk,kd->qgd", W, V[:, h])
                    l[r:e, h * G:(h + 1) * G] = L.T
            os.append(o)
            ls.append(l)
            at += nq
    return torch.cat(os), torch.cat(ls)

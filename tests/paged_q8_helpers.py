"""Plain 64-bit forms of the 8-bit paged cache, of attention over it and of attention behind shared
prefixes, and the bounds their outputs are held to."""
import math

import torch

from paged_helpers import U, check, paged_inputs

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
CODE_HALF = 2.0 ** -4   # half a step of e4m3, relative
FP16_HALF = 2.0 ** -11  # half a step of fp16, relative; 2^-25 below 2^-14


def scale_bytes(amax):
    """The least e >= 0 with amax <= 448 * 2^(e - 127), int."""
    m, x = torch.frexp(amax.double())  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).int() + 127
    return torch.where(amax > 0, e.clamp(min=0), torch.zeros_like(e))


def pow2(e):
    """2^(e - 127) of scale bytes, 64 bits; 255 is NaN."""
    e = e.view(torch.uint8).int()
    return torch.where(e == 255, math.nan, torch.ldexp(torch.ones_like(e, dtype=torch.float64), e - 127))


def quantise(x):
    """(codes, scale bytes) of the rows of x on the CPU: what the append writes for x as it is."""
    x = x.float()
    x = torch.where(x.isinf(), torch.tensor(math.nan), x)
    e = scale_bytes(torch.where(x.isnan(), torch.zeros(()), x.abs()).amax(-1))
    return torch.ldexp(x.double(), 127 - e[..., None]).float().to(E4M3), e.to(torch.uint8).view(E8M0)


def dequantise(codes, scales):
    """Rows in 64 bits: codes [..., d], scales [...]."""
    return codes.view(torch.uint8).view(E4M3).double() * pow2(scales)[..., None]


def q8_inputs(new, lens, Hq, Hkv, d, page, seed=0, device="cuda", heads_first=True, spread=0.5, poison=True, **kw):
    """paged_inputs with the cache in 8 bits; rows of many sizes (exp of spread times a normal), slots that no
    sequence holds NaN in codes and in scales."""
    s = paged_inputs(new, lens, Hq, Hkv, d, page, seed=seed, device="cpu", poison=poison, dtype=torch.bfloat16, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    out = dict(q=s["q"].to(device), bt=s["bt"].to(device), lens=s["lens"].to(device), cu=s["cu"].to(device))
    for n in "kv":
        x = s[n + "p"].float()
        size = torch.exp((spread if n == "v" else min(spread, 0.5)) * torch.randn(x.shape[:3], generator=g))
        c, e = quantise(x * size[..., None])
        e = torch.where(x[..., 0].isnan(), torch.tensor(255, dtype=torch.uint8), e.view(torch.uint8)).view(E8M0)
        c = c.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) if heads_first else c
        out[n + "p"] = c.to(device)
        out[n + "s"] = e.view(torch.uint8).transpose(1, 2).contiguous().view(E8M0).to(device)
    return out


def _rows(s, n, table, length):
    """The first keys or values of a table's row, [length, Hkv, d] in 64 bits, and their scales [length, Hkv]."""
    pages = s[n + "p"].cpu()
    Hkv, d = pages.shape[2:]
    pg = table[:-(-length // pages.shape[1])].long()
    if n + "s" not in s:
        return pages[pg].reshape(-1, Hkv, d)[:length].double(), None
    e = s[n + "s"].cpu().view(torch.uint8)[pg].transpose(1, 2).reshape(-1, Hkv)[:length]
    c = pages.view(torch.uint8)[pg].reshape(-1, Hkv, d)[:length]
    return dequantise(c, e), e


def attention_ref(s, new, lens, causal, scale, groups=None, plens=()):
    """(o, lse, bound of o, bound of lse) [T, Hq, ...] in 64 bits on the CPU; groups: the prefix of every packed
    token (-1: none), of lengths plens in s["pt"].

    Over a bf16 cache the bound is paged_helpers.paged_ref's.  Over codes (exact in the products) a weight
    w = p 2^(f - F) is rounded to fp16: 2^-11 of it, or 2^-25 where it lies under 2^-14 (2^-13 here, as the
    weights are held to a maximum that may lag), which reaches the output as that times code 2^(F - 127)
    over a row sum of at least 1; values 2^15 and more under the largest scale lose bits of their own (2^-25
    of that scale a weight of 1).  The output's rounding (2^-8), the logits' sums ((d + 8) U sum |q k|, twice for
    the row sum) and the exponentials (2^-18) as there.  A prefix's state is merged in fp32: inside the 2^-18."""
    q, bt = s["q"].cpu(), s["bt"].cpu()
    T, Hq, d = q.shape
    Hkv = s["kp"].shape[2]
    G, q8 = Hq // Hkv, "ks" in s
    o, bo = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    lse, bl = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    t = 0
    for b, (nq, n) in enumerate(zip(new, lens)):
        own = [_rows(s, x, bt[b], n) for x in "kv"]
        at = torch.arange(t, t + nq)
        t += nq
        for p in sorted(set(groups[at].tolist())) if groups is not None else [-1]:
            mine = torch.arange(nq) if groups is None else (groups[at] == p).nonzero()[:, 0]
            L = 0 if p < 0 else plens[p]
            pre = [_rows(s, x, s["pt"].cpu()[p], L) for x in "kv"] if L else None
            K, V = (torch.cat([pre[i][0], own[i][0]]) if L else own[i][0] for i in (0, 1))
            if len(K) == 0 or len(mine) == 0:
                continue
            see = torch.ones(len(mine), L + n, dtype=torch.bool)
            if causal:
                see[:, L:] = torch.arange(n)[None, :] <= mine[:, None] + (n - nq)
            rep = lambda x: x.repeat_interleave(G, 1)  # noqa: E731
            Q = q[at[mine]].double()
            X = torch.einsum("ihd,jhd->hij", Q, rep(K)) * scale
            E = torch.einsum("ihd,jhd->hij", Q.abs(), rep(K).abs()) * scale
            E = torch.where(see, E, torch.zeros(()).double())
            X = X.masked_fill(~see, -math.inf)
            M = X.amax(-1, keepdim=True)
            M = torch.where(M.isinf(), torch.zeros(()).double(), M)
            W = torch.exp(X - M)
            l = W.sum(-1, keepdim=True)
            safe = torch.where(l > 0, l, torch.ones(()).double())
            oo = (torch.einsum("hij,jhd->hid", W, rep(V)) / safe).transpose(0, 1)
            A = (torch.einsum("hij,jhd->hid", W, rep(V).abs()) / safe).transpose(0, 1)
            dx = ((d + 8) * U * E.amax(-1)).T
            slack = 2 * dx[..., None] + 2.0 ** -18
            if q8:
                e = torch.cat([pre[1][1], own[1][1]]) if L else own[1][1]
                F = e.int().amax(0)  # of each key head
                unit = torch.ldexp(torch.ones_like(F, dtype=torch.float64), F - 127)
                w = W * torch.ldexp(torch.ones_like(e, dtype=torch.float64), e.int() - F).T.repeat_interleave(G, 0)[:, None]
                codes = torch.where(rep(V) == 0, torch.zeros(()).double(), rep(V / pow2(e.contiguous())[..., None]).abs())
                low = ((w < 2.0 ** -13) & see).double() * 2.0 ** -25
                lost = torch.einsum("hij,jhd->hid", low, codes) + W.sum(-1)[..., None] * 2.0 ** -24 * ((e.int() < F - 14).any(0).double().repeat_interleave(G)[:, None, None])
                lost = (lost * unit.repeat_interleave(G)[:, None, None] / safe).transpose(0, 1)
                bound = 2.0 ** -8 * oo.abs() + FP16_HALF * A + lost + slack * A
            else:
                bound = 2.0 ** -8 * (oo.abs() + A) + slack * A
            o[at[mine]], bo[at[mine]] = oo, bound
            lse[at[mine]] = (M[..., 0] + torch.log(l[..., 0])).T
            bl[at[mine]] = 2 * dx + 2.0 ** -18 * (1 + lse[at[mine]].abs().nan_to_num(0, 0, 0))
    return o, lse, bo, bl


def check_attention(o, lse, s, new, lens, causal, scale, groups=None, plens=(), what=""):
    ro, rl, bo, bl = attention_ref(s, new, lens, causal, scale, groups, plens)
    check(o, ro, bo, what + " o")
    empty = torch.isinf(rl)
    lc = lse.cpu().double()
    assert bool((lc[empty] == -math.inf).all()), f"{what}: empty rows must have lse = -inf"
    assert bool((o.cpu().view(torch.int16)[empty] == 0).all()), f"{what}: empty rows must be +0.0"
    z = torch.zeros(()).double()
    check(torch.where(empty, z, lc), torch.where(empty, z, rl), bl, what + " lse")

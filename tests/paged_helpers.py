"""Plain 64-bit forms of the head norms with rotation and of attention over a paged cache, the
bounds their outputs are held to, and seeded inputs for the tests."""
import math

import torch

U = 2.0 ** -24                      # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}  # half a step of an output's type


def angles(P, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def pair_index(d, rot, inter):
    """Index tensors (a, b) of the pairs of the first rot dimensions."""
    c = torch.arange(rot // 2)
    return (2 * c, 2 * c + 1) if inter else (c, c + rot // 2)


def rotate(t, cs, inter, sign=1.0):
    """t [..., d] turned by the angles cs [..., rot] (cos then sin), 64 bits."""
    rot = cs.shape[-1]
    a, b = pair_index(t.shape[-1], rot, inter)
    co, si = cs[..., :rot // 2].double(), sign * cs[..., rot // 2:].double()
    y = t.clone()
    y[..., a] = t[..., a] * co - t[..., b] * si
    y[..., b] = t[..., a] * si + t[..., b] * co
    return y


def norm_rope(x, w, cs, inter, eps):
    """(y, bound): x [..., d] and cs broadcast against it (None: no rotation).  The bound counts one
    rounding to x's type and the fp32 arithmetic before it: the sum of d squares in a tree (20 U of
    the mean, half of that in its root), the root (2 U), three products and the turn's two products
    and a sum, all within 32 U of the largest |t| of the row in magnitude."""
    f = x.double()
    t = f if w is None else f / (f.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y = t if cs is None else rotate(t, cs, inter)
    return y, HALF[x.dtype] * y.abs() + 32 * U * 1.5 * t.abs().amax(-1, keepdim=True)


def norm_rope_bwd(x, dy, w, cs, inter, eps):
    """(dx, dw, bound of dx, sum |terms| of dw).  dx's bound: one rounding, and 64 U (two sums of d
    terms, the root, six products) of r (max |g| + max |n| mean |g n|)."""
    f, t = x.double(), dy.double()
    if cs is not None:
        t = rotate(t, cs, inter, -1.0)
    if w is None:
        return t, None, HALF[x.dtype] * t.abs() + 8 * U * 1.5 * dy.double().abs().amax(-1, keepdim=True), None
    r = 1 / (f.square().mean(-1, keepdim=True) + eps).sqrt()
    n, g = f * r, w.double() * t
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    size = r * (g.abs().amax(-1, keepdim=True) + n.abs().amax(-1, keepdim=True) * (g * n).abs().mean(-1, keepdim=True))
    dims = tuple(range(x.dim() - 1))
    return dx, (t * n).sum(dims), HALF[x.dtype] * dx.abs() + 64 * U * size, (t * n).abs().sum(dims)


def paged_inputs(new, lens, Hq, Hkv, d, page, seed=0, dtype=torch.bfloat16, device="cuda", spare=3, poison=True,
                 width=None, heads_first=False):
    """A cache whose pages are handed out in a random order; slots no sequence holds are NaN, and
    table entries past a sequence's last page are far out of range."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(lens), sum(new)
    need = [-(-n // page) for n in lens]
    width = max(need + [1]) if width is None else width
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g)
    bt = torch.full((B, width), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        bt[b, :k] = perm[at:at + k].int()
        at += k
    kp = torch.randn(pages, page, Hkv, d, generator=g)
    vp = torch.randn(pages, page, Hkv, d, generator=g)
    if poison:
        held = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                held[bt[b, j], :min(page, n - j * page)] = True
        kp[~held] = math.nan
        vp[~held] = math.nan
    q = torch.randn(T, Hq, d, generator=g)
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    mv = lambda t: t.to(dtype).to(device)  # noqa: E731
    kp, vp = mv(kp), mv(vp)
    if heads_first:  # [pages, Hkv, page, d] in memory
        kp, vp = (t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for t in (kp, vp))
    return dict(q=mv(q), kp=kp, vp=vp, bt=bt.to(device), lens=torch.tensor(lens, dtype=torch.int32, device=device),
                cu=cu.to(device))


def paged_ref(s, new, lens, causal, scale):
    """(o, lse, bound of o, bound of lse) [T, Hq, ...] in 64 bits on the CPU.

    The kernels round the weights to bf16 before the value product (half a step, 2^-8 of each), and
    the output once; with A = sum_j p_j |v_j|, |do| <= 2^-8 |o| + 2^-8 A.  A logit's products are
    exact in fp32 and their sum of d terms is off by at most d U sum |q k|, which moves weights and
    lse by that much (times 2 for the row sum), scaled; the exponential (2 ulp) and the sum of
    a row's weights add 2^-18 of A and of lse's argument."""
    q, kp, vp, bt = (s[n].cpu() for n in ("q", "kp", "vp", "bt"))
    page, Hkv, d = kp.shape[1], kp.shape[2], kp.shape[3]
    T, Hq = q.shape[:2]
    G = Hq // Hkv
    o, A = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, d, dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    dx = torch.zeros(T, Hq, dtype=torch.float64)
    t = 0
    for b, (nq, n) in enumerate(zip(new, lens)):
        if n > 0 and nq > 0:
            pg = bt[b, :-(-n // page)].long()
            K = kp[pg].reshape(-1, Hkv, d)[:n].double().repeat_interleave(G, 1)
            V = vp[pg].reshape(-1, Hkv, d)[:n].double().repeat_interleave(G, 1)
            Q = q[t:t + nq].double()
            X = torch.einsum("ihd,jhd->hij", Q, K) * scale
            E = torch.einsum("ihd,jhd->hij", Q.abs(), K.abs()) * scale
            if causal:
                hid = torch.arange(n)[None, :] > torch.arange(nq)[:, None] + (n - nq)
                X = X.masked_fill(hid, -math.inf)
            L = torch.logsumexp(X, -1)
            P = torch.where(torch.isinf(L)[..., None], torch.zeros(()).double(), torch.exp(X - L[..., None]))
            o[t:t + nq] = torch.einsum("hij,jhd->ihd", P, V)
            A[t:t + nq] = torch.einsum("hij,jhd->ihd", P, V.abs())
            lse[t:t + nq] = L.T
            dx[t:t + nq] = (d + 8) * U * E.amax(-1).T
        t += nq
    slack = 2 * dx[..., None] + 2.0 ** -18
    return o, lse, 2.0 ** -8 * (o.abs() + A) + slack * A, 2 * dx + 2.0 ** -18 * (1 + lse.abs().nan_to_num(0, 0, 0))


def check(got, ref, bound, what):
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert bool(torch.isfinite(g).all()), f"{what}: not finite"
    over = (g - ref).abs() - bound
    assert bool((over <= 0).all()), f"{what}: over its bound by {over.max().item():.3e} at {over.argmax().item()}"


def check_paged(o, lse, s, new, lens, causal, scale, what=""):
    ro, rl, bo, bl = paged_ref(s, new, lens, causal, scale)
    check(o, ro, bo, what + " o")
    empty = torch.isinf(rl)
    lc = lse.cpu().double()
    assert bool((lc[empty] == -math.inf).all()), f"{what}: empty rows must have lse = -inf"
    assert bool((o.cpu().view(torch.int16)[empty] == 0).all()), f"{what}: empty rows must be +0.0"
    check(torch.where(empty, torch.zeros(()).double(), lc), torch.where(empty, torch.zeros(()).double(), rl), bl, what + " lse")

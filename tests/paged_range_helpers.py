"""The 64-bit attention over an 8-bit cache with the bound that include/attn.h states for it: the loss of a key's value goes by
that key's weight and scale in the row itself, never by keys that the row does not see or that weigh nothing in it."""
import math

import torch

from paged_helpers import U, check
from paged_q8_helpers import _rows


def visible_ref(s, new, lens, causal, scale, groups=None, plens=()):
    """(o, lse, bound of o, bound of lse) [T, Hq, ...]; groups and plens as for paged_q8_helpers.attention_ref.

    With p_j a key's weight relative to the row's largest, 2^g_j = 2^(f_j - 127) its value's scale, l = sum p_j and
    A = sum p_j |v_j| / l, |do| is at most
      2^-8 |o|              the output's rounding,
      2^-11 A               the weights' rounding to fp16,
      sum_j 448 (2^g_j min(p_j, 2^-32) + min(p_j 2^g_j, 2^-32 max_i p_i 2^g_i)) / l
                            what fp16 loses of small weights, or of small weights times scales (a code is at most 448; to
                            nearest, nothing loses more than itself),
      sum p_j |v_j| / l over the rows of scale byte 0, which count as zeros beside rows 2^25 above them,
      (2 dx + 2^-18 + 2 U (1.45 max |x| + 256)) A
                            the logits' sums dx = (d + 8) U sum |q k| (twice for the row sum), the exponentials, and the sum of a
                            logit and a scale's exponent in fp32."""
    q, bt = s["q"].cpu(), s["bt"].cpu()
    T, Hq, d = q.shape
    Hkv = s["kp"].shape[2]
    G = Hq // Hkv
    f64 = dict(dtype=torch.float64)
    o, bo = torch.zeros(T, Hq, d, **f64), torch.zeros(T, Hq, d, **f64)
    lse, bl = torch.full((T, Hq), -math.inf, **f64), torch.zeros(T, Hq, **f64)
    zero = torch.zeros((), **f64)
    rep = lambda x: x.repeat_interleave(G, 1)  # noqa: E731
    t = 0
    for b, (nq, n) in enumerate(zip(new, lens)):
        own = [_rows(s, x, bt[b], n) for x in "kv"]
        for i in range(nq):
            p = -1 if groups is None else int(groups[t + i])
            parts = [own] if p < 0 or plens[p] == 0 else [[_rows(s, x, s["pt"].cpu()[p], plens[p]) for x in "kv"], own]
            sees = min(max(n - nq + i + 1, 0), n) if causal else n
            cut = [len(x[0][0]) for x in parts[:-1]] + [sees]
            K, V = (torch.cat([x[k][0][:c] for x, c in zip(parts, cut)]) for k in (0, 1))
            g = torch.cat([x[1][1][:c] for x, c in zip(parts, cut)]).int() - 127
            if len(K) == 0:
                continue
            Q = q[t + i].double()
            X = torch.einsum("hd,jhd->hj", Q, rep(K)) * scale
            E = torch.einsum("hd,jhd->hj", Q.abs(), rep(K).abs()) * scale
            M = X.amax(-1, keepdim=True)
            W = torch.exp(X - M)
            l = W.sum(-1, keepdim=True)
            R, two = rep(V), torch.ldexp(torch.ones_like(g, **f64), g).T.repeat_interleave(G, 0)
            oo = torch.einsum("hj,jhd->hd", W, R) / l
            A = torch.einsum("hj,jhd->hd", W, R.abs()) / l
            most = (W * two).amax(-1, keepdim=True)
            lost = 448 * (W.clamp(max=2.0 ** -32) * two + torch.minimum(W * two, 2.0 ** -32 * most)).sum(-1, keepdim=True) / l
            none = torch.einsum("hj,jhd->hd", torch.where(two == 2.0 ** -127, W, zero), R.abs()) / l
            dx = (d + 8) * U * E.amax(-1)
            slack = 2 * dx + 2.0 ** -18 + 2 * U * (1.45 * X.abs().amax(-1) + 256)
            o[t + i], lse[t + i] = oo, (M + torch.log(l))[:, 0]
            bo[t + i] = 2.0 ** -8 * oo.abs() + 2.0 ** -11 * A + lost + none + slack[:, None] * A
            bl[t + i] = 2 * dx + 2.0 ** -18 * (1 + lse[t + i].abs())
        t += nq
    return o, lse, bo, bl


def check_visible(o, lse, s, new, lens, causal, scale, groups=None, plens=(), what="", fine=None):
    """fine: the share of the largest output that the bound stays below in every row, so that a row of zeros cannot pass."""
    ro, rl, bo, bl = visible_ref(s, new, lens, causal, scale, groups, plens)
    if fine is not None:
        some = ro.abs().amax(-1) > 0
        assert bool((bo.amax(-1) <= fine * ro.abs().amax(-1))[some].all()), f"{what}: a bound too wide to tell"
    empty = torch.isinf(rl)
    lc, z = lse.cpu().double(), torch.zeros((), dtype=torch.float64)
    assert bool((lc[empty] == -math.inf).all()), f"{what}: empty rows must have lse = -inf"
    check(torch.where(empty, z, lc), torch.where(empty, z, rl), bl, what + " lse")
    check(o, ro, bo, what + " o")

"""The operators for drafted tokens as their definitions stand, for the tests:
attention of a tree in 64 bits on torch tensors of any device, verification in
exact rational arithmetic, the move of cache rows one by one."""
import math
from fractions import Fraction

import torch

from layer_reference import f64, relative_bucket


def lines(parents):
    """For each node, the nodes from its first ancestor to it; [] for an absent node."""
    out = []
    for i, p in enumerate(parents):
        if p == -1:
            out.append([i])
        elif 0 <= p < i and out[p]:
            out.append(out[p] + [i])
        else:
            out.append([])
    return out


def tree_attention(q, k, v, parents, cached, scale, table=None, max_distance=128, bidirectional=True):
    """(o, lse, sum P|v|, largest sum|q k| of a seen pair) of one batch entry: q [N, H, D], k and v [L, Hkv, D],
    parents a list, cached a number."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    o, spread = torch.zeros_like(f64(q)), torch.zeros_like(f64(q))
    lse = torch.full((heads, n), -math.inf, dtype=torch.float64, device=q.device)
    most = 0.0
    for i, line in enumerate(lines(parents)):
        if not line:
            continue
        rows = torch.tensor(list(range(cached)) + [cached + t for t in line], device=q.device)
        kk, vv = (f64(x[rows]).repeat_interleave(group, 1) for x in (k, v))
        s = torch.einsum("hd,jhd->hj", f64(q[i]), kk) * scale
        most = max(most, float((torch.einsum("hd,jhd->hj", f64(q[i]).abs(), kk.abs()) * abs(scale)).max()))
        if table is not None:
            position = cached + len(line) - 1
            back = [relative_bucket(max(x - position, -max_distance - 1), table.shape[0], max_distance, bidirectional)
                    for x in range(position + 1)]
            s = s + f64(table)[torch.tensor(back, device=q.device)].T
        lse[:, i] = torch.logsumexp(s, 1)
        prob = torch.exp(s - torch.where(lse[:, i] == -math.inf, 0.0, lse[:, i])[:, None])
        o[i], spread[i] = torch.einsum("hj,jhd->hd", prob, vv), torch.einsum("hj,jhd->hd", prob, vv.abs())
    return o, lse, spread, most


def verify(target, draft, tokens, parents, u):
    """(path, out_tokens) of one batch entry from lists of numbers, in exact arithmetic: target[node][token]."""
    exact = [[max(Fraction(x), Fraction(0)) for x in row] for row in target]
    like = None if draft is None else [[Fraction(x) for x in row] for row in draft]
    vocab, at, path, out = len(target[0]), 0, [0], []
    while True:
        w, mass, stands = list(exact[at]), Fraction(1), None
        for i in range(at + 1, len(parents)):
            if parents[i] != at or not 0 <= tokens[i] < vocab:
                continue
            t = tokens[i]
            bar = Fraction(u[i]) * mass
            if like is not None:
                bar *= like[at][t]
            if 0 < w[t] and bar < w[t]:
                stands = i
                break
            if like is None:
                mass -= w[t]
                w[t] = Fraction(0)
            else:
                w = [max(a - mass * b, Fraction(0)) for a, b in zip(w, like[at])]
                mass = sum(w)
        if stands is None:
            break
        at = stands
        path.append(at)
        out.append(tokens[at])
    if sum(w) == 0:
        w = exact[at]
    bar, up_to, last = Fraction(u[0]) * sum(w), Fraction(0), -1
    for t, x in enumerate(w):
        up_to += x
        if up_to > bar:
            last = t
            break
    return path, out + [last]


def keep(cache, path, accepted, cached):
    """One batch entry's cache [L, H, D] after the move."""
    after = cache.clone()
    for k in range(1, accepted + 1):
        after[cached + k] = cache[cached + path[k]]
    return after

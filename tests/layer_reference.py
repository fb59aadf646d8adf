"""The transformer-layer operators in 64 bits, for the tests: the formulas as
they stand, on torch tensors of any device, the mask from the CPU oracle."""
import math

import numpy as np
import torch


def keep_mask(orc, p, seed, first, shape, device):
    """uniform(seed, first + flat index) >= p, scaled by 1 / (1 - p); 1.0 for p = 0."""
    p = float(np.float32(p))
    if p == 0.0:
        return torch.ones(shape, dtype=torch.float64, device=device)
    n = math.prod(shape)
    kept = orc.dropout(np.ones(n, np.float32), p, seed, first & 0xFFFFFFFF) != 0
    return torch.from_numpy(kept).to(device).double().view(shape) / (1 - p)


def f64(t):
    return None if t is None else t.double()


def norm_fwd(x, bias, residual, gamma, beta, keep, eps):
    h = f64(x)
    if bias is not None:
        h = h + f64(bias)
    h = h * keep
    if residual is not None:
        h = h + f64(residual)
    mean = h.mean(-1)
    rstd = 1 / torch.sqrt(((h - mean[..., None]) ** 2).mean(-1) + eps)
    y = (h - mean[..., None]) * rstd[..., None]
    if gamma is not None:
        y = y * f64(gamma)
    if beta is not None:
        y = y + f64(beta)
    return y, h, mean, rstd


def norm_bwd(dy, h, dh, gamma, mean, rstd, keep):
    """dx, dresidual, dgamma, dbeta, dbias."""
    dy, mean, rstd = f64(dy), f64(mean)[:, None], f64(rstd)[:, None]
    n = (f64(h) - mean) * rstd
    g = dy if gamma is None else dy * f64(gamma)
    dz = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if dh is not None:
        dz = dz + f64(dh)
    dx = dz * keep
    return dx, dz, (dy * n).sum(0), dy.sum(0), dx.sum(0)


def bucket(distance, count, max_distance):
    """One direction's bucket of a distance."""
    exact = count // 2
    if distance < exact:
        return distance
    m = count - exact
    return exact + max(t for t in range(m)
                       if t == 0 or distance ** m >= exact ** (m - t) * max_distance ** t)


def relative_bucket(rel, num_buckets, max_distance, bidirectional):
    if not bidirectional:
        return bucket(max(-rel, 0), num_buckets, max_distance)
    return bucket(abs(rel), num_buckets // 2, max_distance) + (num_buckets // 2 if rel > 0 else 0)


class Pairs:
    """Everything about (query, key) pairs that does not depend on the values:
    visibility [B, 1, Lq, Lk], buckets [B, Lq, Lk] (or None), the mask."""

    def __init__(self, orc, q, k, key_lengths, causal, last, buckets, max_distance, bidirectional, p, seed, first):
        (b, lq, heads, _), lk, dev = q.shape, k.shape[1], q.device
        n = torch.full((b,), lk, device=dev) if key_lengths is None else key_lengths.long().clamp(0, lk)
        pos = torch.arange(lq, device=dev)[None, :] + ((n - lq)[:, None] if last else torch.zeros_like(n)[:, None])
        j = torch.arange(lk, device=dev)
        rel = j[None, None, :] - pos[:, :, None]
        visible = j[None, None, :] < n[:, None, None]
        if causal:
            visible = visible & (rel <= 0)
        self.visible = visible.expand(b, lq, lk)[:, None]
        self.buckets = None
        if buckets:
            far = max_distance + 1
            table = torch.tensor([relative_bucket(r, buckets, max_distance, bidirectional)
                                  for r in range(-far, far + 1)], device=dev)
            self.buckets = table[rel.clamp(-far, far) + far].expand(b, lq, lk)
        self.keep = keep_mask(orc, p, seed, first, (b, heads, lq, lk), dev)


def heads_first(t, group=1):
    return f64(t).transpose(1, 2).repeat_interleave(group, 1)


def scores(q, k, table, pairs, scale):
    s = heads_first(q) @ heads_first(k, q.shape[2] // k.shape[2]).transpose(2, 3) * scale
    if table is not None:
        s = s + f64(table)[pairs.buckets].permute(0, 3, 1, 2)
    return s.masked_fill(~pairs.visible, -math.inf)


def attention_fwd(q, k, v, table, pairs, scale):
    """o [B, Lq, H, D], lse [B, H, Lq] and P [B, H, Lq, Lk]."""
    v = v.masked_fill(~pairs.visible.any(2).any(1)[:, :, None, None], 0)  # unseen keys count for nothing
    k = k.masked_fill(~pairs.visible.any(2).any(1)[:, :, None, None], 0)
    s = scores(q, k, table, pairs, scale)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:-1], -math.inf, dtype=s.dtype, device=s.device)
    prob = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o = (prob * pairs.keep) @ heads_first(v, q.shape[2] // k.shape[2])
    return o.transpose(1, 2), lse, prob


def shared(t, heads_kv):
    """[B, H, Lk, D] summed over the query heads of each key head, [B, Lk, Hkv, D]."""
    b, h, n, d = t.shape
    return t.reshape(b, heads_kv, h // heads_kv, n, d).sum(2).transpose(1, 2)


def attention_bwd(do, q, k, v, o, table, pairs, prob, scale):
    """dq, dk, dv, dtable (or None) and dS."""
    group, hk = q.shape[2] // k.shape[2], k.shape[2]
    do, o = heads_first(do), heads_first(o)
    dp = do @ heads_first(v, group).transpose(2, 3) * pairs.keep
    ds = prob * (dp - (do * o).sum(-1, keepdim=True))
    dq = (ds @ heads_first(k, group) * scale).transpose(1, 2)
    dk = shared(ds.transpose(2, 3) @ heads_first(q) * scale, hk)
    dv = shared((prob * pairs.keep).transpose(2, 3) @ do, hk)
    return dq, dk, dv, by_bucket(ds, table, pairs), ds


def by_bucket(ds, table, pairs):
    if table is None:
        return None
    out = torch.zeros(table.shape, dtype=torch.float64, device=ds.device)
    return out.index_add_(0, pairs.buckets.reshape(-1), ds.permute(0, 2, 3, 1).reshape(-1, ds.shape[1]))

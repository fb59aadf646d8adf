"""Measured cases of the transformer-layer operators: bias + dropout +
residual + layer norm, and attention with a bucketed relative position bias
and dropout on its probabilities, each forward and backward.

Dropout's mask is never an input or an output: element c of a mask is
uniform(seed, first + c) >= p on the lowbias32 hash, c the element's flat
index, in every form below.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5

# ---- the cases ----------------------------------------------------------------


def _norm(name, op, rows, cols, dtype, params, p, **more):
    case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "params": params, "p": p, "bias": True,
            "residual": True}
    return {**({"name": name} if name else {}), **case, **more}


def _attention(name, op, batch, len_q, len_k, heads, kv_heads, dim, dtype, p, **more):
    case = {"op": op, "batch": batch, "len_q": len_q, "len_k": len_k, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "p": p, "causal": False, "last": False, "ragged": False, "buckets": 0,
            "max_distance": 128}
    return {**({"name": name} if name else {}), **case, **more}


def listed():
    return [
        # one token of a decoding step: add the residual, normalise (no dropout in serving)
        _norm("norm_fwd_one_token", "norm_fwd", 1, 1024, "bf16", "bf16", 0.0, bias=False),
        # a training micro-batch's sublayer end in bf16
        _norm("norm_fwd_train", "norm_fwd", 16384, 4096, "bf16", "bf16", 0.1),
        # the dropout configuration [2^20, 256] of f32 activations
        _norm("norm_fwd_f32_long", "norm_fwd", 1 << 20, 256, "f32", "f32", 0.1),
        # the same sublayer's gradient
        _norm("norm_bwd_train", "norm_bwd", 16384, 4096, "bf16", "bf16", 0.1),
        # odd sizes: no row starts on a vector boundary; f32 weights under f16 activations
        _norm("norm_bwd_odd", "norm_bwd", 1531, 769, "f16", "f32", 0.5),
        # one decoding step of a batch over a long cache, ragged lengths, shared key heads
        _attention("attn_fwd_decode", "attn_fwd", 32, 1, 8192, 32, 8, 128, "bf16", 0.0, causal=True, last=True,
                   ragged=True),
        # one short request, one token: latency
        _attention("attn_fwd_one_token", "attn_fwd", 1, 1, 301, 8, 8, 64, "bf16", 0.0, causal=True, last=True,
                   buckets=32),
        # an encoder layer in training: bucketed bias, dropout
        _attention("attn_fwd_encoder", "attn_fwd", 16, 1024, 1024, 16, 16, 64, "bf16", 0.1, buckets=32),
        # a prompt of odd length, causal, grouped heads
        _attention("attn_fwd_prompt", "attn_fwd", 1, 4099, 4099, 32, 8, 128, "bf16", 0.0, causal=True),
        # the encoder layer's gradient, with the bias table's
        _attention("attn_bwd_encoder", "attn_bwd", 16, 1024, 1024, 16, 16, 64, "bf16", 0.1, buckets=32),
        # a decoder layer's gradient: causal, grouped heads, dropout
        _attention("attn_bwd_decoder", "attn_bwd", 2, 4096, 4096, 16, 4, 128, "bf16", 0.1, causal=True),
        # ragged and odd: short padded sentences, a head dimension that fills no tile
        _attention("attn_bwd_ragged", "attn_bwd", 24, 77, 115, 6, 6, 40, "f16", 0.1, ragged=True, buckets=20,
                   max_distance=64),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    if rng.random() < 0.45:
        cols = _spread(rng, 16, 16384)
        if rng.random() < 0.5:
            cols = -(-cols // 40) * 40  # whole vectors of every type
        rows = _spread(rng, 1, min(1 << 20, (1 << 26) // cols))
        dtype = rng.choice(["f32", "bf16", "f16"])
        return _norm("", rng.choice(["norm_fwd", "norm_bwd"]), rows, cols, dtype, rng.choice([dtype, "f32"]),
                     rng.choice([0.0, 0.1, 0.5]), bias=rng.random() < 0.6, residual=rng.random() < 0.7)
    dim = rng.choice([64, 128, 64, 128, 8 * rng.randint(1, 16)])
    kv_heads = rng.randint(1, 8)
    heads = kv_heads * rng.choice([1, 1, 1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    buckets = rng.choice([0, 16, 32, 64])
    common = {"ragged": rng.random() < 0.4, "buckets": buckets,
              "max_distance": rng.choice([64, 128, 300]) if buckets else 128}
    if rng.random() < 0.25:  # serving: a few new tokens against a cache
        len_q, len_k = rng.choice([1, 1, 2, 5, 16]), _spread(rng, 1, 32768)
        batch = _spread(rng, 1, max(1, min(64, (1 << 28) // (len_k * kv_heads * dim))))
        return _attention("", "attn_fwd", batch, len_q, len_k, heads, kv_heads, dim, dtype, 0.0, causal=True,
                          last=True, **common)
    len_k = _spread(rng, 1, 4096)
    len_q = len_k if rng.random() < 0.7 else _spread(rng, 1, 4096)
    batch = _spread(rng, 1, max(1, min(32, (1 << 28) // (len_q * len_k * heads))))
    return _attention("", rng.choice(["attn_fwd", "attn_bwd"]), batch, len_q, len_k, heads, kv_heads, dim, dtype,
                      rng.choice([0.0, 0.1, 0.1, 0.3]), causal=rng.random() < 0.5, last=rng.random() < 0.3, **common)


# ---- what a program holds before the call ---------------------------------------


def _key_lengths(case):
    """Lengths from nothing at all to the whole of len_k, in no order."""
    b, n = case["batch"], case["len_k"]
    return [(n * ((5 * i + 2) % b)) // max(1, b - 1) if b > 1 else (n + 1) // 2 for i in range(b)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(to)

    state = {"case": case, "seed": seed & 0xFFFFFFFF, "first": (seed * 40503) & 0xFFFFFFFF}
    if case["op"].startswith("norm"):
        rows, cols, params = case["rows"], case["cols"], DTYPES[case["params"]]
        state["gamma"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(params)
        state["mean"] = torch.empty(rows, device="cuda")
        state["rstd"] = torch.empty(rows, device="cuda")
        if case["op"] == "norm_fwd":
            state["x"] = normal(rows, cols)
            state["bias"] = normal(cols, scale=0.1, to=params) if case["bias"] else None
            # a residual stream has an offset and a few channels far above the rest
            state["residual"] = None
            if case["residual"]:
                state["residual"] = (torch.randn(rows, cols, generator=g, device="cuda")
                                     * (1 + 8 * (torch.rand(cols, generator=g, device="cuda") < 0.01)) + 0.3).to(dtype)
            state["beta"] = normal(cols, scale=0.2, to=params)
            state["y"], state["h"] = torch.empty_like(state["x"]), torch.empty_like(state["x"])
        else:
            state["h"] = (torch.randn(rows, cols, generator=g, device="cuda")
                          * (1 + 8 * (torch.rand(cols, generator=g, device="cuda") < 0.01)) + 0.3).to(dtype)
            hf = state["h"].float()
            state["mean"] = hf.mean(1)
            state["rstd"] = (hf.var(1, unbiased=False) + EPS).rsqrt()
            state["dy"] = normal(rows, cols)
            state["dh"] = normal(rows, cols) if case["residual"] else None
            state["dx"] = torch.empty_like(state["h"])
            state["dresidual"] = torch.empty_like(state["h"]) if case["residual"] else None
            state["dgamma"], state["dbeta"] = torch.empty_like(state["gamma"]), torch.empty_like(state["gamma"])
            state["dbias"] = torch.empty_like(state["gamma"]) if case["bias"] else None
        return state
    b, d = case["batch"], case["dim"]
    state["q"] = normal(b, case["len_q"], case["heads"], d)
    state["k"] = normal(b, case["len_k"], case["kv_heads"], d)
    state["v"] = normal(b, case["len_k"], case["kv_heads"], d)
    state["table"] = normal(case["buckets"], case["heads"]) if case["buckets"] else None
    state["lengths"] = None
    if case["ragged"]:
        state["lengths"] = torch.tensor(_key_lengths(case), dtype=torch.int32, device="cuda")
    state["o"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty(b, case["heads"], case["len_q"], device="cuda")
    if case["op"] == "attn_bwd":
        state["o"], state["lse"] = _plain_attention(state)
        state["do"] = normal(b, case["len_q"], case["heads"], d)
        for name in ("q", "k", "v"):
            state["d" + name] = torch.empty_like(state[name])
        state["dtable"] = torch.empty_like(state["table"]) if case["buckets"] else None
    return state


# ---- the plain forms --------------------------------------------------------------


def _i32(v):
    return v - (1 << 32) if v >= 1 << 31 else v


def _plain_hash(x):
    """lowbias32 of an int32 tensor: wrapping products, logical shifts."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * 0x7FEB352D
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * _i32(0x846CA68B)
    return x ^ ((x >> 16) & 0xFFFF)


def _plain_keep(state, shape):
    """uniform(seed, first + flat index) >= p for every element of shape."""
    n = math.prod(shape)
    c = (torch.arange(n, device="cuda", dtype=torch.int64) + state["first"]).to(torch.int32)
    key = _plain_hash(torch.tensor(_i32(state["seed"]), dtype=torch.int32, device="cuda"))
    u = (_plain_hash(c ^ key) & 0x7FFFFF).float() * 2.0 ** -23
    return (u >= torch.tensor(state["case"]["p"], device="cuda")).view(shape)


def _plain_drop(state, x):
    p = state["case"]["p"]
    if p == 0.0:
        return x
    return torch.where(_plain_keep(state, x.shape), x / (1 - torch.tensor(p, device="cuda")), 0.0)


def _plain_norm_fwd(state):
    dtype = state["x"].dtype
    x = state["x"].float()
    if state["bias"] is not None:
        x = x + state["bias"].float()
    h = _plain_drop(state, x)
    if state["residual"] is not None:
        h = h + state["residual"].float()
    mean = h.mean(1)
    centred = h - mean[:, None]
    rstd = 1 / torch.sqrt((centred * centred).mean(1) + EPS)
    y = centred * rstd[:, None] * state["gamma"].float() + state["beta"].float()
    return {"y": y.to(dtype), "h": h.to(dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(state):
    dtype, params = state["h"].dtype, state["gamma"].dtype
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    xh = (state["h"].float() - state["mean"][:, None]) * rstd
    g = dy * state["gamma"].float()
    dz = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if state["dh"] is not None:
        dz = dz + state["dh"].float()
    dx = _plain_drop(state, dz)
    out = {"dx": dx.to(dtype), "dgamma": (dy * xh).sum(0).to(params), "dbeta": dy.sum(0).to(params)}
    if state["dresidual"] is not None:
        out["dresidual"] = dz.to(dtype)
    if state["dbias"] is not None:
        out["dbias"] = dx.sum(0).to(params)
    return out


def _bucket_starts(buckets, max_distance):
    """The distances at which one direction's buckets 1, 2, ... begin: single
    distances for the first half, then evenly in the logarithm up to
    max_distance, in whole numbers throughout."""
    exact = buckets // 2
    m = buckets - exact
    starts = list(range(1, exact + 1))
    for t in range(1, m):
        n = int(exact * (max_distance / exact) ** (t / m)) - 1
        while n ** m < exact ** (m - t) * max_distance ** t:
            n += 1
        starts.append(n)
    return starts


def _plain_buckets(state):
    """The bucket of every (query, key) pair, [B or 1, Lq, Lk]."""
    case = state["case"]
    pos = _plain_positions(state)
    rel = torch.arange(case["len_k"], device="cuda")[None, None, :] - pos[:, :, None]
    half = case["buckets"] // 2
    starts = torch.tensor(_bucket_starts(half, case["max_distance"]), device="cuda")
    return torch.bucketize(rel.abs(), starts, right=True) + half * (rel > 0)


def _plain_positions(state):
    """The position of every query among the keys, [B or 1, Lq]."""
    case = state["case"]
    pos = torch.arange(case["len_q"], device="cuda")[None, :]
    if case["last"]:
        ends = torch.tensor([case["len_k"]], device="cuda") if state["lengths"] is None else state["lengths"].long()
        pos = pos + (ends - case["len_q"])[:, None]
    return pos


def _plain_probabilities(state):
    """softmax(S) and its log-sum, [B, H, Lq, Lk] and [B, H, Lq]."""
    case = state["case"]
    q, k = state["q"].float().transpose(1, 2), state["k"].float().transpose(1, 2)
    k = k.repeat_interleave(case["heads"] // case["kv_heads"], 1)
    s = torch.matmul(q, k.transpose(2, 3)) * case["dim"] ** -0.5
    if state["table"] is not None:
        s = s + state["table"].float()[_plain_buckets(state)].permute(0, 3, 1, 2)
    j = torch.arange(case["len_k"], device="cuda")
    if state["lengths"] is not None:
        s = s.masked_fill(j >= state["lengths"][:, None, None, None], -math.inf)
    if case["causal"]:
        s = s.masked_fill((j > _plain_positions(state)[:, :, None])[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total), (top + torch.log(total))[..., 0]


def _plain_attention(state):
    case = state["case"]
    prob, lse = _plain_probabilities(state)
    v = state["v"].float().transpose(1, 2).repeat_interleave(case["heads"] // case["kv_heads"], 1)
    o = torch.matmul(_plain_drop(state, prob), v)
    return o.transpose(1, 2).contiguous().to(state["q"].dtype), lse


def _plain_attention_fwd(state):
    o, lse = _plain_attention(state)
    return {"o": o, "lse": lse}


def _plain_attention_bwd(state):
    case, dtype = state["case"], state["q"].dtype
    group, shared = case["heads"] // case["kv_heads"], (case["batch"], case["kv_heads"], -1, case["len_k"], case["dim"])
    q, do, o = (state[n].float().transpose(1, 2) for n in ("q", "do", "o"))
    k, v = (state[n].float().transpose(1, 2).repeat_interleave(group, 1) for n in ("k", "v"))
    prob, _ = _plain_probabilities(state)
    dv = torch.matmul(_plain_drop(state, prob).transpose(2, 3), do)
    dprob = _plain_drop(state, torch.matmul(do, v.transpose(2, 3)))
    ds = prob * (dprob - (do * o).sum(-1, keepdim=True))
    scale = case["dim"] ** -0.5
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(2, 3), q) * scale
    out = {"dq": dq.transpose(1, 2).contiguous().to(dtype)}
    for name, d in (("dk", dk), ("dv", dv)):
        out[name] = d.reshape(shared).sum(2).transpose(1, 2).contiguous().to(dtype)
    if state["table"] is not None:
        where = _plain_buckets(state).expand(case["batch"], -1, -1).reshape(-1)
        flat = ds.permute(0, 2, 3, 1).reshape(-1, case["heads"])
        dtable = torch.zeros(case["buckets"], case["heads"], device="cuda")
        out["dtable"] = dtable.index_add_(0, where, flat).to(dtype)
    return out


# ---- the framework's calls ----------------------------------------------------------


def _own_norm_fwd(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_dropout_layer_norm_fwd(
        state["x"], state["gamma"], state["beta"], state["y"], state["mean"], state["rstd"], bias=state["bias"],
        residual=state["residual"], h=state["h"], p=state["case"]["p"], seed=state["seed"],
        first_counter=state["first"], eps=EPS)
    return {n: state[n] for n in ("y", "h", "mean", "rstd")}


def _own_norm_bwd(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_dropout_layer_norm_bwd(
        state["dy"], state["h"], state["gamma"], state["mean"], state["rstd"], state["dx"], state["dgamma"],
        state["dbeta"], dh=state["dh"], dresidual=state["dresidual"], dbias=state["dbias"], p=state["case"]["p"],
        seed=state["seed"], first_counter=state["first"])
    return {n: state[n] for n in ("dx", "dgamma", "dbeta", "dresidual", "dbias") if state[n] is not None}


def _own_options(state):
    case = state["case"]
    return {"key_lengths": state["lengths"], "causal": case["causal"], "queries_last": case["last"],
            "bias_table": state["table"], "max_distance": case["max_distance"], "p": case["p"],
            "seed": state["seed"], "first_counter": state["first"]}


def _own_attention_fwd(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_attention_fwd(state["q"], state["k"], state["v"], state["o"], lse=state["lse"], **_own_options(state))
    return {"o": state["o"], "lse": state["lse"]}


def _own_attention_bwd(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_attention_bwd(state["do"], state["q"], state["k"], state["v"], state["o"], state["lse"], state["dq"],
                          state["dk"], state["dv"], dbias_table=state["dtable"], **_own_options(state))
    return {n: state[n] for n in ("dq", "dk", "dv", "dtable") if state[n] is not None}


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "attn_fwd": _plain_attention_fwd,
          "attn_bwd": _plain_attention_bwd}
_OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "attn_fwd": _own_attention_fwd,
        "attn_bwd": _own_attention_bwd}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------


def _pairs(case):
    """(visible query-key pairs of one head over the batch, keys read over the batch)."""
    lengths = _key_lengths(case) if case["ragged"] else [case["len_k"]] * case["batch"]
    pairs = 0
    for n in lengths:
        at = n - case["len_q"] if case["last"] else 0
        if case["causal"]:
            seen = np.clip(np.arange(case["len_q"]) + at + 1, 0, n)
            pairs += int(seen.sum())
        else:
            pairs += case["len_q"] * n
    return pairs, sum(lengths)


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"].startswith("norm"):
        n, pe = case["rows"] * case["cols"], SIZE[case["params"]]
        moved = (4 if case["residual"] else 3) if case["op"] == "norm_fwd" else (5 if case["residual"] else 3)
        small = case["cols"] * pe * (3 if case["bias"] else 2) * (1 if case["op"] == "norm_fwd" else 2)
        return {"bytes": n * moved * e + 8 * case["rows"] + small, "flops": n * (12 if case["op"] == "norm_fwd" else 20)}
    pairs, keys = _pairs(case)
    q = case["batch"] * case["len_q"] * case["heads"] * case["dim"] * e
    kv = keys * case["kv_heads"] * case["dim"] * e
    lse = 4 * case["batch"] * case["heads"] * case["len_q"]
    table = case["buckets"] * case["heads"] * e
    if case["op"] == "attn_fwd":
        return {"bytes": 2 * q + 2 * kv + lse + table, "flops": 4 * case["dim"] * pairs * case["heads"]}
    written = case["batch"] * case["len_k"] * case["kv_heads"] * case["dim"] * e * 2
    return {"bytes": 4 * q + 2 * kv + written + lse + 2 * table, "flops": 10 * case["dim"] * pairs * case["heads"]}


# ---- the definitions in 64 bits ------------------------------------------------------


def _exact_mask(seed, first, n, p, offset=0):
    """uniform(seed, first + offset + i) >= p for i < n, as 0.0 or 1.0, from unsigned 64-bit arithmetic."""
    full = 0xFFFFFFFF

    def rounds(x):
        x = x ^ (x >> 16)
        x = (x * 0x7FEB352D) & full
        x = x ^ (x >> 15)
        lo, hi = (x & 0xFFFF) * 0x846CA68B, (x >> 16) * 0x846CA68B  # the product passes 63 bits
        x = (lo + ((hi & 0xFFFF) << 16)) & full
        return x ^ (x >> 16)

    key = rounds(torch.tensor(seed, dtype=torch.int64, device="cuda"))
    c = (torch.arange(n, dtype=torch.int64, device="cuda") + (first + offset)) & full
    u = (rounds(c ^ key) & 0x7FFFFF).double() / 8388608.0
    return (u >= float(np.float32(p))).double()


def _exact_norm(case, state):
    rows, cols, p = case["rows"], case["cols"], float(np.float32(case["p"]))
    keep = 1.0
    if p:
        keep = _exact_mask(state["seed"], state["first"], rows * cols, p).view(rows, cols) / (1 - p)
    gamma = state["gamma"].double()
    if case["op"] == "norm_fwd":
        z = state["x"].double()
        if state["bias"] is not None:
            z += state["bias"].double()
        z = z * keep
        if state["residual"] is not None:
            z += state["residual"].double()
        var, mean = torch.var_mean(z, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(state["beta"].double(), (z - mean[:, None]).mul_(rstd[:, None]), gamma)
        return {"y": y, "h": z, "mean": mean, "rstd": rstd}
    dy, rstd = state["dy"].double(), state["rstd"].double()[:, None]
    unit = (state["h"].double() - state["mean"].double()[:, None]) * rstd
    out = {"dgamma": torch.einsum("rc,rc->c", dy, unit), "dbeta": dy.sum(0)}
    up = dy * gamma
    inner = torch.einsum("rc,rc->r", up, unit)[:, None] / cols
    dz = (up - up.sum(1, keepdim=True) / cols - unit * inner) * rstd
    if state["dh"] is not None:
        dz += state["dh"].double()
    if state["dresidual"] is not None:
        out["dresidual"] = dz
    out["dx"] = dz * keep
    if state["dbias"] is not None:
        out["dbias"] = out["dx"].sum(0)
    return out


def _exact_bucket(distance, buckets, max_distance):
    """One direction's bucket of a distance: floor of the logarithm, by whole numbers."""
    exact = buckets // 2
    if distance < exact:
        return distance
    m = buckets - exact
    t = m - 1
    while t > 0 and distance ** m < exact ** (m - t) * max_distance ** t:
        t -= 1
    return exact + t


def _exact_attention(case, state):
    b_n, h_n, lq, lk, d = case["batch"], case["heads"], case["len_q"], case["len_k"], case["dim"]
    group, p, back = h_n // case["kv_heads"], float(np.float32(case["p"])), case["op"] == "attn_bwd"
    f64 = {"dtype": torch.float64, "device": "cuda"}
    q, k, v = (state[n].double() for n in ("q", "k", "v"))
    if back:
        do, delta = state["do"].double(), (state["do"].double() * state["o"].double()).sum(3)
        out = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
        if case["buckets"]:
            out["dtable"] = torch.zeros(case["buckets"], h_n, **f64)
    else:
        out = {"o": torch.zeros_like(q), "lse": torch.full((b_n, h_n, lq), -math.inf, **f64)}
    lengths = _key_lengths(case) if case["ragged"] else [lk] * b_n
    half, far = case["buckets"] // 2, case["max_distance"]
    one_way = [_exact_bucket(x, half, far) for x in range(far + 1)] if half else []
    for b in range(b_n):
        n = lengths[b]
        if n == 0:
            continue
        at = n - lq if case["last"] else 0
        rel = torch.arange(n, device="cuda")[None, :] - (torch.arange(lq, device="cuda")[:, None] + at)
        where = None
        if half:
            where = torch.tensor(one_way, device="cuda")[rel.abs().clamp(max=far)] + torch.where(rel > 0, half, 0)
        for h in range(h_n):
            kb, vb = k[b, :n, h // group], v[b, :n, h // group]
            s = q[b, :, h] @ kb.T / math.sqrt(d)
            if half:
                s = s + state["table"].double()[:, h][where]
            if case["causal"]:
                s = torch.where(rel > 0, -math.inf, s)
            lse = torch.logsumexp(s, 1)
            prob = torch.exp(s - lse[:, None]).nan_to_num_(nan=0.0)
            keep = 1.0
            if p:
                keep = _exact_mask(state["seed"], state["first"], lq * lk, p, (b * h_n + h) * lq * lk)
                keep = keep.view(lq, lk)[:, :n] / (1 - p)
            if not back:
                out["o"][b, :, h], out["lse"][b, h] = (prob * keep) @ vb, lse
                continue
            g = do[b, :, h]
            ds = prob * ((g @ vb.T) * keep - delta[b, :, h, None])
            out["dq"][b, :, h] = ds @ kb / math.sqrt(d)
            out["dk"][b, :n, h // group] += ds.T @ q[b, :, h] / math.sqrt(d)
            out["dv"][b, :n, h // group] += (prob * keep).T @ g
            if half:
                out["dtable"][:, h].index_add_(0, where.reshape(-1), ds.reshape(-1))
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return (_exact_norm if case["op"].startswith("norm") else _exact_attention)(case, state)

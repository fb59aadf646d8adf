"""Measured cases of the operators that run drafted tokens: attention of a tree
of drafted tokens over a cache, verification of the drafts against the target's
probabilities, and the move of the accepted tokens' cache rows.

A tree of a batch entry is `nodes` tokens in an order in which a parent comes
before its children.  Node 0 is the newest token that is known; the others are
drafts.  parents[i] is the node before node i, -1 for none, and anything else
outside 0 .. i - 1 says that there is no such node (a padded tree).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}

# ---- the cases ----------------------------------------------------------------


def _tree(name, batch, nodes, len_k, heads, kv_heads, dim, dtype, **more):
    case = {"op": "tree", "batch": batch, "nodes": nodes, "len_k": len_k, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "chain": False, "ragged": False, "padded": False, "buckets": 0,
            "max_distance": 128}
    return {**({"name": name} if name else {}), **case, **more}


def _verify(name, batch, nodes, vocab, dtype, **more):
    case = {"op": "verify", "batch": batch, "nodes": nodes, "vocab": vocab, "dtype": dtype, "chain": False,
            "draft": True, "given": True}
    return {**({"name": name} if name else {}), **case, **more}


def _keep(name, caches, batch, nodes, len_k, kv_heads, dim, dtype, **more):
    case = {"op": "keep", "caches": caches, "batch": batch, "nodes": nodes, "len_k": len_k, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "stacked": True}
    return {**({"name": name} if name else {}), **case, **more}


def listed():
    return [
        # one short request, a small tree, the layer's relative bias: latency
        _tree("tree_one_request", 1, 8, 309, 8, 8, 64, "bf16", buckets=32),
        # a batch of requests with long caches of ragged lengths, a tree of 16 each
        _tree("tree_serving", 32, 16, 8208, 32, 8, 128, "bf16", ragged=True),
        # few requests that draft widely
        _tree("tree_wide", 8, 64, 4163, 32, 8, 128, "bf16"),
        # one long request that drafts a chain
        _tree("tree_long_chain", 1, 5, 32773, 32, 8, 128, "f16", chain=True),
        # a served decoder with a relative bias: grouped heads, trees of different sizes
        _tree("tree_bias_serving", 16, 12, 4108, 16, 4, 128, "bf16", ragged=True, padded=True, buckets=32),
        # many short requests, a head dimension and lengths that fill no tile
        _tree("tree_short_odd", 96, 7, 122, 6, 6, 40, "f16", ragged=True, buckets=20, max_distance=64),
        # one request, a chain of four drafts, a small vocabulary: latency
        _verify("verify_one_request", 1, 5, 32768, "f32", chain=True),
        # a batch of requests with trees, a large vocabulary
        _verify("verify_serving", 128, 16, 131072, "f32"),
        # a vocabulary whose rows start on no vector boundary, 16-bit probabilities, draws of the library's hash
        _verify("verify_odd_bf16", 33, 9, 50001, "bf16", given=False),
        # drafts without probabilities of their own (looked up, or taken greedily)
        _verify("verify_point_drafts", 64, 24, 131072, "f32", draft=False),
        # one request of a decoder of two layers, its caches in a list
        _keep("keep_one_request", 4, 1, 8, 309, 2, 64, "bf16", stacked=False),
        # all layers' caches of a served batch, in one tensor
        _keep("keep_serving", 64, 32, 16, 256, 8, 128, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.random()
    if kind < 0.5:
        dim = rng.choice([64, 128, 64, 128, 8 * rng.randint(1, 16)])
        kv_heads = rng.randint(1, 8)
        heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 4, 8])
        nodes = _spread(rng, 1, 128)
        len_k = nodes + _spread(rng, 1, 32768) - 1
        most = min(64, (1 << 28) // (len_k * kv_heads * dim), (1 << 27) // (len_k * heads * nodes))
        buckets = rng.choice([0, 0, 16, 32, 64])
        return _tree("", _spread(rng, 1, max(1, most)), nodes, len_k, heads, kv_heads, dim,
                     rng.choice(["bf16", "bf16", "f16"]), chain=rng.random() < 0.25, ragged=rng.random() < 0.6,
                     padded=rng.random() < 0.3, buckets=buckets,
                     max_distance=rng.choice([64, 128, 300]) if buckets else 128)
    if kind < 0.8:
        vocab, nodes = _spread(rng, 32, 200000), _spread(rng, 1, 64)
        batch = _spread(rng, 1, max(1, min(256, (1 << 28) // (vocab * nodes))))
        return _verify("", batch, nodes, vocab, rng.choice(["f32", "f32", "bf16", "f16"]), chain=rng.random() < 0.4,
                       draft=rng.random() < 0.7, given=rng.random() < 0.6)
    dim = rng.choice([64, 128, 8 * rng.randint(1, 16)])
    kv_heads, caches, nodes = rng.randint(1, 8), 2 * _spread(rng, 1, 40), _spread(rng, 1, 64)
    len_k = nodes + rng.randint(0, 256)
    batch = _spread(rng, 1, max(1, min(64, (1 << 29) // (caches * len_k * kv_heads * dim))))
    return _keep("", caches, batch, nodes, len_k, kv_heads, dim, rng.choice(["bf16", "bf16", "f16"]),
                 stacked=rng.random() < 0.5)


# ---- what a program holds before the call ---------------------------------------


def _cache_lengths(case):
    """Cached tokens of each entry: from none to what leaves room for the tree, in no order."""
    b, n = case["batch"], case["len_k"] - case["nodes"]
    if case["op"] == "tree" and not case["ragged"]:
        return [n] * b
    return [(n * ((5 * i + 2) % b)) // max(1, b - 1) if b > 1 else (n + 1) // 2 for i in range(b)]


def _present(case):
    """Nodes that each entry's tree has."""
    n = case["nodes"]
    return [n - (3 * i + 1) % (n // 2 + 1) if case["padded"] else n for i in range(case["batch"])]


def _paths(case):
    """The accepted nodes of each entry, the root first: what a verification would give."""
    r, paths = random.Random(case["batch"] * 1000003 + case["nodes"]), []
    for _ in range(case["batch"]):
        paths.append([0] + sorted(r.sample(range(1, case["nodes"]), r.randint(0, min(7, case["nodes"] - 1)))))
    return paths


def _random_parents(g, batch, nodes):
    """Each node's parent is an earlier one, the first few more often: bushy at the root, some levels deep."""
    u = torch.rand(batch, nodes, generator=g, device="cuda")
    i = torch.arange(nodes, device="cuda")
    parents = (u * u * i).long().clamp(max=nodes).minimum((i - 1).clamp(min=0)).to(torch.int32)
    parents[:, 0] = -1
    return parents


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype, b, n = DTYPES[case["dtype"]], case["batch"], case["nodes"]
    state = {"case": case}

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)

    if case["op"] == "tree":
        cache = (b, case["len_k"], case["kv_heads"], case["dim"])
        state["q"] = normal(b, n, case["heads"], case["dim"])
        state["k"], state["v"] = normal(*cache), normal(*cache)
        state["table"] = normal(case["buckets"], case["heads"]) if case["buckets"] else None
        state["lengths"] = torch.tensor(_cache_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        state["parents"] = None
        if not case["chain"] or case["padded"]:
            state["parents"] = _random_parents(g, b, n)
            if case["chain"]:
                state["parents"] = (torch.arange(n, device="cuda", dtype=torch.int32) - 1).repeat(b, 1)
            if case["padded"]:
                there = torch.tensor(_present(case), device="cuda")[:, None] > torch.arange(n, device="cuda")
                state["parents"] = torch.where(there, state["parents"], -2)
        state["o"] = torch.empty_like(state["q"])
        state["lse"] = torch.empty(b, case["heads"], n, device="cuda")
        return state
    if case["op"] == "verify":
        parents = _random_parents(g, b, n)
        if case["chain"]:
            parents = (torch.arange(n, device="cuda", dtype=torch.int32) - 1).repeat(b, 1)
        # the model's logits, and a draft's that are near them
        logits = torch.randn(b, n, case["vocab"], generator=g, device="cuda").mul_(2.5)
        state["target"] = torch.softmax(logits, 2).to(dtype)
        logits += torch.randn(b, n, case["vocab"], generator=g, device="cuda").mul_(0.5)
        draft = torch.softmax(logits, 2).to(dtype)
        # every draft is drawn from its parent's row: the token of the first of exponentials by their rates
        rows = draft.float().gather(1, parents.clamp(min=0).long()[:, :, None].expand_as(draft))
        times = torch.empty_like(rows).exponential_(generator=g)
        state["tokens"] = (rows / times).argmax(2).to(torch.int32)
        state["draft"] = draft if case["draft"] else None
        state["parents"] = None if case["chain"] else parents
        state["uniforms"] = torch.rand(b, n, generator=g, device="cuda") if case["given"] else None
        state["seed"], state["first"] = seed & 0xFFFFFFFF, (seed * 40503) & 0xFFFFFFFF
        for name, shape in (("path", (b, n)), ("accepted", (b,)), ("out_tokens", (b, n))):
            state[name] = torch.empty(shape, dtype=torch.int32, device="cuda")
        return state
    # all caches in one tensor, a cache (a layer's keys or values) to an entry
    state["caches"] = normal(case["caches"], b, case["len_k"], case["kv_heads"], case["dim"])
    state["given"] = state["caches"] if case["stacked"] else list(state["caches"])
    state["lengths"] = torch.tensor(_cache_lengths(case), dtype=torch.int32, device="cuda")
    paths = _paths(case)
    state["path"] = torch.tensor([p + [-1] * (n - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    state["accepted"] = torch.tensor([len(p) - 1 for p in paths], dtype=torch.int32, device="cuda")
    state["new_lengths"] = torch.empty(b, dtype=torch.int32, device="cuda")
    return state


# ---- the plain forms --------------------------------------------------------------


def _plain_parents(state):
    """The parents of every entry's nodes, -2 for what is not there, [B, N]."""
    n, parents = state["case"]["nodes"], state["parents"]
    i = torch.arange(n, device="cuda")
    if parents is None:
        return (i - 1).expand(state["case"]["batch"], n)
    parents = parents.long()
    return torch.where((parents >= -1) & (parents < i), parents, -2)


def _plain_ancestors(parents):
    """Whether node t is node i or before it, [B, N, N]; none where a node or one before it is not there."""
    n = parents.shape[1]
    steps = torch.arange(n, device="cuda") == parents[:, :, None]  # one step up
    reach = (steps | torch.eye(n, dtype=torch.bool, device="cuda")).float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    there = (reach * (parents < -1)[:, None, :]).sum(2) == 0
    return (reach > 0) & there[:, :, None]


def _plain_starts(count, max_distance):
    """The distances at which one direction's buckets 1, 2, ... begin: single distances for the first half, then
    evenly in the logarithm up to max_distance, in whole numbers throughout."""
    exact = count // 2
    m = count - exact
    starts = list(range(1, exact + 1))
    for t in range(1, m):
        d = int(exact * (max_distance / exact) ** (t / m)) - 1
        while d ** m < exact ** (m - t) * max_distance ** t:
            d += 1
        starts.append(d)
    return torch.tensor(starts, device="cuda")


def _plain_tree(state):
    case, dtype = state["case"], state["q"].dtype
    b, n, lk, hk = case["batch"], case["nodes"], case["len_k"], case["kv_heads"]
    group, d = case["heads"] // hk, case["dim"]
    cached = torch.full((b,), lk - n, device="cuda") if state["lengths"] is None else state["lengths"].long()
    seen = _plain_ancestors(_plain_parents(state))
    depth = seen.sum(2) - 1
    node = torch.arange(lk, device="cuda") - cached[:, None]  # of each key: below 0 in the cache
    of_tree = node.clamp(0, n - 1)
    visible = seen.gather(2, of_tree[:, None, :].expand(b, n, lk)) & (node < n)[:, None]
    visible = torch.where(node[:, None] < 0, seen.any(2)[:, :, None], visible)
    # [B, key heads, heads of one x nodes, D]
    q = state["q"].float().view(b, n, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * n, d)
    k, v = state["k"].float().permute(0, 2, 3, 1), state["v"].float().permute(0, 2, 1, 3)
    s = (torch.matmul(q, k) * d ** -0.5).view(b, hk, group, n, lk)
    if state["table"] is not None:
        place = torch.where(node < 0, node, depth.gather(1, of_tree))
        distance = (depth[:, :, None] - place[:, None, :]).clamp(min=0)  # of what is seen
        bucket = torch.bucketize(distance, _plain_starts(case["buckets"] // 2, case["max_distance"]), right=True)
        s = s + state["table"].float()[bucket].permute(0, 3, 1, 2).view(b, hk, group, n, lk)
    s = s.masked_fill(~visible[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    e = e / torch.where(total == 0, 1.0, total)
    o = torch.matmul(e.view(b, hk, group * n, lk), v).view(b, case["heads"], n, d)
    return {"o": o.transpose(1, 2).contiguous().to(dtype), "lse": (top + torch.log(total)).view(b, case["heads"], n)}


def _i32(v):
    return v - (1 << 32) if v >= 1 << 31 else v


def _plain_hash(x):
    """lowbias32 of an int32 tensor: wrapping products, logical shifts."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * 0x7FEB352D
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * _i32(0x846CA68B)
    return x ^ ((x >> 16) & 0xFFFF)


def _plain_uniforms(state):
    """The random numbers [B, N]: given, or uniform(seed, first + flat index)."""
    case = state["case"]
    if state["uniforms"] is not None:
        return state["uniforms"].double()
    c = torch.arange(case["batch"] * case["nodes"], device="cuda") + state["first"]
    key = _plain_hash(torch.tensor(_i32(state["seed"]), dtype=torch.int32, device="cuda"))
    u = (_plain_hash(c.to(torch.int32) ^ key) & 0x7FFFFF).double() * 2.0 ** -23
    return u.view(case["batch"], case["nodes"])


def _plain_weights(state, row, at, c, removed):
    """What is left of the target's row after the rejections so far, [B, V], in 64 bits: the sums decide whole
    numbers."""
    p = state["target"][row, at].double()
    if state["draft"] is not None:
        return (p - c[:, None] * state["draft"][row, at].double()).clamp(min=0)
    return p.masked_fill(removed, 0)


def _plain_verify(state):
    case, u, parents = state["case"], _plain_uniforms(state), _plain_parents(state)
    b, n, vocab = case["batch"], case["nodes"], case["vocab"]
    row, at = torch.arange(b, device="cuda"), torch.zeros(b, dtype=torch.long, device="cuda")
    c, mass = torch.zeros(b, dtype=torch.float64, device="cuda"), torch.ones(b, dtype=torch.float64, device="cuda")
    removed = torch.zeros(b, vocab, dtype=torch.bool, device="cuda")
    accepted = torch.zeros(b, dtype=torch.long, device="cuda")
    path, out = torch.full((b, n), -1, device="cuda"), torch.full((b, n), -1, device="cuda")
    path[:, 0] = 0
    for i in range(1, n):
        t = state["tokens"][:, i].long()
        p = state["target"][row, at, t].double()
        if state["draft"] is not None:
            q = state["draft"][row, at, t].double()
            w, bar = (p - c * q).clamp(min=0), u[:, i] * mass * q
        else:
            w, bar = torch.where(removed[row, t], 0.0, p), u[:, i] * mass
        child = parents[:, i] == at
        yes, no = child & (bar < w), child & ~(bar < w)
        # a rejected draft's share leaves the row
        if state["draft"] is not None:
            c = torch.where(no, c + mass, c)
            mass = torch.where(no, _plain_weights(state, row, at, c, removed).sum(1), mass)
        else:
            mass = torch.where(no, mass - w, mass)
            removed[row, t] = removed[row, t] | no
        # an accepted one is the next row's place
        out[row, accepted] = torch.where(yes, t, out[row, accepted])
        accepted = accepted + yes
        path[row, accepted] = torch.where(yes, i, path[row, accepted])
        at, c, mass = torch.where(yes, i, at), torch.where(yes, 0.0, c), torch.where(yes, 1.0, mass)
        removed = removed & ~yes[:, None]
    w = _plain_weights(state, row, at, c, removed)
    empty = w.sum(1) == 0
    w = torch.where(empty[:, None], _plain_weights(state, row, at, c * 0, removed & False), w)
    up_to = w.cumsum(1)
    first = ((up_to > (u[:, 0] * up_to[:, -1])[:, None]) & (w > 0)).int().argmax(1)
    out[row, accepted] = torch.where(up_to[:, -1] > 0, first, -1)
    return {"path": path.int(), "accepted": accepted.int(), "out_tokens": out.int()}


def _plain_keep(state):
    case, n = state["case"], state["case"]["nodes"]
    k = torch.arange(n, device="cuda")
    moves = k <= state["accepted"][:, None]
    entry, place = moves.nonzero(as_tuple=True)
    start = state["lengths"].long()[entry]
    rows = state["caches"][:, entry, start + state["path"][entry, place].long()]
    state["caches"][:, entry, start + place] = rows
    state["new_lengths"].copy_(state["lengths"] + state["accepted"] + 1)
    return {"caches": state["caches"], "new_lengths": state["new_lengths"]}


# ---- the framework's calls ----------------------------------------------------------


def _own_tree(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_tree_attention_fwd(
        state["q"], state["k"], state["v"], state["o"], lse=state["lse"], cache_lengths=state["lengths"],
        parents=state["parents"], bias_table=state["table"], max_distance=state["case"]["max_distance"])
    return {"o": state["o"], "lse": state["lse"]}


def _own_verify(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_verify_drafts(
        state["target"], state["tokens"], state["path"], state["accepted"], state["out_tokens"], draft=state["draft"],
        parents=state["parents"], uniforms=state["uniforms"], seed=state["seed"], first_counter=state["first"])
    return {n: state[n] for n in ("path", "accepted", "out_tokens")}


def _own_keep(state):
    import dropout_lowbias32_hash32_gb300 as rng
    rng.rng_cache_keep(state["given"], state["path"], state["accepted"], state["lengths"], state["new_lengths"])
    return {"caches": state["caches"], "new_lengths": state["new_lengths"]}


_PLAIN = {"tree": _plain_tree, "verify": _plain_verify, "keep": _plain_keep}
_OWN = {"tree": _own_tree, "verify": _own_verify, "keep": _own_keep}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    e, b, n = SIZE[case["dtype"]], case["batch"], case["nodes"]
    if case["op"] == "tree":
        present = _present(case)
        rows = sum(present) * case["heads"]
        keys = sum(_cache_lengths(case)) + sum(present)
        # a node sees the cache, itself and the nodes before it (not counted: they differ with the inputs)
        pairs = sum(m * (c + 1) for m, c in zip(present, _cache_lengths(case))) * case["heads"]
        moved = 2 * rows * case["dim"] * e + 2 * keys * case["kv_heads"] * case["dim"] * e
        return {"bytes": moved + 4 * rows + 4 * b * n + case["buckets"] * case["heads"] * e, "flops": 4 * case["dim"] * pairs}
    if case["op"] == "verify":
        # the row where the walk ends, and the draft's there; a few numbers for every draft
        rows = 2 if case["draft"] else 1
        return {"bytes": b * rows * case["vocab"] * e + 28 * b * n, "flops": b * case["vocab"] * (4 if case["draft"] else 2)}
    moved = sum(p != k for path in _paths(case) for k, p in enumerate(path))
    return {"bytes": 2 * case["caches"] * moved * case["kv_heads"] * case["dim"] * e + 4 * b * (n + 3), "flops": 0}


# ---- the definitions in 64 bits ------------------------------------------------------


def _exact_bucket(distance, count, max_distance):
    """One direction's bucket of a distance: floor of the logarithm, by whole numbers."""
    exact = count // 2
    if distance < exact:
        return distance
    m = count - exact
    t = m - 1
    while t > 0 and distance ** m < exact ** (m - t) * max_distance ** t:
        t -= 1
    return exact + t


def _exact_lines(parents):
    """For each node the nodes from the root to it; none where one of them is not there."""
    lines = []
    for i, p in enumerate(parents):
        if p == -1:
            lines.append([i])
        elif 0 <= p < i and lines[p]:
            lines.append(lines[p] + [i])
        else:
            lines.append([])
    return lines


def _exact_tree(case, state):
    b_n, n, h_n, d, far = case["batch"], case["nodes"], case["heads"], case["dim"], case["max_distance"]
    group, f64 = h_n // case["kv_heads"], {"dtype": torch.float64, "device": "cuda"}
    o, lse = torch.zeros(b_n, n, h_n, d, **f64), torch.full((b_n, h_n, n), -math.inf, **f64)
    parents = [[i - 1 for i in range(n)]] * b_n if state["parents"] is None else state["parents"].tolist()
    half = case["buckets"] // 2
    one_way = torch.tensor([_exact_bucket(x, half, far) for x in range(far + 1)], device="cuda") if half else None
    for b, cached in enumerate(_cache_lengths(case)):
        lines = _exact_lines(parents[b])
        mask, level = torch.zeros(n, n), torch.zeros(n, dtype=torch.long)
        for i, line in enumerate(lines):
            mask[i, line] = 1
            level[i] = len(line) - 1
        mask, level = mask.cuda() > 0, level.cuda()
        if not any(lines):
            continue
        keep = mask.any(1)
        place = torch.cat([torch.arange(cached, device="cuda"), cached + level])
        hidden = torch.cat([torch.zeros(n, cached, dtype=torch.bool, device="cuda"), ~mask], 1)
        kb, vb, qb = (state[x][b].double().transpose(0, 1) for x in ("k", "v", "q"))
        kb, vb = (x[:, : cached + n].repeat_interleave(group, 0) for x in (kb, vb))
        s = torch.einsum("hid,hjd->hij", qb, kb) / math.sqrt(d)
        if half:
            back = ((cached + level)[:, None] - place[None, :]).clamp(0, far)
            s += state["table"].double().T[:, one_way[back]]
        s[:, hidden] = -math.inf
        row = torch.logsumexp(s, 2)
        o[b, keep] = torch.einsum("hij,hjd->ihd", torch.exp(s - row[:, :, None]), vb)[keep]
        lse[b][:, keep] = row[:, keep]
    return {"o": o, "lse": lse}


def _exact_uniform(seed, counter):
    """uniform(seed, counter) from unsigned whole numbers."""
    def rounds(x):
        x ^= x >> 16
        x = x * 0x7FEB352D & 0xFFFFFFFF
        x ^= x >> 15
        x = x * 0x846CA68B & 0xFFFFFFFF
        return x ^ x >> 16

    return (rounds((counter & 0xFFFFFFFF) ^ rounds(seed)) & 0x7FFFFF) / 8388608.0


def _exact_verify(case, state):
    b_n, n = case["batch"], case["nodes"]
    answer = {"path": [], "accepted": [], "out_tokens": []}
    for b in range(b_n):
        tokens = state["tokens"][b].tolist()
        parents = list(range(-1, n - 1)) if state["parents"] is None else state["parents"][b].tolist()
        if state["uniforms"] is None:
            u = [_exact_uniform(state["seed"], state["first"] + b * n + i) for i in range(n)]
        else:
            u = state["uniforms"][b].tolist()
        at, path, taken, tried = 0, [0], [], []
        while True:
            p = state["target"][b, at].double()
            q = None if state["draft"] is None else state["draft"][b, at].double()
            left, share, step = p.clone(), 1.0, None
            for i in (i for i in range(at + 1, n) if parents[i] == at):
                t = tokens[i]
                there = 1.0 if q is None else q[t].item()
                if u[i] * share * there < left[t].item():
                    step = i
                    break
                if q is None:
                    share -= left[t].item()
                    left[t] = 0
                else:
                    left = torch.relu(left - share * q)
                    share = left.sum().item()
                tried.append(i)
            if step is None:
                break
            at = step
            path.append(at)
            taken.append(tokens[at])
        if left.sum().item() == 0:
            left = p
        up_to = left.cumsum(0)
        more = (up_to > u[0] * up_to[-1].item()).nonzero()
        taken.append(int(more[0]) if len(more) else -1)
        answer["path"].append(path + [-1] * (n - len(path)))
        answer["accepted"].append(len(path) - 1)
        answer["out_tokens"].append(taken + [-1] * (n - len(taken)))
    return {k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in answer.items()}


def _exact_keep(case, state):
    after = state["caches"].clone()
    new = []
    for b, (path, c) in enumerate(zip(_paths(case), _cache_lengths(case))):
        for k, node in enumerate(path):
            after[:, b, c + k] = state["caches"][:, b, c + node]
        new.append(c + len(path))
    return {"caches": after, "new_lengths": torch.tensor(new, dtype=torch.int32, device="cuda")}


def exact(case, seed):
    return {"tree": _exact_tree, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](case, prepare(case, seed))

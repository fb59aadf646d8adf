"""rng_attention_{fwd,bwd} and rng_relative_bucket against the formulas in 64
bits.

Tolerances.  ut is the type's unit roundoff (2^-11 f16, 2^-8 bf16), u = 2^-24.
A score is a sum of D products accumulated in f32 (matrix units may truncate:
2 u a step) and scaled: within e = (D + 8) 2 u scale sum|q k| + 2^-21 (|s| +
|bias|) of itself, the latter for the exponential's argument in base two; e is
taken at its largest over the visible pairs, so P and l are within 2 e + 2^-20
of themselves.  P is rounded to ut for the product with V, so
  o:  (ut + 4 e) sum P'|v| + ut |o|,   P' = P / (1 - p),
plus, for f16, P's smallest step 2^-25 (relative to the row's largest) times
sum|v|.  lse is within e + 2^-20 (1 + |lse|).
Backward, with E = (D + 8) 2 u (sum|do v| / (1 - p) + sum|do o|) the error of
dP - delta: dS is rounded to ut, so each dS is within ut|dS| + 4 e |dS| + 2 P E
(+ 2^-25 for f16) = w, and dq is within scale sum w|k| + ut |dq|, dk alike with
|q|; dv within (ut + 4 e) sum P'|do| + ut |dv|; the table's gradient is not
rounded before its sum of n terms: 4 e sum|dS| + 2 sum P E + 4096 u sum|dS| +
ut |dtable| (a chain is at most 4096 terms long here).
Where P and dS are two terms (few rows), their part of this is ut^2, not ut.
"""
import ctypes as C
import math

import pytest

U = 2.0 ** -24
UT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def rng():
    import dropout_lowbias32_hash32_gb300 as rng
    return rng


def case(b=2, lq=64, lk=None, h=2, hk=None, d=64, dtype="bfloat16", lengths=None, causal=False, last=False, buckets=0,
         far=64, two_way=True, p=0.0, seed=5, first=0, spread=1.0):
    return dict(b=b, lq=lq, lk=lq if lk is None else lk, h=h, hk=hk or h, d=d, dtype=dtype, lengths=lengths,
                causal=causal, last=last, buckets=buckets, far=far, two_way=two_way, p=p, seed=seed, first=first,
                spread=spread)


def assert_within(name, got, want, tol):
    got = got.double()
    same = (got == want)  # infinities
    bad = ~(same | ((got - want).abs() <= tol))
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[0].tolist(),
                           float(((got - want).abs() / tol)[bad].max()))


class Run:
    """Inputs of a case, the kernels' outputs, the 64-bit ones and their tolerances."""

    def __init__(self, torch, rng, orc, c, garbage=True, **layout):
        import layer_reference as ref
        self.torch, self.rng, self.c = torch, rng, c
        g = torch.Generator(device="cuda").manual_seed(c["seed"] * 1000 + c["lq"] + c["lk"])
        dt = getattr(torch, c["dtype"])

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

        self.q = normal(c["b"], c["lq"], c["h"], c["d"], scale=c["spread"])
        self.k, self.v = (normal(c["b"], c["lk"], c["hk"], c["d"]) for _ in range(2))
        self.do = normal(c["b"], c["lq"], c["h"], c["d"])
        self.table = normal(c["buckets"], c["h"]) if c["buckets"] else None
        self.lengths = None
        if c["lengths"] is not None:
            self.lengths = torch.tensor(c["lengths"], dtype=torch.int32, device="cuda")
            if garbage:  # what lies past a length has no influence, whatever its bits
                for b, n in enumerate(c["lengths"]):
                    n = min(max(n, 0), c["lk"])
                    self.k[b, n:], self.v[b, n:] = float("nan"), float("inf")
        self.scale = c["d"] ** -0.5
        self.term = UT[c["dtype"]]  # what rounding P and dS may change of them
        self.pairs = ref.Pairs(orc, self.q, self.k, self.lengths, c["causal"], c["last"], c["buckets"], c["far"],
                               c["two_way"], c["p"], c["seed"], c["first"])
        self.options = dict(key_lengths=self.lengths, causal=c["causal"], queries_last=c["last"], bias_table=self.table,
                            max_distance=c["far"], bidirectional=c["two_way"], p=c["p"], seed=c["seed"],
                            first_counter=c["first"])

    def forward(self, **more):
        torch = self.torch
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full((self.c["b"], self.c["h"], self.c["lq"]), float("nan"), device="cuda")
        self.rng.rng_attention_fwd(self.q, self.k, self.v, o, lse=lse, **{**self.options, **more})
        return o, lse

    def backward(self, o, lse, **more):
        torch = self.torch
        out = {n: torch.full_like(t, float("nan")) for n, t in (("dq", self.q), ("dk", self.k), ("dv", self.v))}
        out["dtable"] = None if self.table is None else torch.full_like(self.table, float("nan"))
        self.rng.rng_attention_bwd(self.do, self.q, self.k, self.v, o, lse, out["dq"], out["dk"], out["dv"],
                                   dbias_table=out["dtable"], **{**self.options, **more})
        return out

    def clean(self):
        """k and v with zeros past the lengths."""
        gone = ~self.pairs.visible.any(2).any(1)[:, :, None, None]
        return self.k.masked_fill(gone, 0), self.v.masked_fill(gone, 0)

    def score_error(self):
        import layer_reference as ref
        k, _ = self.clean()
        big = ref.heads_first(self.q.abs()) @ ref.heads_first(k.abs(), self.c["h"] // self.c["hk"]).transpose(2, 3)
        big = big * abs(self.scale)
        bias = 0.0 if self.table is None else float(self.table.double().abs().max())
        err = (self.c["d"] + 8) * 2 * U * big + 2.0 ** -21 * (big + bias)
        err = err.masked_fill(~self.pairs.visible, 0)
        return float(err.max()) if err.numel() else 0.0

    def check_forward(self, o, lse):
        import layer_reference as ref
        ut, group = UT[self.c["dtype"]], self.c["h"] // self.c["hk"]
        k, v = self.clean()
        want, wlse, prob = ref.attention_fwd(self.q, k, v, self.table, self.pairs, self.scale)
        e, hv = self.score_error(), ref.heads_first(v, group).abs()
        tol = (self.term + 4 * e + 2.0 ** -19) * ((prob * self.pairs.keep) @ hv)
        if self.c["dtype"] == "float16":
            tol = tol + 2.0 ** -25 / (1 - self.c["p"]) * hv.sum(2, keepdim=True)
        assert_within("lse", lse, wlse, (e + 2.0 ** -20 * (1 + wlse.abs())).nan_to_num(posinf=0.0))
        assert_within("o", o, want, tol.transpose(1, 2) + ut * want.abs() + TINY[self.c["dtype"]])
        return prob

    def check_backward(self, o, prob, out):
        import layer_reference as ref
        c = self.c
        ut, group, tiny = UT[c["dtype"]], c["h"] // c["hk"], TINY[c["dtype"]]
        k, v = self.clean()
        dq, dk, dv, dtable, ds = ref.attention_bwd(self.do, self.q, k, v, o, self.table, self.pairs, prob, self.scale)
        e = self.score_error() + 2.0 ** -20
        ado, ao = ref.heads_first(self.do).abs(), ref.heads_first(o).abs()
        av, ak, aq = ref.heads_first(v, group).abs(), ref.heads_first(k, group).abs(), ref.heads_first(self.q).abs()
        kept = prob * self.pairs.keep
        err = (c["d"] + 8) * 2 * U * (ado @ av.transpose(2, 3) / (1 - c["p"]) + (ado * ao).sum(-1, keepdim=True))
        step = 2.0 ** -25 if c["dtype"] == "float16" else 0.0
        w = (self.term + 4 * e) * ds.abs() + 2 * prob * err + step * self.pairs.visible
        assert_within("dq", out["dq"], dq, (w @ ak * abs(self.scale)).transpose(1, 2) + ut * dq.abs() + tiny)
        assert_within("dk", out["dk"], dk, ref.shared(w.transpose(2, 3) @ aq * abs(self.scale), c["hk"]) + ut * dk.abs() + tiny)
        wv = (self.term + 4 * e) * kept + step / (1 - c["p"]) * self.pairs.visible
        assert_within("dv", out["dv"], dv, ref.shared(wv.transpose(2, 3) @ ado, c["hk"]) + ut * dv.abs() + tiny)
        if self.table is not None:
            tol = ref.by_bucket((4 * e + 4096 * U) * ds.abs() + 2 * prob * err, self.table, self.pairs)
            assert_within("dtable", out["dtable"], dtable, tol + ut * dtable.abs() + tiny)

    def check(self):
        o, lse = self.forward()
        prob = self.check_forward(o, lse)
        self.check_backward(o, prob, self.backward(o, lse))


CASES = {
    "one_token": case(b=1, lq=1, lk=1, h=1),
    "one_query": case(lq=1, lk=300, p=0.2),
    "one_key": case(lq=70, lk=1, buckets=8),
    "tile": case(lq=128, h=1, b=1),
    "tile_less_one": case(lq=127, lk=63, p=0.1),
    "tile_and_one": case(lq=129, lk=65, p=0.1, dtype="float16"),
    "keys_64": case(lq=33, lk=64), "keys_128": case(lq=130, lk=128, d=128), "keys_192": case(lq=5, lk=192),
    "odd": case(b=3, lq=77, lk=115, h=3, d=40, dtype="float16", p=0.1, buckets=20),
    "dim_8": case(lq=65, lk=70, d=8, p=0.5), "dim_72": case(lq=65, lk=70, d=72, p=0.1),
    "dim_120": case(lq=200, d=120, causal=True, dtype="float16"), "dim_128": case(lq=257, d=128, p=0.1),
    "causal": case(lq=300, causal=True, p=0.1), "causal_wide": case(lq=70, lk=400, causal=True),
    "causal_tall": case(lq=400, lk=70, causal=True, dtype="float16"),
    "last": case(lq=70, lk=400, causal=True, last=True, buckets=32),
    "last_empty_rows": case(lq=300, lk=140, causal=True, last=True, p=0.1),
    "ragged": case(b=5, lq=100, lk=200, lengths=[0, 200, 1, 129, 64], p=0.1),
    "ragged_out_of_range": case(b=3, lq=40, lk=90, lengths=[-5, 1000, 90]),
    "ragged_causal": case(b=4, lq=150, lengths=[150, 0, 33, 128], causal=True, buckets=32, dtype="float16"),
    "ragged_last": case(b=4, lq=40, lk=200, lengths=[200, 0, 33, 128], causal=True, last=True, buckets=16, p=0.1),
    "group_2": case(lq=150, h=4, hk=2, causal=True, p=0.1), "group_3": case(lq=90, h=6, hk=2, d=128, p=0.1),
    "group_8": case(lq=40, lk=170, h=8, hk=1, causal=True, last=True), "group_16": case(lq=9, lk=100, h=16, hk=1, d=128),
    "group_32": case(lq=5, lk=70, h=32, hk=1),
    "group_4_bias": case(lq=150, h=4, hk=1, buckets=32, p=0.1),
    "buckets": case(lq=300, buckets=32, far=128), "buckets_far": case(lq=700, h=1, b=1, buckets=64, far=1024),
    "buckets_one_way": case(lq=200, buckets=32, two_way=False, causal=True, p=0.1),
    "buckets_one_way_free": case(lq=200, buckets=7, far=20, two_way=False, dtype="float16"),
    "buckets_few": case(lq=200, buckets=4, far=2), "buckets_many": case(lq=300, buckets=128, far=300, h=3),
    "buckets_tall": case(lq=600, lk=130, buckets=32, h=1),
    "long": case(b=1, lq=1100, h=2, hk=1, p=0.1, causal=True, first=(1 << 32) - 12345),
    "long_keys": case(b=1, lq=3, lk=5000, h=2, buckets=32),
    "sharp": case(lq=150, spread=20.0, p=0.1), "sharp_f16": case(lq=150, spread=20.0, dtype="float16", causal=True),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_against_the_formulas(torch, rng, orc, name):
    Run(torch, rng, orc, CASES[name]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("group,lq,lk,b", ((1, 1, 4099, 3), (8, 1, 2049, 2), (4, 1, 129, 5), (2, 5, 1000, 2),
                                           (3, 1, 1500, 2), (16, 2, 600, 1), (1, 16, 700, 2)))
@pytest.mark.parametrize("dtype,d", (("bfloat16", 128), ("float16", 64), ("bfloat16", 96)))
def test_new_tokens_against_a_cache(torch, rng, orc, group, lq, lk, b, dtype, d):
    lengths = [lk, max(1, lk // 3), 0, 7, lk - 1][:b]
    r = Run(torch, rng, orc, case(b=b, lq=lq, lk=lk, h=2 * group, hk=2, d=d, dtype=dtype, lengths=lengths, causal=True,
                                  last=True))
    r.check_forward(*r.forward())


FEW = {
    "one_token": case(b=1, lq=1, lk=301, h=8, causal=True, last=True, buckets=32),
    "one_token_128": case(b=2, lq=1, lk=2500, h=16, hk=2, d=128, causal=True, last=True, dtype="float16"),
    "five": case(b=2, lq=5, h=6, d=8, buckets=32), "six": case(lq=6, h=9, hk=3, dtype="float16", p=0.1, buckets=32),
    "causal_128": case(lq=100, h=2, hk=1, d=128, causal=True, p=0.1), "tiles": case(b=1, lq=120, lk=250, h=2, p=0.2),
    "few_keys": case(b=2, lq=300, lk=20, h=8, d=40, dtype="float16", p=0.1), "five_queries": case(lq=5, lk=900, h=8, hk=2, d=128, buckets=16),
    "tiles_f16": case(b=1, lq=70, lk=128, h=4, hk=4, d=96, causal=True, last=True, dtype="float16", buckets=16),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", FEW)
def test_few_rows_take_two_terms(torch, rng, orc, name):
    """The forward pass for at most 512 queries of all heads; the backward pass for 512 queries, or keys, of all heads."""
    c = FEW[name]
    r = Run(torch, rng, orc, c)
    r.term = UT[c["dtype"]] ** (2 if c["b"] * c["h"] * c["lq"] <= 512 else 1)
    o, lse = r.forward()
    prob = r.check_forward(o, lse)
    r.term = UT[c["dtype"]] ** 2
    r.check_backward(o, prob, r.backward(o, lse))


@pytest.mark.gpu
@pytest.mark.parametrize("scale", (1.0, 0.0, -0.2))
@pytest.mark.parametrize("buckets,lk", ((0, 200), (32, 200), (0, 900)))
def test_scales(torch, rng, orc, scale, buckets, lk):
    """Of either sign: the maximum is then another score's; 0: every visible key counts alike."""
    for lq in (1, 150):
        r = Run(torch, rng, orc, case(lq=lq, lk=lk, h=4, hk=2, buckets=buckets, p=0.1, causal=True, last=True, spread=0.5))
        r.scale = r.options["scale"] = scale
        r.check()


# More work than there are SMs: every block takes several pieces, of unequal lengths, one after the other.
MANY = {
    "encoder": case(b=24, lq=300, lk=333, h=16, buckets=32, far=128, p=0.1),
    "causal": case(b=12, lq=385, h=24, hk=6, d=128, causal=True, p=0.1, dtype="float16"),
    "one_tile": case(b=64, lq=40, lk=30, h=12, d=40, dtype="float16", buckets=20, p=0.2),
    "odd_tiles": case(b=40, lq=130, lk=129, h=8, hk=4, d=128),
    "ragged": case(b=40, lq=150, lk=260, h=16, hk=8, lengths=[0, 260, 1, 64, 65, 128, 200, 7] * 5, causal=True, p=0.1),
    "ragged_bias": case(b=30, lq=70, lk=500, h=12, d=96, lengths=[500, 3, 0, 450, 129] * 6, causal=True, last=True,
                        buckets=32, dtype="float16"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", MANY)
def test_many_heads(torch, rng, orc, name):
    Run(torch, rng, orc, MANY[name]).check()
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("b,h,hk,lk,d,dtype", ((64, 16, 16, 1100, 128, "bfloat16"), (80, 32, 8, 1301, 64, "float16"),
                                               (200, 8, 2, 577, 128, "float16"), (7, 8, 4, 20000, 128, "bfloat16"),
                                               (300, 4, 4, 100, 64, "bfloat16")))
def test_many_new_tokens_against_a_cache(torch, rng, orc, b, h, hk, lk, d, dtype):
    lengths = [[lk, max(1, lk // 3), 0, 7, lk - 1, lk // 2][i % 6] for i in range(b)]
    r = Run(torch, rng, orc, case(b=b, lq=1, lk=lk, h=h, hk=hk, d=d, dtype=dtype, lengths=lengths, causal=True, last=True))
    r.check_forward(*r.forward())
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
def test_layouts(torch, rng, orc):
    """[B, H, L, D] storage, one packed q, k, v array, gradients into one packed
    array, a slice of a wider array: nothing beside it is written."""
    r = Run(torch, rng, orc, case(lq=140, h=3, d=64, p=0.1, buckets=32))
    o, lse = r.forward()
    out = r.backward(o, lse)
    prob = r.check_forward(o, lse)
    r.check_backward(o, prob, out)
    plain = {n: getattr(r, n) for n in ("q", "k", "v", "do")}
    for n, t in plain.items():
        setattr(r, n, t.transpose(1, 2).contiguous().transpose(1, 2))
    again, lse2 = r.forward()
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    packed = torch.stack([plain["q"], plain["k"], plain["v"]], 2)
    r.q, r.k, r.v = packed.unbind(2)
    again, lse2 = r.forward()
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    grads = torch.full_like(packed, float("nan"))
    dq, dk, dv = grads.unbind(2)
    dtable = torch.empty_like(r.table)
    rng.rng_attention_bwd(r.do, r.q, r.k, r.v, o, lse, dq, dk, dv, dbias_table=dtable, **r.options)
    assert torch.equal(dq, out["dq"]) and torch.equal(dk, out["dk"]) and torch.equal(dv, out["dv"])
    assert torch.equal(dtable, out["dtable"])
    wide = torch.full((2, 150, 5, 80), 7.0, dtype=o.dtype, device="cuda")
    rng.rng_attention_fwd(r.q, r.k, r.v, wide[:, 4:144, 1:4, 8:72], **r.options)
    assert torch.equal(wide[:, 4:144, 1:4, 8:72], o)
    wide[:, 4:144, 1:4, 8:72] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.gpu
def test_no_keys_and_no_queries(torch, rng):
    q = torch.randn(2, 5, 2, 64, device="cuda", dtype=torch.bfloat16)
    none = torch.empty(2, 0, 2, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = torch.full_like(q, float("nan")), torch.empty(2, 2, 5, device="cuda")
    rng.rng_attention_fwd(q, none, none, o, lse=lse)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    dq = torch.full_like(q, float("nan"))
    rng.rng_attention_bwd(q, q, none, none, o, lse, dq, none.clone(), none.clone())
    assert bool((dq == 0).all())
    table = torch.randn(8, 2, device="cuda", dtype=torch.bfloat16)
    dk, dv, dtable = (torch.full_like(t, float("nan")) for t in (q, q, table))
    lse0 = torch.empty(2, 2, 0, device="cuda")
    rng.rng_attention_bwd(none, none, q, q, none, lse0, none.clone(), dk, dv, bias_table=table, dbias_table=dtable)
    assert bool((dk == 0).all()) and bool((dv == 0).all()) and bool((dtable == 0).all())
    rng.rng_attention_fwd(none, q, q, none.clone(), lse=lse0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
def test_bias_as_a_mask(torch, rng, orc, dtype):
    """Table entries of -inf and of the type's lowest value: those pairs get
    nothing, a row of the former alone is empty, a row of the latter alone
    averages its keys."""
    c = case(lq=90, lk=90, h=3, buckets=8, far=16, dtype=dtype)
    r = Run(torch, rng, orc, c)
    lowest = torch.finfo(r.q.dtype).min
    r.table[0:2], r.table[4:, 0] = 0.5, -math.inf
    r.table[3, 1] = lowest
    r.table[:, 2] = lowest
    r.options["bias_table"] = r.table
    o, lse = r.forward()
    import layer_reference as ref
    want, _, prob = ref.attention_fwd(r.q, r.k, r.v, r.table, r.pairs, r.scale)
    tol = (2 * UT[dtype] + 1e-3) * (prob @ ref.heads_first(r.v).abs()).transpose(1, 2) + 1e-3
    assert_within("o", o[:, :, :2], want[:, :, :2], tol[:, :, :2])
    if dtype == "bfloat16":  # the lowest f16 still leaves room for the scores
        mean = r.v.double().mean(1, keepdim=True).expand(-1, 90, -1, -1)
        assert_within("o", o[:, :, 2], mean[:, :, 2], tol[:, :, 2])
    r.table[:, 0] = -math.inf
    o, lse = r.forward()
    assert bool((o[:, :, 0] == 0).all()) and bool((lse[:, 0] == -math.inf).all())
    out = r.backward(o, lse)
    assert bool((out["dq"][:, :, 0] == 0).all()) and bool((out["dtable"][:, 0] == 0).all())
    assert not any(bool(out[n].isnan().any()) for n in out)


@pytest.mark.gpu
def test_scores_that_are_not_finite(torch, rng, orc):
    """A NaN in a query reaches that query's row alone; one in a key reaches the
    rows that see it."""
    r = Run(torch, rng, orc, case(lq=150, h=1, b=1, causal=True))
    clean, _ = r.forward()
    r.q[0, 7] = float("nan")
    o, _ = r.forward()
    assert bool(o[0, 7].isnan().all()) and torch.equal(o[0, :7], clean[0, :7]) and torch.equal(o[0, 8:], clean[0, 8:])
    r = Run(torch, rng, orc, case(lq=150, h=1, b=1, causal=True))
    r.k[0, 100] = float("nan")
    o, _ = r.forward()
    assert bool(o[0, 100:].isnan().all()) and torch.equal(o[0, :100], clean[0, :100])


@pytest.mark.gpu
def test_gradients_that_are_not_finite_stay_in_their_bucket(torch, rng, orc):
    """Query 0 sees key 0 alone: what its gradient holds reaches bucket 0 and its own row of dq."""
    r = Run(torch, rng, orc, case(lq=150, h=2, b=1, causal=True, buckets=16, two_way=False))
    o, lse = r.forward()
    clean = r.backward(o, lse)
    r.do[0, 0] = float("inf")
    out = r.backward(o, lse)
    assert bool(out["dtable"][0].isnan().all()) and torch.equal(out["dtable"][1:], clean["dtable"][1:])
    assert bool(out["dq"][0, 0].isnan().all()) and torch.equal(out["dq"][0, 1:], clean["dq"][0, 1:])


@pytest.mark.gpu
def test_twice_the_same_bits_and_another_stream(torch, rng, orc):
    r = Run(torch, rng, orc, case(lq=300, h=4, hk=2, buckets=32, p=0.1, causal=True))
    o, lse = r.forward()
    out = r.backward(o, lse)
    o2, lse2 = r.forward()
    out2 = r.backward(o, lse)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(out[n], out2[n]) for n in out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = r.forward(stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        out2 = r.backward(o, lse)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(out[n], out2[n]) for n in out)


@pytest.mark.gpu
def test_captured_graph(torch, rng, orc):
    r = Run(torch, rng, orc, case(b=1, lq=1, lk=3000, h=8, hk=2, d=128, causal=True, last=True))
    want, _ = r.forward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = r.forward()
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


@pytest.mark.gpu
def test_gradient_against_differences(torch, rng, orc):
    """The kernels' gradient along a direction against central differences of
    the 64-bit forward of the same inputs: loss = <do, o>.  The outputs carry
    the type's rounding (2^-8 of each term, independent from term to term: 2^-8
    of the terms' 2-norm, times 8 for safety) and that of the saved o."""
    import layer_reference as ref
    r = Run(torch, rng, orc, case(b=2, lq=90, lk=70, h=4, hk=2, buckets=8, p=0.2, lengths=[70, 45]), garbage=False)
    o, lse = r.forward()
    out = r.backward(o, lse)
    g = torch.Generator(device="cuda").manual_seed(3)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("table", "dtable")):
        d = torch.randn(getattr(r, name).shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(step):
            v = {n: getattr(r, n).double() for n in ("q", "k", "v", "table")}
            v[name] = v[name] + step * d
            o, _, _ = ref.attention_fwd(v["q"], v["k"], v["v"], v["table"], r.pairs, r.scale)
            return (o * r.do).sum()

        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        terms = out[grad].double() * d
        size = terms.norm() if name != "table" else terms.abs().sum()
        assert abs(terms.sum() - want) <= 8 * 2.0 ** -8 * size + 1e-4 * terms.abs().sum(), name


@pytest.mark.gpu
def test_offsets_past_32_bits(torch, rng, orc):
    """Batch entries more than 2^32 elements apart."""
    far = (1 << 32) + 64
    store = torch.empty(far + (1 << 16), dtype=torch.bfloat16, device="cuda")

    def pair(t):
        view = store.as_strided(t.shape, (far, t.shape[2] * t.shape[3], t.shape[3], 1), at[0])
        at[0] += t[0].numel()
        return view

    at = [0]
    r = Run(torch, rng, orc, case(lq=40, lk=50, h=2, p=0.1))
    o, lse = r.forward()
    out = r.backward(o, lse)
    for n in ("q", "k", "v", "do"):
        view = pair(getattr(r, n))
        view.copy_(getattr(r, n))
        setattr(r, n, view)
    o2 = pair(o)
    rng.rng_attention_fwd(r.q, r.k, r.v, o2, **r.options)
    grads = {n: pair(out[n]) for n in ("dq", "dk", "dv")}
    rng.rng_attention_bwd(r.do, r.q, r.k, r.v, o2, lse, grads["dq"], grads["dk"], grads["dv"], **r.options)
    assert torch.equal(o, o2) and all(torch.equal(out[n], grads[n]) for n in grads)
    del store, o2, grads, r
    torch.cuda.empty_cache()


# ---- the buckets (no GPU) ----------------------------------------------------------


@pytest.mark.parametrize("buckets,far,two_way", ((32, 128, True), (32, 128, False), (4, 2, True), (2, 2, False),
                                                 (20, 64, True), (7, 20, False), (128, 1024, False), (64, 1024, True)))
def test_buckets(rng, buckets, far, two_way):
    import layer_reference as ref
    for rel in [*range(-300, 301), -far, far, -far - 1, far + 1, 1 << 40, -(1 << 63)]:
        d = max(-far, min(far, rel))
        assert rng.rng_relative_bucket(rel, buckets, far, two_way) == ref.relative_bucket(d, buckets, far, two_way)


@pytest.mark.parametrize("buckets,far,two_way", ((31, 128, True), (2, 64, True), (130, 300, True), (1, 64, False),
                                                 (32, 8, True), (32, 1025, True), (-4, 64, True)))
def test_buckets_refused(rng, buckets, far, two_way):
    with pytest.raises(rng.RngError):
        rng.rng_relative_bucket(0, buckets, far, two_way)


# ---- refusals (nothing below reaches the GPU) ---------------------------------------

A = 0x10000000  # an address that is never dereferenced


def args(rng, **change):
    a = rng.AttentionArgs()
    a.dtype, a.batch, a.len_q, a.len_k, a.heads_q, a.heads_kv, a.head_dim = rng.RNG_BF16, 2, 4, 4, 2, 2, 64
    for i, n in enumerate(("q", "k", "v", "o", "d_o", "dq", "dk", "dv")):
        setattr(a, n, (i + 1) * A)
        setattr(a, "do_stride" if n == "d_o" else n + "_stride", (512, 128, 64))
    a.lse, a.scale, a.workspace, a.workspace_bytes = 9 * A, 0.125, 10 * A, 1 << 30
    for n, v in change.items():
        setattr(a, n, v)
    return a


BOTH = [
    ({"dtype": 0}, "dtype"), ({"dtype": 9}, "dtype"), ({"batch": -1}, "negative"), ({"head_dim": 12}, "head_dim"),
    ({"head_dim": 136}, "head_dim"), ({"head_dim": 0}, "head_dim"), ({"heads_kv": 0}, "multiple"),
    ({"heads_q": 3}, "multiple"), ({"p": 1.0}, "outside"), ({"p": math.nan}, "outside"),
    ({"scale": math.inf}, "scale"), ({"q": None}, "NULL"), ({"k": A + 8}, "16-byte"),
    ({"v_stride": (512, 100, 64)}, "stride"), ({"k_stride": (0, 128, 64)}, "stride"),
    ({"q_stride": (512, -128, 64)}, "stride"), ({"q_stride": (1 << 40, 128, 64)}, "stride"),
    ({"lse": A + 2}, "aligned"), ({"key_lengths": A + 1}, "aligned"),
    ({"bias_table": 11 * A, "num_buckets": 31, "max_distance": 64, "bidirectional": 1}, "num_buckets"),
    ({"bias_table": 11 * A, "num_buckets": 32, "max_distance": 4, "bidirectional": 1}, "max_distance"),
    ({"batch": 1 << 30, "heads_q": 4, "heads_kv": 4}, "2^30"), ({"len_k": (1 << 30) + 1}, "2^30")]


@pytest.mark.parametrize("bad,says", BOTH + [({"o": A}, "overlap"), ({"o": 2 * A + 64}, "overlap"),
                                             ({"o_stride": (512, 64, 64)}, "overlaps itself")])
def test_forward_refuses(rng, bad, says):
    assert rng.raw("rng_attention_fwd")(C.byref(args(rng, **bad)), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error()


@pytest.mark.parametrize("bad,says", BOTH + [
    ({"dq": A}, "overlap"), ({"dv": 7 * A + 64}, "overlap"), ({"dk_stride": (256, 128, 64)}, "overlaps itself"),
    ({"lse": None}, "lse"), ({"workspace": None}, "workspace"), ({"workspace_bytes": 4}, "workspace"),
    ({"workspace": A + 4}, "workspace"), ({"dbias_table": 12 * A, "num_buckets": 32, "max_distance": 64}, "bias_table")])
def test_backward_refuses(rng, bad, says):
    assert rng.raw("rng_attention_bwd")(C.byref(args(rng, **bad)), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error()


def test_nothing_to_do_is_fine(rng):
    assert rng.raw("rng_attention_fwd")(None, None) == rng.RNG_EINVAL
    assert rng.raw("rng_attention_fwd")(C.byref(args(rng, batch=0, q=None, o=None)), None) == rng.RNG_OK
    assert rng.raw("rng_attention_fwd")(C.byref(args(rng, len_q=0)), None) == rng.RNG_OK
    assert rng.raw("rng_attention_bwd")(C.byref(args(rng, batch=0)), None) == rng.RNG_OK


@pytest.mark.gpu
def test_python_refusals(torch, rng):
    q = torch.zeros(2, 4, 2, 64, device="cuda", dtype=torch.bfloat16)
    o = torch.empty_like(q)
    call = rng.rng_attention_fwd
    with pytest.raises(TypeError):
        call(q.cpu(), q, q, o)
    with pytest.raises(TypeError):
        call(q, q.half(), q, o)
    with pytest.raises(ValueError):
        call(q[0], q[0], q[0], o[0])
    with pytest.raises(ValueError):
        call(q, q, q[:, :3], o)
    with pytest.raises(ValueError):
        call(q, q, q, o.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(TypeError):
        call(q, q, q, o, key_lengths=torch.zeros(2, device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        call(q, q, q, o, bias_table=torch.zeros(32, 3, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        call(q, q, q, o, bias_table=torch.zeros(32, 2, device="cuda"))
    with pytest.raises(rng.RngError):  # f32 activations
        call(q.float(), q.float(), q.float(), o.float())
    with pytest.raises(ValueError):
        rng.rng_attention_bwd(o, q, q, q, o, torch.zeros(2, 2, 4, device="cuda"), o, o, o, dbias_table=o)


@pytest.mark.gpu
def test_no_wait_ran_out(rng):
    assert rng.rng_debug_stalled_waits() == 0

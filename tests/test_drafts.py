"""rng_tree_attention_fwd, rng_verify_drafts and rng_cache_keep against their
definitions.

Tolerances of the attention.  As for the attention without a tree: with u =
2^-24 and ut the type's unit roundoff (2^-11 f16, 2^-8 bf16), a score is within
e = (D + 8) 2 u scale sum|q k| + 2^-21 (|s| + |bias|) of itself, e taken at its
largest over the seen pairs; lse is within e + 2^-20 (1 + |lse|), and with P
rounded to ut for the product with v, o within (ut + 4 e + 2^-19) sum P|v| +
ut |o|, plus for f16 P's smallest step 2^-25 times sum|v|.  Where P enters as two
terms, its part is ut^2, not ut.

Verification gives whole numbers, which have to be those of exact rational
arithmetic: the kernel's sums hold 2^-44, and no comparison of these inputs is
nearer to equality than that unless it is exactly equal.
"""
import ctypes as C
import itertools
import math
import random

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


# ---- attention of a tree ---------------------------------------------------------------


def bushy(r, n, roots=1):
    """Parents of a random tree: the first nodes often, the last one seldom."""
    return [-1 if i < roots else min(int(r.random() ** 2 * i), i - 1) for i in range(n)]


def case(b=2, n=8, lk=200, h=2, hk=None, d=64, dtype="bfloat16", cached=None, parents="bushy", buckets=0, far=64,
         two_way=True, seed=5, spread=1.0, scale=None):
    return dict(b=b, n=n, lk=lk, h=h, hk=hk or h, d=d, dtype=dtype, cached=cached, parents=parents, buckets=buckets,
                far=far, two_way=two_way, seed=seed, spread=spread, scale=scale)


class Run:
    """A case's inputs, with garbage where nothing may look, the kernels' outputs and the definition's."""

    def __init__(self, torch, rng, c):
        self.torch, self.rng, self.c = torch, rng, c
        g = torch.Generator(device="cuda").manual_seed(c["seed"] * 1000 + c["n"] + c["lk"])
        dt, r = getattr(torch, c["dtype"]), random.Random(c["seed"])

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

        self.q = normal(c["b"], c["n"], c["h"], c["d"], scale=c["spread"])
        self.k, self.v = (normal(c["b"], c["lk"], c["hk"], c["d"]) for _ in range(2))
        self.table = normal(c["buckets"], c["h"]) if c["buckets"] else None
        room = c["lk"] - c["n"]
        self.cached = [room] * c["b"] if c["cached"] is None else [min(max(x, 0), room) for x in c["cached"]]
        self.lengths = None if c["cached"] is None else torch.tensor(c["cached"], dtype=torch.int32, device="cuda")
        self.trees = {"chain": lambda i: list(range(-1, c["n"] - 1)), "bushy": lambda i: bushy(r, c["n"]),
                      "star": lambda i: [-1] + [0] * (c["n"] - 1), "roots": lambda i: bushy(r, c["n"], 1 + c["n"] // 3),
                      "apart": lambda i: [-1] * c["n"],
                      # smaller trees: the last nodes absent, or one in the middle with all below it
                      "padded": lambda i: [p if j < max(0, c["n"] - 3 * i) else -2 for j, p in enumerate(bushy(r, c["n"]))],
                      "broken": lambda i: [r.choice([p, p, p, j, j + 5, -7, 1 << 30, -(1 << 31)]) for j, p in enumerate(bushy(r, c["n"]))],
                      }
        self.trees = [self.trees[c["parents"]](i) for i in range(c["b"])]
        self.parents = None
        if c["parents"] != "chain":
            self.parents = torch.tensor(self.trees, dtype=torch.int32, device="cuda")
        import draft_reference as ref
        for b, n in enumerate(self.cached):
            gone = [n + i for i, line in enumerate(ref.lines(self.trees[b])) if not line] + list(range(n + c["n"], c["lk"]))
            self.k[b, gone], self.v[b, gone] = float("nan"), float("inf")
        self.scale = c["d"] ** -0.5 if c["scale"] is None else c["scale"]
        self.options = dict(cache_lengths=self.lengths, parents=self.parents, bias_table=self.table,
                            max_distance=c["far"], bidirectional=c["two_way"], scale=c["scale"])

    def forward(self, **more):
        torch, c = self.torch, self.c
        o = torch.full_like(self.q, float("nan"))
        lse = torch.full((c["b"], c["h"], c["n"]), float("nan"), device="cuda")
        self.rng.rng_tree_attention_fwd(self.q, self.k, self.v, o, lse=lse, **{**self.options, **more})
        return o, lse

    def check(self, o=None, lse=None, term=None):
        import draft_reference as ref
        torch, c = self.torch, self.c
        if o is None:
            o, lse = self.forward()
        ut = UT[c["dtype"]]
        term = ut if term is None else term
        bias = 0.0 if self.table is None else float(self.table.double().abs().max())
        for b in range(c["b"]):
            want, wlse, spread, most = ref.tree_attention(self.q[b], self.k[b], self.v[b], self.trees[b], self.cached[b],
                                                          self.scale, self.table, c["far"], c["two_way"])
            e = (c["d"] + 8) * 2 * U * most + 2.0 ** -21 * (most + bias)
            tol = (term + 4 * e + 2.0 ** -19) * spread + ut * want.abs() + TINY[c["dtype"]]
            if c["dtype"] == "float16":
                seen = self.v[b, : self.cached[b] + c["n"]].double().abs().nan_to_num(posinf=0.0).sum(0)
                tol = tol + 2.0 ** -25 * seen.repeat_interleave(c["h"] // c["hk"], 0)
            for name, got, w, t in (("o", o[b], want, tol), ("lse", lse[b], wlse, e + 2.0 ** -20 * (1 + wlse.abs().nan_to_num(posinf=0.0)))):
                bad = ~((got.double() == w) | ((got.double() - w).abs() <= t))
                assert not bad.any(), (name, b, int(bad.sum()), bad.nonzero()[0].tolist(), float(((got.double() - w).abs() / t)[bad].max()))


CASES = {
    "one_token": case(b=1, n=1, lk=1, h=1), "one_token_cached": case(b=1, n=1, lk=300, h=8, d=64, buckets=32),
    "nothing_cached": case(n=9, lk=9), "two": case(n=2, lk=65, dtype="float16"), "chain": case(n=17, lk=300, parents="chain"),
    "tile": case(n=16, lk=128), "tile_less_one": case(n=7, lk=127), "tile_and_one": case(n=9, lk=129, dtype="float16"),
    "straddles": case(b=5, n=40, lk=300, cached=[100, 127, 128, 90, 0]),
    "nodes_127": case(n=127, lk=400, h=1), "nodes_128": case(n=128, lk=500, h=2, d=128, dtype="float16"),
    "star": case(n=33, lk=200, parents="star"), "apart": case(n=65, lk=200, parents="apart"),
    "roots": case(n=50, lk=170, parents="roots", buckets=16),
    "padded": case(b=4, n=12, lk=150, parents="padded", cached=[138, 5, 0, 77]),
    "broken": case(b=7, n=30, lk=260, parents="broken", cached=[230, 0, 1, 98, 128, 99, 64]),
    "ragged": case(b=6, n=6, lk=700, cached=[0, 694, 1, 122, 128, 333], h=4, hk=2),
    "ragged_out_of_range": case(b=3, n=5, lk=90, cached=[-5, 1000, 85]),
    "group_2": case(n=64, lk=333, h=4, hk=2, d=128), "group_3": case(n=20, lk=333, h=6, hk=2, d=128),
    "group_3_wide": case(n=100, lk=333, h=3, hk=1), "group_5": case(n=3, lk=222, h=5, hk=1, d=72),
    "group_8": case(n=16, lk=444, h=8, hk=1, d=128), "group_8_wide": case(n=64, lk=600, h=16, hk=2, d=128),
    "group_16": case(n=8, lk=100, h=16, hk=1, d=96, dtype="float16"), "group_64": case(n=3, lk=300, h=64, hk=1),
    "group_200": case(b=1, n=2, lk=300, h=200, hk=1, d=16),
    "dim_8": case(n=5, lk=70, d=8), "dim_40": case(b=5, n=7, lk=122, h=6, d=40, dtype="float16", buckets=20, cached=[0, 115, 3, 64, 80]),
    "dim_72": case(n=11, lk=200, d=72), "dim_120": case(n=60, lk=300, d=120, h=4, hk=1, dtype="float16"),
    "buckets": case(n=12, lk=700, h=4, hk=1, buckets=32, far=128), "buckets_far": case(b=1, n=30, lk=1500, h=2, hk=1, buckets=64, far=1024),
    "buckets_one_way": case(n=20, lk=200, buckets=32, two_way=False), "buckets_few": case(n=20, lk=200, buckets=4, far=2),
    "buckets_many": case(n=9, lk=300, buckets=128, far=300, h=3, hk=1, d=128), "buckets_wide": case(n=90, lk=400, h=4, hk=1, buckets=32, d=128),
    "buckets_group_20": case(n=4, lk=1300, h=20, hk=1, buckets=32, far=1024, two_way=False),
    "buckets_chain": case(n=128, lk=260, parents="chain", buckets=16, far=40, dtype="float16"),
    "long": case(b=1, n=5, lk=9000, h=2, d=128, dtype="float16", parents="chain"), "long_wide": case(b=1, n=64, lk=5000, h=8, hk=2, d=128),
    "sharp": case(n=30, lk=300, spread=20.0), "sharp_f16": case(n=30, lk=300, spread=20.0, dtype="float16"),
    "scale_0": case(n=9, lk=200, scale=0.0), "scale_below_0": case(n=9, lk=200, scale=-0.2, buckets=16),
    "scale_1": case(n=40, lk=400, scale=1.0, h=4, hk=1, spread=0.5),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_tree_attention_against_its_definition(torch, rng, name):
    Run(torch, rng, CASES[name]).check()
    assert rng.rng_debug_stalled_waits() == 0


# more pieces of work than SMs, of unequal lengths
MANY = {
    "requests": case(b=64, n=8, lk=400, h=8, hk=2, d=128, cached=[(97 * i) % 393 for i in range(64)]),
    "short": case(b=300, n=3, lk=20, h=4, hk=4, cached=[i % 18 for i in range(300)], dtype="float16"),
    "long_and_short": case(b=24, n=16, lk=3000, h=8, hk=4, d=64, cached=[2984 if i % 7 == 3 else i for i in range(24)], parents="padded"),
    "wide": case(b=12, n=96, lk=700, h=16, hk=4, d=128, cached=[(211 * i) % 605 for i in range(12)]),
    "bias": case(b=20, n=12, lk=900, h=12, hk=3, d=96, buckets=32, cached=[(331 * i) % 889 for i in range(20)], dtype="float16"),
    # more entries than a block has threads
    "a_thousand": case(b=1000, n=2, lk=40, h=2, hk=1, d=16, cached=[(7 * i) % 39 for i in range(1000)], parents="padded"),
    "hundreds_wide": case(b=660, n=17, lk=130, h=8, hk=1, d=8, cached=[(7 * i) % 114 for i in range(660)], dtype="float16"),
    "hundreds_cut": case(b=500, n=3, lk=1500, h=4, hk=2, d=64, cached=[1497 if i % 61 == 7 else i % 50 for i in range(500)], buckets=8),
    "empty": case(b=40, n=6, lk=300, h=6, hk=2, parents="broken", cached=[(53 * i) % 295 for i in range(40)]),
}


# (Since these were written, past six key tiles two tiles of rows share their keys from ten key tiles a block on: CUT_PAIRS
# below has those; and test_as_much_work_as_the_device_holds the borders themselves.)
# More than 128 rows of a key head, and work enough that two tiles of rows share their keys: more tiles than SMs, or, past
# six key tiles, more than three of those for each SM and pair.
WIDE = {
    "group_2": case(n=128, lk=260, h=80, hk=40), "group_3": case(n=100, lk=333, h=180, hk=60),
    "group_8": case(n=64, lk=600, h=160, hk=20, d=128), "group_64": case(n=3, lk=300, h=2560, hk=40),
    "group_200": case(b=1, n=2, lk=300, h=10000, hk=50, d=16), "dim_120": case(n=60, lk=300, d=120, h=160, hk=40, dtype="float16"),
    "nothing_cached": case(n=90, lk=90, h=104, hk=26, parents="roots"), "apart": case(n=65, lk=200, h=104, hk=26, parents="apart"),
    "padded": case(b=20, n=70, lk=300, h=16, hk=4, parents="padded", cached=[(37 * i) % 231 for i in range(20)]),
    "broken": case(b=20, n=70, lk=300, h=16, hk=4, parents="broken", cached=[(37 * i) % 231 for i in range(20)], buckets=16),
    "buckets": case(n=90, lk=400, h=104, hk=26, buckets=32, d=128), "buckets_group_20": case(n=30, lk=600, h=280, hk=14, buckets=32, far=128, two_way=False),
    "sharp": case(n=64, lk=300, h=160, hk=40, spread=20.0, dtype="float16"),
    "cut": case(b=2, n=64, lk=9000, h=32, hk=8, d=128), "cut_one": case(b=1, n=100, lk=9000, h=16, hk=4, dtype="float16"),
    "cut_ragged": case(b=12, n=96, lk=1500, h=16, hk=4, d=128, cached=[(211 * i) % 1405 for i in range(12)]),
    "cut_buckets": case(b=12, n=96, lk=1500, h=16, hk=4, buckets=32, cached=[(211 * i) % 1405 for i in range(12)], dtype="float16", parents="padded"),
    "cut_chain": case(b=8, n=128, lk=1300, h=16, hk=8, buckets=16, far=40, parents="chain"),
}
# and nearly: the most tiles of rows that have an SM each, three key tiles for each SM and pair
NEAR = {"uncut": case(b=1, n=64, lk=700, h=152, hk=38), "uncut_bias": case(b=3, n=100, lk=300, h=48, hk=12, buckets=32, dtype="float16", d=128),
        "cut": case(b=2, n=64, lk=1700, h=64, hk=16, d=128), "cut_bias": case(b=3, n=40, lk=1800, h=28, hk=4, buckets=20, cached=[0, 1760, 900]),
        "cut_long": case(b=1, n=64, lk=9000, h=16, hk=4, d=128, parents="chain")}


@pytest.mark.gpu
@pytest.mark.parametrize("name", WIDE)
def test_tree_attention_of_many_rows(torch, rng, name):
    Run(torch, rng, WIDE[name]).check()
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", NEAR)
def test_tree_attention_of_many_rows_and_little_work(torch, rng, name):
    Run(torch, rng, NEAR[name]).check()
    assert rng.rng_debug_stalled_waits() == 0


# Two tiles of rows to a block past six key tiles: an even number of them, and more than ten key tiles a block.
CUT_PAIRS = {
    "long": case(b=4, n=64, lk=9000, h=32, hk=8, d=128), "long_f16": case(b=2, n=100, lk=9100, h=64, hk=16, dtype="float16"),
    "ragged": case(b=24, n=100, lk=1500, h=16, hk=4, d=128, cached=[(211 * i) % 1401 for i in range(24)]),
    "ragged_padded": case(b=24, n=97, lk=1500, h=16, hk=4, cached=[(307 * i) % 1404 for i in range(24)], parents="padded", dtype="float16"),
    "ragged_broken": case(b=24, n=128, lk=1500, h=16, hk=4, cached=[(101 * i) % 1373 for i in range(24)], parents="broken", buckets=16),
    "buckets": case(b=12, n=64, lk=3000, h=32, hk=8, d=96, buckets=32, far=128, cached=[2936 - 200 * i for i in range(12)]),
    "chain": case(b=24, n=128, lk=1300, h=16, hk=8, buckets=16, far=40, parents="chain"),
    "sharp": case(b=20, n=64, lk=900, h=32, hk=8, spread=20.0), "short_and_long": case(b=24, n=64, lk=2000, h=32, hk=8, cached=[1936 if i % 5 == 2 else i for i in range(24)]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CUT_PAIRS)
def test_tree_attention_of_many_rows_cut(torch, rng, name):
    Run(torch, rng, CUT_PAIRS[name]).check(term=UT[CUT_PAIRS[name]["dtype"]] ** 2)
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lk", (200, 1280))
@pytest.mark.parametrize("sms,more", ((0.5, 0), (0.5, 1), (1, 0), (1, 1), (1.5, 0), (1.5, 1), (2, 0)))
def test_as_much_work_as_the_device_holds(torch, rng, lk, sms, more):
    """Pairs of tiles of rows for a share of the SMs and one more: on each side of where one or two tiles go to a block."""
    pairs = int(torch.cuda.get_device_properties(0).multi_processor_count * sms) + more
    Run(torch, rng, case(b=1, n=64, lk=lk, h=4 * pairs, hk=pairs)).check(term=UT["bfloat16"] ** 2)
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", MANY)
def test_tree_attention_of_many_requests(torch, rng, name):
    Run(torch, rng, MANY[name]).check()
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("buckets", (0, 8))
def test_each_node_sees_its_line(torch, rng, buckets):
    """Keys of 0 and a value of its own axis for each node: a node's output says whom it sees.  300 trees of 128 nodes, as
    deep as there are and as steps that double reach, several a block."""
    r, n, b = random.Random(8), 128, 300
    kinds = (lambda i: i - 1, lambda i: i - 2, lambda i: i - 31, lambda i: i // 2, lambda i: i - 1 - r.randrange(3),
             lambda i: r.randrange(i), lambda i: i - 33 if i > 40 else i - 1, lambda i: r.choice([i - 1, i - 1, i - 1, i - 5, i + 1]))
    trees = [[-1] + [max(kinds[e % len(kinds)](i), -1 if e % 3 else 0) for i in range(1, n)] for e in range(b)]
    import draft_reference as ref
    lines = [ref.lines(t) for t in trees]
    sees = torch.zeros(b, n, n, dtype=torch.bool)
    for e in range(b):
        for i, line in enumerate(lines[e]):
            sees[e, i, line] = True
    sees = sees.cuda()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.randn(b, n, 1, n, **bf), torch.zeros(b, n, 1, n, **bf)
    v = torch.eye(n, **bf).expand(b, n, n).contiguous().view(b, n, 1, n)
    table = torch.zeros(buckets, 1, **bf) if buckets else None
    o, lse = torch.empty_like(q), torch.empty(b, 1, n, device="cuda")
    for _ in range(3):
        rng.rng_tree_attention_fwd(q, k, v, o, lse=lse, parents=torch.tensor(trees, dtype=torch.int32, device="cuda"),
                                   bias_table=table, max_distance=16)
        assert torch.equal(o[:, :, 0] != 0, sees)
        count = sees.sum(2).double()
        # log of the count of terms 1, each to 2^-22
        assert bool(((lse[:, 0].double() - count.log()).abs() <= 2.0 ** -20 * (1 + count.log()))[count > 0].all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("d,h,hk,n", ((128, 8, 2, 16), (64, 4, 4, 128), (40, 3, 1, 9)))
def test_few_rows_of_a_key_head_take_two_terms(torch, rng, dtype, d, h, hk, n):
    r = Run(torch, rng, case(n=n, lk=700, h=h, hk=hk, d=d, dtype=dtype))
    r.check(term=UT[dtype] ** 2)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ("group_3", "group_8", "dim_120", "padded", "buckets", "sharp", "cut", "cut_one", "cut_ragged", "cut_buckets"))
def test_many_rows_of_a_key_head_take_two_terms(torch, rng, name):
    Run(torch, rng, WIDE[name]).check(term=UT[WIDE[name]["dtype"]] ** 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("n,lk", ((64, 700), (64, 4163), (128, 400)))
def test_neighbours_do_not_change_a_requests_rounding(torch, rng, dtype, n, lk):
    """A request alone, among few and among many, and with a cache that has room for more: two terms throughout."""
    for b, room in ((1, 0), (8, 0), (24, 0), (1, 3000)):
        r = Run(torch, rng, case(b=b, n=n, lk=lk + room, h=32, hk=8, d=64, dtype=dtype, cached=[lk - n] * b))
        o, lse = r.forward()
        r.c["b"] = 1  # (the others are checked in one of the batches)
        r.check(o[:1], lse[:1], term=UT[dtype] ** 2)


@pytest.mark.gpu
def test_tree_attention_as_attention_sees_a_chain(torch, rng):
    """A chain is what causal attention gives the last queries, to both operators' roundings."""
    for n, h, hk, d, buckets in ((5, 8, 2, 128, 0), (9, 4, 4, 64, 32)):
        r = Run(torch, rng, case(b=3, n=n, lk=500, h=h, hk=hk, d=d, parents="chain", cached=[100, 0, 495], buckets=buckets))
        o, lse = r.forward()
        same, lse2 = torch.empty_like(o), torch.empty_like(lse)
        rng.rng_attention_fwd(r.q, r.k, r.v, same, lse=lse2, key_lengths=r.lengths.clamp(max=500 - n) + n, causal=True,
                              queries_last=True, bias_table=r.table, max_distance=64)
        assert float((lse - lse2).abs().max()) < 1e-4
        assert float((o.float() - same.float()).abs().max()) < 2.0 ** -6 * float(same.float().abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("buckets", (0, 16))
@pytest.mark.parametrize("n,h,hk,d", ((20, 4, 2, 64), (100, 8, 2, 128), (100, 80, 20, 128)))
def test_what_a_node_does_not_see_has_no_influence(torch, rng, buckets, n, h, hk, d):
    """Infinities and NaN in one node's query, key or value reach the nodes below it alone."""
    r = Run(torch, rng, case(b=2, n=n, lk=300, h=h, hk=hk, d=d, cached=[123, 40], buckets=buckets))
    clean, clean_lse = r.forward()
    import draft_reference as ref
    bad = 7
    sees = torch.tensor([bad in line for line in ref.lines(r.trees[0])], device="cuda")
    for name, value in (("v", math.inf), ("v", math.nan), ("k", math.nan), ("v", -math.inf), ("q", math.nan)):
        t = getattr(r, name)
        row = t[0, bad] if name == "q" else t[0, 123 + bad]
        before = row.clone()
        row[0 if name != "v" else slice(None), :] = value
        o, lse = r.forward()
        hit = torch.zeros_like(sees) if name == "q" else sees.clone()
        hit[bad] = True
        assert torch.equal(o[0][~hit], clean[0][~hit]) and torch.equal(o[1], clean[1]), name
        assert torch.equal(lse[0][:, ~hit], clean_lse[0][:, ~hit])
        if name == "v":
            assert torch.equal(lse, clean_lse)
            assert bool((o[0][hit] == value).all() if value == value else o[0][hit].isnan().all())
        else:
            assert bool(o[0, bad, 0].isnan().all())
        row.copy_(before)
    assert rng.rng_debug_stalled_waits() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lk", (300, 3000, 20000))
@pytest.mark.parametrize("value", (math.inf, -math.inf, math.nan))
def test_an_infinite_value_of_hardly_any_weight(torch, rng, lk, value):
    """A node's value that is not finite reaches whoever sees it, also where a cached row's score is 400 above all others
    and the keys are cut: P is more than 0 there, whatever of it f32 holds."""
    n, h, d = 9, 8, 64
    r = Run(torch, rng, case(b=2, n=n, lk=lk, h=h, hk=2, d=d))
    r.q[:] = 1.0
    r.k.mul_(0.01)
    r.k[:, 5] = 50.0  # 64 x 50 / 8 = 400
    clean, _ = r.forward()
    import draft_reference as ref
    bad = 3
    sees = torch.tensor([bad in line for line in ref.lines(r.trees[0])], device="cuda")
    r.v[0, lk - n + bad] = value
    o, _ = r.forward()
    assert torch.equal(o[0][~sees], clean[0][~sees]) and torch.equal(o[1], clean[1])
    assert bool((o[0][sees] == value).all() if value == value else o[0][sees].isnan().all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
def test_tree_attention_with_a_bias_as_a_mask(torch, rng, dtype):
    """-inf hides distances; everywhere, it leaves rows that see nothing; the type's lowest value everywhere leaves
    the average (bf16; in f16 it leaves room for the scores)."""
    r = Run(torch, rng, case(n=10, lk=200, h=3, hk=1, buckets=8, far=16, dtype=dtype))
    lowest = torch.finfo(r.q.dtype).min
    r.table[:, 0] = -math.inf
    r.table[1:, 1] = -math.inf  # itself alone
    r.table[:, 2] = lowest
    o, lse = r.forward()
    assert bool((o[:, :, 0] == 0).all()) and bool((lse[:, 0] == -math.inf).all())
    assert torch.equal(o[:, :, 1], r.v[:, 190:, 0])
    if dtype == "bfloat16":
        import draft_reference as ref
        for b in range(2):
            for i, line in enumerate(ref.lines(r.trees[b])):
                mean = r.v[b, list(range(190)) + [190 + t for t in line], 0].double().mean(0)
                assert bool(((o[b, i, 2].double() - mean).abs() <= 2.0 ** -7).all())


@pytest.mark.gpu
def test_tree_attention_layouts(torch, rng):
    """Heads outermost, keys and values in one array, a slice of a wider output: nothing beside it is written."""
    r = Run(torch, rng, case(b=3, n=11, lk=333, h=6, hk=2, d=64, buckets=16, cached=[10, 322, 128]))
    o, lse = r.forward()
    r.check(o, lse)
    plain = {n: getattr(r, n) for n in "qkv"}
    for n, t in plain.items():
        setattr(r, n, t.transpose(1, 2).contiguous().transpose(1, 2))
    again, lse2 = r.forward()
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    r.q, (r.k, r.v) = plain["q"], torch.stack([plain["k"], plain["v"]], 2).unbind(2)
    again, lse2 = r.forward()
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    wide = torch.full((5, 15, 9, 80), 7.0, dtype=o.dtype, device="cuda")
    rng.rng_tree_attention_fwd(r.q, r.k, r.v, wide[1:4, 2:13, 1:7, 8:72], **r.options)
    assert torch.equal(wide[1:4, 2:13, 1:7, 8:72], o)
    wide[1:4, 2:13, 1:7, 8:72] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,hk,d,lk,b", ((6, 8, 2, 128, 3000, 3), (64, 8, 2, 128, 900, 2), (4, 2, 2, 64, 60, 2), (64, 64, 16, 128, 2000, 3),
                                            (64, 96, 24, 64, 700, 4)))
def test_tree_attention_twice_in_a_graph_and_on_another_stream(torch, rng, n, h, hk, d, lk, b):
    r = Run(torch, rng, case(b=b, n=n, h=h, hk=hk, d=d, lk=lk))
    o, lse = r.forward()
    o2, lse2 = r.forward()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = r.forward(stream=side)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    need = rng.rng_tree_attention_fwd_workspace(r.q, r.k)
    workspace = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):  # of one workspace, replayed one after the other
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(r.forward(workspace=workspace if need else None))
    for _ in range(3):
        for g, (og, lg) in zip(graphs, outs):
            og.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(og, o) and torch.equal(lg, lse)


@pytest.mark.gpu
def test_tree_attention_refuses_a_workspace(torch, rng):
    """(How the work is cut, and so the size, goes by the device.)"""
    r = Run(torch, rng, case(b=4, n=6, h=8, hk=2, d=128, lk=8000))
    need = rng.rng_tree_attention_fwd_workspace(r.q, r.k)
    assert 0 < need <= r.k.numel() * 2 and rng.rng_tree_attention_fwd_workspace(r.q[:, :2], r.k[:, :600]) == 0
    for workspace in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need + 16, dtype=torch.uint8, device="cuda")[1:]):
        with pytest.raises(rng.RngError, match="workspace"):
            r.forward(workspace=workspace)
    with pytest.raises(rng.RngError, match="k and workspace overlap"):
        r.forward(workspace=r.k.view(-1))
    o, lse = r.forward(workspace=torch.full((need + 1000,), 255, dtype=torch.uint8, device="cuda"))
    r.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("h,hk", ((8, 2), (64, 16)))
def test_calls_on_two_streams_at_once(torch, rng, h, hk):
    runs = [Run(torch, rng, case(b=3, n=n, h=h, hk=hk, d=128, lk=3000, seed=n, buckets=b)) for n, b in ((6, 0), (40, 32))]
    want = [r.forward() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        got.append([])
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                got[-1].append(r.forward())
    torch.cuda.synchronize()
    for pair in got:
        for (o, lse), (wo, wlse) in zip(pair, want):
            assert torch.equal(o, wo) and torch.equal(lse, wlse)


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,hk", ((8, 8, 2), (64, 64, 16)))
def test_lengths_that_a_graph_sees_change(torch, rng, n, h, hk):
    """The cut of the work goes by the lengths that a replay finds."""
    r = Run(torch, rng, case(b=4, n=n, lk=2500, h=h, hk=hk, d=128, cached=[2000, 0, 17, 900]))
    graph = torch.cuda.CUDAGraph()
    r.forward()
    with torch.cuda.graph(graph):
        o, lse = r.forward()
    for lengths in ([2000, 0, 17, 900], [0, 0, 0, 0], [2492, 2492, 2492, 2492], [1, 2000, 128, 127]):
        r.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        want, wlse = r.forward()
        assert torch.equal(o, want) and torch.equal(lse, wlse)
        r.cached = [min(x, 2500 - n) for x in lengths]
        r.k.nan_to_num_(nan=0.5), r.v.nan_to_num_(posinf=0.5)
        graph.replay()
        torch.cuda.synchronize()
        r.check(o, lse)


@pytest.mark.gpu
def test_caches_past_2_to_32_elements(torch, rng):
    """Batch entries that lie more than 2^32 elements apart, in every operator."""
    step = (1 << 32) + 64
    store = torch.empty(2 * step, dtype=torch.bfloat16, device="cuda")
    far = store.as_strided((2, 300, 2, 64), (step, 128, 64, 1))
    far.copy_(torch.randn(2, 300, 2, 64, device="cuda"))
    r = Run(torch, rng, case(b=2, n=6, lk=300, h=4, hk=2))
    r.k = r.v = far
    r.check()
    path = torch.tensor([[0, 2, 4, -1, -1, -1], [0, 5, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    before = far.contiguous()
    import draft_reference as ref
    rng.rng_cache_keep([far], path, torch.tensor([2, 1], dtype=torch.int32, device="cuda"))
    for b, kept in enumerate((2, 1)):
        assert torch.equal(far[b], ref.keep(before[b], path[b].tolist(), kept, 294))
    probabilities = store.as_strided((2, 2, 50), (step, 50, 1))
    probabilities.copy_(torch.softmax(torch.randn(2, 2, 50, device="cuda"), 2))
    check_verify(torch, rng, probabilities, None, torch.tensor([[0, 3], [0, 4]]), None, torch.rand(2, 2))


# ---- verification ------------------------------------------------------------------------


def run_verify(torch, rng, target, draft, tokens, parents, u, **more):
    b, n = tokens.shape
    path, out = (torch.full((b, n), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    accepted = torch.full((b,), -9, dtype=torch.int32, device="cuda")
    move = lambda t, dtype: None if t is None else t.to("cuda", dtype)  # noqa: E731
    rng.rng_verify_drafts(target, move(tokens, torch.int32), path, accepted, out, draft=draft,
                          parents=move(parents, torch.int32), uniforms=move(u, torch.float32), **more)
    return path, accepted, out


def check_verify(torch, rng, target, draft, tokens, parents, u, got=None):
    import draft_reference as ref
    path, accepted, out = run_verify(torch, rng, target, draft, tokens, parents, u) if got is None else got
    n = tokens.shape[1]
    target = target.double().tolist()
    draft = None if draft is None else draft.double().tolist()
    for b in range(len(target)):
        tree = list(range(-1, n - 1)) if parents is None else parents[b].tolist()
        want_path, want_out = ref.verify(target[b], None if draft is None else draft[b], tokens[b].tolist(), tree,
                                         u[b].float().tolist())
        assert accepted[b] == len(want_path) - 1, b
        assert path[b].tolist() == want_path + [-1] * (n - len(want_path)), b
        assert out[b].tolist() == want_out + [-1] * (n - len(want_out)), b


def drafted(torch, g, b, n, vocab, dtype, near=0.5, sharp=2.0):
    """Probabilities of a target and of a draft near it, on the GPU."""
    logits = torch.randn(b, n, vocab, generator=g) * sharp
    draft = logits + near * torch.randn(b, n, vocab, generator=g)
    return (torch.softmax(x, 2).to("cuda", getattr(torch, dtype)) for x in (logits, draft))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("float32", "bfloat16", "float16"))
@pytest.mark.parametrize("kind", ("drawn", "chosen"))
@pytest.mark.parametrize("b,n,vocab,tree", ((1, 1, 1, "chain"), (5, 1, 40, "chain"), (40, 2, 2, "chain"), (30, 6, 33, "chain"), (30, 9, 64, "bushy"),
                                            (30, 17, 7, "star"), (12, 128, 5, "bushy"), (6, 33, 257, "star"), (10, 40, 12, "broken"),
                                            (4, 6, 2049, "bushy"), (3, 5, 4099, "star"), (2, 4, 20011, "chain")))
def test_verification_against_exact_arithmetic(torch, rng, dtype, kind, b, n, vocab, tree):
    g = torch.Generator().manual_seed(n * 1000 + vocab)
    r = random.Random(n + vocab)
    target, draft = drafted(torch, g, b, n, vocab, dtype)
    trees = [[-1] + [0] * (n - 1) if tree == "star" else bushy(r, n) for _ in range(b)]
    if tree == "broken":
        trees = [[r.choice([p, p, p, j, j + 3, -1, -2, 1 << 30]) for j, p in enumerate(t)] for t in trees]
    parents = None if tree == "chain" else torch.tensor(trees)
    row = torch.arange(-1, n - 1).expand(b, n) if parents is None else parents
    row = torch.where((row >= 0) & (row < n), row, 0)
    tokens = torch.multinomial(draft.float().cpu().gather(1, row[:, :, None].expand(b, n, vocab)).reshape(b * n, vocab), 1,
                               generator=g).view(b, n)
    if tree == "broken":
        tokens = torch.where(torch.rand(b, n, generator=g) < 0.2, torch.tensor(r.choice([-1, vocab, 1 << 30])), tokens)
    u = torch.rand(b, n, generator=g)
    u[0, 0] = 0.0
    check_verify(torch, rng, target, draft if kind == "drawn" else None, tokens, parents, u)


@pytest.mark.gpu
def test_verification_at_its_borders(torch, rng):
    """Probabilities in eighths and random numbers in sixteenths: sums and products are exact, many comparisons equal."""
    g = torch.Generator().manual_seed(4)
    b, n, vocab = 300, 6, 9
    eighths = torch.zeros(2, b, n, vocab)
    for _ in range(8):
        eighths.scatter_add_(3, torch.randint(vocab, (2, b, n, 1), generator=g), torch.full((2, b, n, 1), 0.125))
    tokens, u = torch.randint(vocab, (b, n), generator=g), torch.randint(16, (b, n), generator=g) / 16
    target, draft = eighths.cuda()
    r = random.Random(3)
    parents = torch.tensor([bushy(r, n) for _ in range(b)])
    check_verify(torch, rng, target, draft, tokens, parents, u)
    check_verify(torch, rng, target, None, tokens, parents, u)
    check_verify(torch, rng, target, target, tokens, None, u)  # the draft's distribution itself: all is accepted, or was not drawn


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", (6, 700, 9000))
def test_verification_without_any_weight(torch, rng, vocab):
    """Drafts above the target everywhere leave nothing: p itself then; a row of zeros, NaN or less: -1."""
    p = torch.zeros(4, 2, vocab)
    p[:2, 0, 5] = 1.0
    p[2, 0], p[3, 0] = float("nan"), -1.0
    q = torch.full((4, 2, vocab), 2.0)
    u = torch.full((4, 2), 0.999)
    for draft in (q.cuda(), None):
        path, accepted, out = run_verify(torch, rng, p.cuda(), draft, torch.zeros(4, 2), None, u)
        assert accepted.tolist() == [0] * 4 and path.tolist() == [[0, -1]] * 4
        assert out.tolist() == [[5, -1], [5, -1], [-1, -1], [-1, -1]]


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", (7, 3001, 20000))
@pytest.mark.parametrize("kind", ("drawn", "chosen"))
def test_numbers_that_are_no_probabilities(torch, rng, vocab, kind):
    """Infinities, NaN and less than 0 among the probabilities, any random numbers and tokens: each walk ends with a path of
    its tree, the same each time, and other entries are what they are without them."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    b, n = 24, 9
    target, draft = torch.rand(2, b, n, vocab, generator=g, device="cuda") * (2.0 / vocab)
    tokens = torch.randint(vocab, (b, n), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(b, n, generator=g, device="cuda")
    r = random.Random(vocab)
    trees = [bushy(r, n) for _ in range(b)]
    parents = torch.tensor(trees, dtype=torch.int32, device="cuda")
    with_draft = lambda: draft if kind == "drawn" else None
    plain = run_verify(torch, rng, target, with_draft(), tokens, parents, u)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -1.0, 3e38, 1e-45], device="cuda")
    for t in (target, draft):
        for e in range(0, b, 2):
            t[e, :, r.randrange(vocab)] = odd[e // 2 % 6]
            t[e, 0, tokens[e, 1 + e % (n - 1)].item()] = odd[(e // 2 + 1) % 6]
    for e in range(0, b, 2):
        u[e, r.randrange(n)] = (math.nan, math.inf, -1.0, 1.0)[e // 2 % 4]
        tokens[e, r.randrange(1, n)] = (-1, vocab, 2 ** 31 - 1, -2 ** 31)[e // 2 % 4]
    got = run_verify(torch, rng, target, with_draft(), tokens, parents, u)
    for x, y in zip(got, run_verify(torch, rng, target, with_draft(), tokens, parents, u)):
        assert torch.equal(x, y)
    for x, y in zip(got, plain):
        assert torch.equal(x[1::2], y[1::2])
    path, accepted, out = (x.tolist() for x in got)
    for e in range(b):
        k = accepted[e]
        assert 0 <= k < n and path[e][0] == 0 and path[e][k + 1:] == [-1] * (n - 1 - k) and out[e][k + 1:] == [-1] * (n - 1 - k)
        assert all(trees[e][y] == x for x, y in zip(path[e][:k], path[e][1:k + 1]))
        assert out[e][:k] == [int(tokens[e, i]) for i in path[e][1:k + 1]] and all(0 <= t < vocab for t in out[e][:k])
        assert -1 <= out[e][k] < vocab


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("float32", "bfloat16"))
@pytest.mark.parametrize("vocab", (7, 33, 256, 700, 2049, 4096, 8200, 32768))
@pytest.mark.parametrize("odd", (math.nan, math.inf, -math.inf, "all"))
def test_draft_probabilities_that_nothing_was_drawn_from_have_no_say(torch, rng, vocab, dtype, odd):
    """Where no child was rejected w is p, whatever the draft row holds: rows of leaves, of nodes whose children have no
    valid token and of nodes that the walk passes by; and, where the first child stands, all of its row but its token's."""
    import draft_reference as ref
    g, r = torch.Generator().manual_seed(vocab), random.Random(vocab)
    b, n = (12, 6) if vocab < 3000 else (5, 4)
    # sums that are known but for the rounding of their type: the draft is the target for some entries, so that whole lines stand
    target, draft = drafted(torch, g, b, n, vocab, dtype)
    draft[::2] = target[::2]
    trees = [list(range(-1, n - 1)) if e % 4 == 0 else bushy(r, n) for e in range(b)]
    rows = torch.tensor(trees).clamp(min=0)
    tokens = torch.multinomial(draft.float().cpu().gather(1, rows[:, :, None].expand(b, n, vocab)).reshape(b * n, vocab), 1,
                               generator=g).view(b, n)
    tokens[1::4, 1:] = torch.tensor([vocab, -1] * n)[:n - 1]  # none of them valid
    u = torch.rand(b, n, generator=g)
    given = draft.clone()
    filling = torch.tensor([math.nan, math.inf, -math.inf, 3.0]) if odd == "all" else torch.tensor([odd])
    wanted = []
    for e in range(b):
        path, out = ref.verify(target[e].double().tolist(), draft[e].double().tolist(), tokens[e].tolist(), trees[e], u[e].tolist())
        wanted.append((path, out))
        for i in range(n):
            tried = [j for j in range(n) if trees[e][j] == i and 0 <= tokens[e, j] < vocab]
            used = torch.zeros(vocab, dtype=torch.bool)
            if i in path and tried:
                if i != path[-1] and path[path.index(i) + 1] == tried[0]:
                    used[tokens[e, tried[0]]] = True
                else:
                    used[:] = True
            poison = filling[torch.randint(len(filling), (vocab,), generator=g)]
            given[e, i] = torch.where(used.cuda(), given[e, i], poison.cuda().to(given.dtype))
    assert not torch.equal(given.nan_to_num(9.0), draft)
    path, accepted, out = run_verify(torch, rng, target, given, tokens, torch.tensor(trees), u)
    for e, (want_path, want_out) in enumerate(wanted):
        assert path[e].tolist() == want_path + [-1] * (n - len(want_path)), e
        assert accepted[e] == len(want_path) - 1 and out[e].tolist() == want_out + [-1] * (n - len(want_out)), e


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", (6, 700, 9000))
def test_an_infinite_draft_leaves_the_target(torch, rng, vocab):
    """A draft row of infinities rejects its child and leaves nothing: p itself then."""
    p = torch.zeros(3, 3, vocab, device="cuda")
    p[0, 0, 5], p[1, 0, vocab - 1], p[2, 0, 0], p[2, 0, 3] = 1.0, 1.0, 0.5, 0.5
    q = torch.full_like(p, math.inf)
    u = torch.full((3, 3), 0.75)
    path, accepted, out = run_verify(torch, rng, p, q, torch.tensor([[0, 5, 5], [0, 1, 2], [0, 3, 3]]), torch.tensor([[-1, 0, 0]] * 3), u)
    assert accepted.tolist() == [0] * 3 and out.tolist() == [[5, -1, -1], [vocab - 1, -1, -1], [3, -1, -1]]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ("drawn", "chosen"))
@pytest.mark.parametrize("vocab", (2048, 2100, 8192, 20000, 33000))
def test_the_size_of_a_batch_changes_no_token(torch, rng, vocab, kind):
    """How many blocks share a request goes by the batch too: a request's tokens are what they are alone."""
    g, n, most = torch.Generator(device="cuda").manual_seed(vocab), 5, 700
    logits = torch.randn(3, n, vocab, generator=g, device="cuda") * 2
    target, draft = torch.softmax(logits, 2), torch.softmax(logits + 0.5 * torch.randn(3, n, vocab, generator=g, device="cuda"), 2)
    parents = torch.tensor([[-1, 0, 0, 1, 0], [-1, 0, 1, 2, 3], [-1, 0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    rows = draft.gather(1, parents.clamp(min=0).long()[:, :, None].expand_as(draft)).reshape(3 * n, vocab)
    tokens = torch.multinomial(rows, most // 3 + 1, replacement=True, generator=g).view(3, n, -1).permute(2, 0, 1).reshape(-1, n)[:most].int()
    u = torch.rand(most, n, generator=g, device="cuda")
    entry = torch.arange(most, device="cuda") % 3
    fewer = None
    for b in (1, 2, 57, 114, 153, 228, 457, most):
        like = entry[:b]
        got = run_verify(torch, rng, target[like], draft[like] if kind == "drawn" else None, tokens[:b], parents[like], u[:b])
        if fewer:
            assert all(torch.equal(x[:len(y)], y) for x, y in zip(got, fewer)), b
        fewer = got
    if vocab < 9000:
        like = entry[:6]
        check_verify(torch, rng, target[like], draft[like] if kind == "drawn" else None, tokens[:6].cpu(), parents[like].cpu(), u[:6].cpu(),
                     tuple(x[:6] for x in fewer))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("float32", "float16"))
@pytest.mark.parametrize("vocab", (75000, 131072))
def test_rows_that_leave_more_than_a_block_keeps(torch, rng, vocab, dtype):
    """Draft rows below the target's at most tokens, and children that are all tried: later sums read what is kept and,
    from where there was no more room, the rows."""
    g = torch.Generator().manual_seed(vocab)
    n = 5
    target = torch.softmax(torch.randn(3, n, vocab, generator=g), 2)
    draft = target * (0.25 + 0.5 * torch.rand(3, n, vocab, generator=g))  # less than the target nearly everywhere,
    tokens = torch.randint(vocab, (3, n), generator=g)
    heavy = tokens[:, :, None].expand(3, n, n).transpose(1, 2)  # but not at the drafts
    draft.scatter_(2, heavy, 0.08)
    target, draft = (t.to("cuda", getattr(torch, dtype)) for t in (target, draft))
    u = torch.rand(3, n, generator=g)
    u[:, 1:] = 0.5 + u[:, 1:] / 2
    parents = torch.tensor([[-1, 0, 0, 0, 0]] * 3)
    check_verify(torch, rng, target, draft, tokens, parents, u)
    assert run_verify(torch, rng, target, draft, tokens, parents, u)[1].tolist() == [0] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ("drawn", "chosen"))
def test_the_largest_vocabulary(torch, rng, kind):
    """2^23 tokens of which 300 have any weight, the first and the last among them: as the 300 alone say."""
    import draft_reference as ref
    g, n, vocab, some = torch.Generator().manual_seed(2), 5, 1 << 23, 300
    at = torch.cat([torch.tensor([0, 1, vocab - 1]), torch.randperm(vocab - 10, generator=g)[:some - 3] + 5]).sort().values
    target, draft = drafted(torch, g, 1, n, some, "float32", near=1.0)
    wide = torch.zeros(2, 1, n, vocab, device="cuda")
    wide[0, :, :, at], wide[1, :, :, at] = target, draft
    for seed in range(12):
        parents = bushy(random.Random(seed), n)
        tokens, u = torch.randint(some, (n,), generator=g), torch.rand(n, generator=g)
        path, out = ref.verify(target[0].double().tolist(), draft[0].double().tolist() if kind == "drawn" else None, tokens.tolist(), parents, u.tolist())
        got = run_verify(torch, rng, wide[0], wide[1] if kind == "drawn" else None, at[tokens][None], torch.tensor([parents]), u[None])
        assert got[0][0].tolist() == path + [-1] * (n - len(path)) and got[1].item() == len(path) - 1
        assert got[2][0].tolist() == [int(at[t]) for t in out] + [-1] * (n - len(out))


def how_often(p, q, drawn):
    total = 0.0
    for triple in itertools.product(range(len(p)), repeat=3):
        w, mass, none = list(p), 1.0, 1.0
        for t in triple:
            none *= 1 - min(1.0, w[t] / (mass * q[t] if drawn else mass))
            if drawn:
                w = [max(a - mass * b, 0.0) for a, b in zip(w, q)]
                mass = sum(w)
                if mass == 0.0:
                    break  # (then all of w was at most q, and a draft stood)
            else:
                mass, w[t] = mass - w[t], 0.0
        total += math.prod(q[t] for t in triple) * (1 - none)
    return total


@pytest.mark.gpu
def test_the_first_token_has_the_targets_distribution(torch, rng):
    """200000 verifications of drafts drawn from q: the first token that comes out is distributed as p, whatever q,
    and a draft stands as often as the definition says.  Each count is within 5 of its standard deviations, which one
    in about 10^6 exceeds.  How often: over the 216 triples of drafts, one stands but for the product of 1 - a_n, a_n
    = min(1, w(t) / (W q(t))), or w(t) / W of chosen ones: 0.608 drawn, 0.266 chosen."""
    g = torch.Generator(device="cuda").manual_seed(11)
    p = torch.tensor([0.35, 0.05, 0.2, 0.0, 0.15, 0.25])
    q = torch.tensor([0.05, 0.4, 0.1, 0.15, 0.25, 0.05])
    b, n = 200000, 4
    tokens = torch.multinomial(q.cuda(), b * n, replacement=True, generator=g).view(b, n)
    parents = torch.tensor([[-1, 0, 0, 0]]).expand(b, n).contiguous()
    rows = p.cuda().expand(b, n, 6), q.cuda().expand(b, n, 6)
    for draft in (rows[1], None):
        for first in (0, 17):
            _, accepted, out = run_verify(torch, rng, rows[0], draft, tokens, parents, None, seed=9, first_counter=first)
            count = torch.bincount(out[:, 0], minlength=6).double().cpu()
            assert bool(((count - b * p).abs() <= 5 * (b * p * (1 - p)).sqrt()).all()), count
            stands = how_often(p.tolist(), q.tolist(), draft is not None)
            assert count[3] == 0 and abs(float(accepted.sum()) - b * stands) <= 5 * (b * stands * (1 - stands)) ** 0.5


@pytest.mark.gpu
def test_verification_draws_the_librarys_uniforms(torch, rng):
    g = torch.Generator().manual_seed(4)
    b, n, vocab, seed, first = 20, 7, 300, 0xDEADBEEF, (1 << 32) - 60
    target, draft = drafted(torch, g, b, n, vocab, "float32")
    tokens = torch.randint(vocab, (b, n), generator=g)
    u = torch.empty(b * n, device="cuda")
    rng.rng_fill_f32(seed, first, u)
    got = run_verify(torch, rng, target, draft, tokens, None, None, seed=seed, first_counter=first)
    check_verify(torch, rng, target, draft, tokens, None, u.view(b, n).cpu(), got)


@pytest.mark.gpu
def test_verification_in_a_graph_on_a_stream_and_of_strided_rows(torch, rng):
    g = torch.Generator().manual_seed(8)
    b, n, vocab = 150, 8, 5001
    target, draft = drafted(torch, g, b, n, vocab, "float32")
    tokens, u = torch.randint(vocab, (b, n), generator=g).int().cuda(), torch.rand(b, n, generator=g).cuda()
    want = run_verify(torch, rng, target, draft, tokens, None, u)
    # nodes outermost, in a wider array
    wide = torch.full((n, b, vocab + 3), 9.0, device="cuda")
    wide[:, :, 1:-2] = target.transpose(0, 1)
    again = run_verify(torch, rng, wide[:, :, 1:-2].transpose(0, 1), draft, tokens, None, u)
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run_verify(torch, rng, target, draft, tokens, None, u, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    graph, out = torch.cuda.CUDAGraph(), [torch.full_like(t, -9) for t in want]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rng.rng_verify_drafts(target, tokens, *out, draft=draft, uniforms=u)
    for _ in range(2):
        for t in out:
            t.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,nodes", ((2049, 1), (2100, 9), (8000, 3), (20011, 128)))
def test_verifications_whose_blocks_wait_for_room(torch, rng, vocab, nodes):
    """More requests than the SMs hold, beside another stream's products and each other: blocks of a cluster begin when
    there is room for them, and none writes to another before both run."""
    g = torch.Generator().manual_seed(vocab)
    b = 400 if nodes < 100 else 30
    target, draft = drafted(torch, g, b, nodes, vocab, "float32")
    tokens, u = torch.randint(vocab, (b, nodes), generator=g).int().cuda(), torch.rand(b, nodes, generator=g).cuda()
    parents = torch.tensor([bushy(random.Random(i), nodes) for i in range(b)], dtype=torch.int32, device="cuda")
    want = [run_verify(torch, rng, target, d, tokens, parents, u) for d in (draft, None)]
    if nodes < 100:
        check_verify(torch, rng, target[:4], draft[:4], tokens[:4].cpu(), parents[:4].cpu(), u[:4].cpu(), tuple(x[:4] for x in want[0]))
    busy = torch.randn(2048, 2048, device="cuda").bfloat16()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        with torch.cuda.stream(streams[2]):
            for _ in range(4):
                busy @ busy
        for s, d in zip(streams, (draft, None)):
            with torch.cuda.stream(s):
                got.append(run_verify(torch, rng, target, d, tokens, parents, u))
    torch.cuda.synchronize()
    for i, result in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(result, want[i % 2]))


# ---- the accepted rows' move -------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("count,b,n,lk,h,d,dtype", ((1, 1, 1, 1, 1, 8, "float16"), (2, 1, 8, 309, 2, 64, "bfloat16"), (3, 5, 128, 200, 3, 40, "float16"),
                                                    (130, 2, 6, 40, 2, 16, "bfloat16"), (4, 33, 17, 60, 8, 128, "bfloat16"), (2, 300, 5, 9, 40, 72, "float16")))
def test_rows_move_where_the_path_says(torch, rng, count, b, n, lk, h, d, dtype):
    import draft_reference as ref
    g, r = torch.Generator(device="cuda").manual_seed(n), random.Random(n)
    caches = torch.randn(count, b, lk, h, d, generator=g, device="cuda").to(getattr(torch, dtype))
    paths = [[0] + sorted(r.sample(range(1, n), r.randint(0, n - 1))) for _ in range(b)]
    paths[-1] = list(range(n))  # already in place
    kept = [len(p) - 1 for p in paths]
    given = [r.choice([0, lk - n, r.randint(0, lk - n), -3, lk]) for _ in range(b)]
    cached = [min(max(c, 0), lk - n) for c in given]
    i32 = dict(dtype=torch.int32, device="cuda")
    path = torch.tensor([p + [-1] * (n - len(p)) for p in paths], **i32)
    accepted, lengths, new = torch.tensor(kept, **i32), torch.tensor(given, **i32), torch.full((b,), -9, **i32)
    want = caches.clone()
    for i in range(b):
        for c in range(count):
            want[c, i] = ref.keep(caches[c, i], paths[i], kept[i], cached[i])
    for form in ("stacked", "list"):
        now = caches.clone()
        rng.rng_cache_keep(now if form == "stacked" else list(now), path, accepted, lengths, new)
        assert torch.equal(now, want), form
        assert new.tolist() == [c + k + 1 for c, k in zip(cached, kept)]
    # heads outermost, keys and values in one array, and lengths that end at the cache's end
    packed = torch.stack([caches[0], caches[0].flip(1)], 3)
    pair = packed.transpose(1, 2).contiguous().transpose(1, 2).unbind(3)
    rng.rng_cache_keep(pair, path, accepted, new_lengths=new)
    for t, source in zip(pair, (caches[0], caches[0].flip(1))):
        for i in range(b):
            assert torch.equal(t[i], ref.keep(source[i], paths[i], kept[i], lk - n))


@pytest.mark.gpu
def test_paths_that_say_nothing_valid_move_nothing(torch, rng):
    cache = torch.randn(6, 20, 2, 64, device="cuda").half()
    before = cache.clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 1, 2, 3], [0, 0, 1, 2], [0, 4, 1 << 30, -5], [3, -1, -(1 << 31), 9], [0, 3, 3, 3], [0, 2, 3, -1]], **i32)
    new = torch.empty(6, **i32)
    rng.rng_cache_keep([cache], path, torch.tensor([3, 3, 3, 3, -7, 100], **i32), torch.zeros(6, **i32), new)
    before[5, 1], before[5, 2] = before[5, 2].clone(), before[5, 3].clone()
    assert torch.equal(cache, before) and new.tolist() == [4, 4, 4, 4, 1, 4]


@pytest.mark.gpu
def test_rows_move_in_a_graph_and_on_another_stream(torch, rng):
    caches = torch.randn(4, 3, 50, 2, 64, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    path, accepted = torch.tensor([[0, 2, 5, -1, -1, -1]] * 3, **i32), torch.tensor([2, 1, 0], **i32)
    want, now = caches.clone(), caches.clone()
    rng.rng_cache_keep(want, path, accepted)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rng.rng_cache_keep(list(now), path, accepted, stream=side)
    side.synchronize()
    assert torch.equal(now, want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):  # (the list of addresses is read when the call is made)
        rng.rng_cache_keep(list(now), path, accepted)
    now.copy_(caches)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(now, want)


# ---- what is refused ---------------------------------------------------------------------

A = 1 << 20  # addresses that are never followed


def tree_args(rng, strides=(1024, 256, 64), **change):
    """[2, 4, 2, 64] arrays, a position's two heads side by side and a gap of 128 elements after them."""
    a = rng.TreeAttentionArgs(dtype=rng.RNG_BF16, batch=2, nodes=4, len_k=4, heads_q=2, heads_kv=2, head_dim=64,
                              scale=0.125, num_buckets=32, max_distance=128, bidirectional=1, workspace_bytes=1 << 19)
    for i, n in enumerate(("q", "k", "v", "o", "lse", "cache_lengths", "parents", "bias_table", "workspace")):
        setattr(a, n, (i + 1) * A)
        if i < 4:
            setattr(a, n + "_stride", strides)
    for n, v in change.items():
        setattr(a, n, v)
    return C.byref(a)


@pytest.mark.parametrize("bad,says", [
    ({"dtype": 0}, "dtype"), ({"batch": -1}, "negative"), ({"nodes": -1}, "negative"), ({"nodes": 129, "len_k": 500}, "129 exceeds 128"),
    ({"nodes": 5}, "exceeds len_k"), ({"len_k": 3}, "exceeds len_k"), ({"head_dim": 60}, "head_dim"), ({"head_dim": 136}, "head_dim"),
    ({"heads_kv": 0}, "multiple"), ({"heads_q": 3}, "multiple"), ({"q": None}, "q is NULL"), ({"k": None}, "k is NULL"),
    ({"v": None}, "v is NULL"), ({"o": None}, "o is NULL"), ({"k": 2 * A + 8}, "16-byte"), ({"q_stride": (1024, 250, 64)}, "stride"),
    ({"v_stride": (1024, 256, -64)}, "stride"), ({"o_stride": (1024, 64, 64)}, "overlaps itself"), ({"scale": math.inf}, "scale"),
    ({"num_buckets": 3}, "num_buckets"), ({"max_distance": 2000}, "max_distance"), ({"lse": 5 * A + 2}, "aligned"),
    ({"parents": 7 * A + 1}, "parents is not aligned"), ({"cache_lengths": 6 * A + 2}, "aligned"), ({"bias_table": 8 * A + 1}, "aligned"),
    ({"o": A}, "overlap"), ({"o": 2 * A + 512}, "overlap"), ({"lse": 4 * A}, "o and lse"), ({"lse": 7 * A}, "parents and lse"),
    ({"lse": 6 * A + 4}, "cache_lengths and lse"), ({"parents": 4 * A + 200}, "o and parents"), ({"bias_table": 5 * A}, "bias_table and lse"),
    ({"len_k": 1 << 30, "k_stride": (1 << 38, 1 << 38, 64)}, "address space"), ({"batch": 1 << 30}, "2^30")])
def test_tree_attention_refuses(rng, bad, says):
    assert rng.raw("rng_tree_attention_fwd")(tree_args(rng, **bad), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error(), rng.rng_last_error()


def test_tree_attention_of_nothing_and_of_no_struct(rng):
    for none in ({"batch": 0}, {"nodes": 0}, {"heads_q": 0}):
        assert rng.raw("rng_tree_attention_fwd")(tree_args(rng, **none, q=None, o=None), None) == rng.RNG_OK
        assert rng.raw("rng_tree_attention_fwd_workspace")(tree_args(rng, **none)) == 0
    for name in ("rng_tree_attention_fwd", "rng_verify_drafts", "rng_cache_keep"):
        assert rng.raw(name)(None, None) == rng.RNG_EINVAL and "args is NULL" in rng.rng_last_error()
    assert rng.raw("rng_tree_attention_fwd_workspace")(None) == 0


def verify_args(rng, **change):
    """[2, 3, 10] arrays of 240 bytes, [2, 3] ones of 24."""
    a = rng.VerifyDraftsArgs(dtype=rng.RNG_F32, batch=2, nodes=3, vocab=10, target_stride=(30, 10), draft_stride=(30, 10))
    for i, n in enumerate(("target", "draft", "tokens", "parents", "uniforms", "path", "accepted", "out_tokens")):
        setattr(a, n, (i + 1) * A)
    for n, v in change.items():
        setattr(a, n, v)
    return C.byref(a)


@pytest.mark.parametrize("bad,says", [
    ({"dtype": 3}, "dtype"), ({"batch": -1}, "batch"), ({"batch": (1 << 24) + 1}, "batch"), ({"nodes": 0}, "nodes"), ({"nodes": 129}, "nodes"),
    ({"vocab": 0}, "vocab"), ({"vocab": (1 << 23) + 1}, "vocab"), ({"target": None}, "target is NULL"), ({"tokens": None}, "tokens is NULL"),
    ({"path": None}, "path is NULL"), ({"accepted": None}, "accepted is NULL"), ({"out_tokens": None}, "out_tokens is NULL"),
    ({"target": A + 2}, "target is not aligned"), ({"draft": 2 * A + 1}, "draft is not aligned"), ({"uniforms": 5 * A + 1}, "uniforms is not aligned"),
    ({"target_stride": (-30, 10)}, "stride"), ({"draft_stride": (30, -1)}, "stride"), ({"target_stride": (1 << 62, 10)}, "stride"),
    ({"draft": (1 << 64) - 64}, "address space"), ({"path": A + 236}, "target and path"), ({"path": 2 * A}, "draft and path"),
    ({"accepted": 3 * A + 20}, "tokens and accepted"), ({"out_tokens": 6 * A + 4}, "path and out_tokens"), ({"out_tokens": 7 * A + 4}, "accepted and out_tokens"),
    ({"accepted": 4 * A}, "parents and accepted"), ({"path": 5 * A - 20}, "uniforms and path")])
def test_verification_refuses(rng, bad, says):
    assert rng.raw("rng_verify_drafts")(verify_args(rng, **bad), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error(), rng.rng_last_error()


def keep_args(rng, given=(8 * A, 9 * A), **change):
    """[2, 6, 2, 64] caches, trees of 4 nodes."""
    array = (C.c_void_p * max(1, len(given)))(*given)
    a = rng.CacheKeepArgs(caches=C.addressof(array), count=len(given), batch=2, nodes=4, len_k=6, heads=2, head_dim=64,
                          stride=(768, 128, 64), cache_lengths=A, path=2 * A, accepted=3 * A, new_lengths=4 * A)
    for n, v in change.items():
        setattr(a, n, v)
    a.hold = array
    return a


@pytest.mark.parametrize("bad,says", [
    ({"batch": -1}, "negative"), ({"heads": -1}, "negative"), ({"count": -1}, "negative"), ({"count": 4097}, "4096"), ({"head_dim": 4}, "head_dim"),
    ({"nodes": 0}, "nodes"), ({"nodes": 7}, "nodes"), ({"nodes": 129, "len_k": 200}, "nodes"), ({"path": None}, "path is NULL"),
    ({"accepted": None}, "accepted is NULL"), ({"path": 2 * A + 2}, "path is not aligned"), ({"new_lengths": 4 * A + 1}, "new_lengths is not aligned"),
    ({"caches": None}, "caches is NULL"), ({"stride": (768, 100, 64)}, "stride"), ({"stride": (768, 64, 64)}, "overlaps itself"),
    ({"new_lengths": A}, "cache_lengths and new_lengths"), ({"new_lengths": A + 4}, "cache_lengths and new_lengths"),
    ({"new_lengths": 3 * A}, "accepted and new_lengths"), ({"new_lengths": 2 * A + 28}, "path and new_lengths"),
    ({"path": 8 * A + 100}, "path"), ({"accepted": 9 * A}, "accepted"), ({"new_lengths": 8 * A + 3068}, "new_lengths")])
def test_the_move_refuses(rng, bad, says):
    a = keep_args(rng, **bad)
    assert rng.raw("rng_cache_keep")(C.byref(a), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error(), rng.rng_last_error()


@pytest.mark.parametrize("caches,says", [((8 * A, None), "NULL"), ((8 * A, 8 * A), "overlap"), ((8 * A, 9 * A, 8 * A + 3056), "overlap"),
                                         ((9 * A, 8 * A + 8), "16-byte"), ((8 * A, 10 * A, 9 * A, 10 * A + 128), "overlap")])
def test_the_move_refuses_caches(rng, caches, says):
    a = keep_args(rng, caches)
    assert rng.raw("rng_cache_keep")(C.byref(a), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error(), rng.rng_last_error()


def without_a_device(torch):
    """Calls that nothing refuses end at the launch: only where there is no GPU, whose memory they would follow."""
    if torch.cuda.is_available():
        pytest.skip("addresses that no GPU may follow")


# of `count` caches in one array, [batch, len, heads] strides and what lies between two of them, in elements
SLICES = {"entries": lambda n, ln, h, d: ((n * ln * h * d, h * d, d), ln * h * d), "rows": lambda n, ln, h, d: ((ln * n * h * d, n * h * d, d), h * d),
          "heads": lambda n, ln, h, d: ((ln * h * n * d, h * n * d, n * d), d), "apart": lambda n, ln, h, d: ((ln * h * d, h * d, d), 5 * ln * h * d)}


@pytest.mark.parametrize("layout", SLICES)
@pytest.mark.parametrize("arrays", (1, 3))
def test_many_caches_in_one_array_are_told_apart_quickly(torch, rng, layout, arrays):
    """4095 slices of one array, or of three, in no order: their ranges all touch.  (Every pair compared: 0.1 s.)"""
    import time
    without_a_device(torch)
    n, (stride, step) = 4095 // arrays, SLICES[layout](4095 // arrays, 20, 2, 64)
    given = [(1 << 33) + k * ((1 << 40) + 96) + 2 * step * i for k in range(arrays) for i in range(n)]
    random.Random(1).shuffle(given)
    a, times = keep_args(rng, given, batch=3, len_k=20, stride=stride), []
    for _ in range(5):
        start = time.perf_counter()
        assert rng.raw("rng_cache_keep")(C.byref(a), None) not in (rng.RNG_OK, rng.RNG_EINVAL), rng.rng_last_error()
        times.append(time.perf_counter() - start)
    assert min(times) < 0.02
    a = keep_args(rng, given + [given[7] + 2 * (step // 2 // 8 * 8)], batch=3, len_k=20, stride=stride)
    assert rng.raw("rng_cache_keep")(C.byref(a), None) == rng.RNG_EINVAL  # one more, in the middle of another
    assert "two caches overlap" in rng.rng_last_error()


def test_caches_that_share_an_element_are_refused(torch, rng):
    """Any strides and addresses, against the sets of their elements; slices of one array are not refused."""
    without_a_device(torch)
    r, shared, apart = random.Random(3), 0, 0
    for _ in range(3000):
        b, ln, h = r.choice((1, 2, 3)), r.randint(4, 6), r.choice((1, 2, 3))
        unit = r.choice((8, 8, 16))
        stride = tuple(8 * r.choice((1, 2, 3, 4, 6, 8, 12, 24, 48, 96, 7, 50)) for _ in range(3))
        given = [8 * A + 16 * r.randrange(0, 400) for _ in range(r.choice((2, 2, 3, 5)))]
        elements = [{(p - 8 * A) // 2 + i * stride[0] + j * stride[1] + k * stride[2] + e for i in range(b) for j in range(ln) for k in range(h)
                     for e in range(unit)} for p in given]
        status = rng.raw("rng_cache_keep")(C.byref(keep_args(rng, given, batch=b, len_k=ln, heads=h, head_dim=unit, stride=stride)), None)
        if any(x & y for x, y in itertools.combinations(elements, 2)):
            assert status == rng.RNG_EINVAL
            shared += 1
        elif status != rng.RNG_EINVAL:
            apart += 1
    assert min(shared, apart) > 300  # (the draws reach both)
    for layout, (n, b, ln, h) in itertools.product(SLICES, ((2, 1, 4, 1), (7, 3, 4, 2), (40, 1, 9, 3), (5, 4, 5, 1))):
        stride, step = SLICES[layout](n, ln, h, 64)
        given = [8 * A + 2 * step * i for i in range(n)]
        for change, refused in ((0, False), (16, True)):
            given[0] += change
            status = rng.raw("rng_cache_keep")(C.byref(keep_args(rng, given, batch=b, len_k=ln, heads=h, stride=stride)), None)
            assert (status == rng.RNG_EINVAL) == (refused and layout != "apart"), (layout, n, rng.rng_last_error())


@pytest.mark.gpu
@pytest.mark.parametrize("dims", ((1, 0, 2, 3, 4), (1, 2, 0, 3, 4), (1, 2, 3, 0, 4), (0, 1, 2, 3, 4)))
def test_rows_move_in_slices_of_one_array(torch, rng, dims):
    """Caches between each other's entries, rows or heads, as a list and as one tensor."""
    import draft_reference as ref
    count, b, n, lk, h, d = 70, 3, 6, 40, 2, 64
    plain = torch.randn(count, b, lk, h, d, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    path, accepted, lengths = torch.tensor([[0, 2, 5, -1, -1, -1], [0, 1, 3, 4, 5, -1], [0] + [-1] * 5], **i32), torch.tensor([2, 4, 0], **i32), torch.tensor([30, 0, 11], **i32)
    want = plain.clone()
    for c in range(count):
        for i, kept in enumerate((2, 4, 0)):
            want[c, i] = ref.keep(plain[c, i], path[i].tolist(), kept, int(lengths[i]))
    back = [dims.index(i) for i in range(5)]
    for form in (list, lambda t: t):
        now = plain.clone().permute(dims).contiguous().permute(back)
        rng.rng_cache_keep(form(now), path, accepted, lengths)
        assert torch.equal(now, want)


@pytest.mark.gpu
def test_the_binding_checks_its_tensors(torch, rng):
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    q, k = torch.zeros(2, 4, 2, 64, **bf), torch.zeros(2, 30, 2, 64, **bf)
    o = torch.empty_like(q)
    for error, call in ((TypeError, dict(q=q.float())), (ValueError, dict(v=k[:, :-1])), (ValueError, dict(o=o[:, :3])), (TypeError, dict(parents=torch.zeros(2, 4, device="cuda"))),
                        (ValueError, dict(parents=torch.zeros(2, 3, **i32))), (ValueError, dict(cache_lengths=torch.zeros(3, **i32))),
                        (ValueError, dict(lse=torch.zeros(2, 4, 2, device="cuda"))), (ValueError, dict(bias_table=torch.zeros(8, 3, **bf))),
                        (ValueError, dict(bias_table=torch.zeros(0, 2, **bf))), (TypeError, dict(q=q.cpu()))):
        with pytest.raises(error):
            rng.rng_tree_attention_fwd(**{**dict(q=q, k=k, v=k, o=o), **call})
    p = torch.zeros(2, 4, 10, device="cuda")
    small = dict(tokens=torch.zeros(2, 4, **i32), path=torch.zeros(2, 4, **i32), accepted=torch.zeros(2, **i32), out_tokens=torch.zeros(2, 4, **i32))
    for error, call in ((TypeError, dict(target=p.long())), (ValueError, dict(target=p[0])), (TypeError, dict(tokens=small["tokens"].long())),
                        (ValueError, dict(draft=p[:, :, :9])), (TypeError, dict(draft=p.half())), (ValueError, dict(target=p.transpose(1, 2).contiguous().transpose(1, 2))),
                        (TypeError, dict(uniforms=torch.zeros(2, 4, device="cuda").double())), (ValueError, dict(accepted=torch.zeros(3, **i32)))):
        with pytest.raises(error):
            rng.rng_verify_drafts(**{**dict(target=p), **small, **call})
    path, accepted = torch.zeros(2, 4, **i32), torch.zeros(2, **i32)
    for error, call in ((ValueError, dict(caches=[])), (ValueError, dict(caches=k)), (ValueError, dict(caches=[k, k[:, :20]])), (ValueError, dict(caches=[k.float()])),
                        (ValueError, dict(caches=[k[0]])), (ValueError, dict(caches=[k], path=path[:1])), (TypeError, dict(caches=[k], path=path.long())),
                        (rng.RngError, dict(caches=[k, k])), (ValueError, dict(caches=[k, k.half()]))):
        with pytest.raises(error):
            rng.rng_cache_keep(**{**dict(path=path, accepted=accepted), **call})

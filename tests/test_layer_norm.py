"""rng_dropout_layer_norm_{fwd,bwd} against the formulas in 64 bits.

Tolerances.  u = 2^-24 is binary32's unit roundoff, ut the output type's
(2^-24, 2^-11, 2^-8).  A row's sum over N columns is a thread's own chain of at
most 32 terms (N / 1024 above 32768) and a tree of ten levels, so it is within
c u sum|terms| with c = 48 + N / 1024.  With H the row's largest |x + bias| /
(1 - p) + |residual|, each h is within 5 u H and the mean within (c + 5) u H;
that moves n = (h - mean) rstd by (c + 10) u H rstd, and rstd, through the
variance (mean square of the deviations), by (2 (c + 10) H rstd + c + 4) u of
itself.  The backward pass starts from given h, mean and rstd, so its n is within
3 u M, M = (|h| + |mean|) rstd, and its two means within (c + 4) u of the means
of |g| and of |g| M.  A weight's gradient is a chain of at most `rows` terms, a
few levels of trees, and the terms' own errors.
"""
import ctypes as C

import numpy as np
import pytest

U = 2.0 ** -24
UT = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -134}
EPS = 1e-5
TYPES = [("float32", "float32"), ("float16", "float16"), ("float16", "float32"), ("bfloat16", "bfloat16"),
         ("bfloat16", "float32")]
# one column; odd; a vector; a warp's and a block's edges; the fused backward's edge; past every register form
COLS = (1, 2, 3, 8, 31, 64, 255, 256, 257, 264, 769, 1000, 1024, 4096, 4104, 4097, 8192, 8200, 8193, 16384, 16387,
        32776)


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def rng():
    import dropout_lowbias32_hash32_gb300 as rng
    return rng


def unit(t):
    return UT[str(t.dtype).replace("torch.", "")]


def assert_within(name, got, want, tol):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(((got - want).abs() / tol)[bad].max()))


def rounded(got, want):
    """What rounding the output once may cost."""
    name = str(got.dtype).replace("torch.", "")
    return UT[name] * want.abs() + TINY[name]


def make(torch, rows, cols, dtype, wtype, seed, weights=True, bias=True, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, wt = getattr(torch, dtype), getattr(torch, wtype)

    def normal(*shape, to=dt, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(to)

    return {"x": normal(rows, cols), "residual": normal(rows, cols, scale=2.0, shift=0.5) if residual else None,
            "bias": normal(cols, to=wt) if bias else None,
            "gamma": normal(cols, to=wt, scale=0.3, shift=1.0) if weights else None,
            "beta": normal(cols, to=wt) if weights else None, "dy": normal(rows, cols), "dh": normal(rows, cols)}


def check_fwd(torch, orc, t, p, seed, first, y, h, mean, rstd):
    import layer_reference as ref
    rows, cols = t["x"].shape
    keep = ref.keep_mask(orc, p, seed, first, (rows, cols), "cuda")
    wy, wh, wm, wr = ref.norm_fwd(t["x"], t["bias"], t["residual"], t["gamma"], t["beta"], keep, EPS)
    c = 48 + cols / 1024
    top = t["x"].double().abs()
    if t["bias"] is not None:
        top = top + t["bias"].double().abs()
    top = top / (1 - p)
    if t["residual"] is not None:
        top = top + t["residual"].double().abs()
    top = top.amax(1)
    n = (wh - wm[:, None]) * wr[:, None]
    if h is not None:
        assert_within("h", h, wh, rounded(h, wh) + 5 * U * top[:, None])
    rel_rstd = (2 * (c + 10) * top * wr + c + 4) * U
    if mean is not None:
        assert_within("mean", mean, wm, (c + 5) * U * top)
        assert_within("rstd", rstd, wr, rel_rstd * wr)
    gamma = 1.0 if t["gamma"] is None else t["gamma"].double().abs()
    beta = 0.0 if t["beta"] is None else t["beta"].double().abs()
    tol = ((c + 10) * U * (top * wr)[:, None] + n.abs() * rel_rstd[:, None]) * gamma + 4 * U * (n.abs() * gamma + beta)
    assert_within("y", y, wy, tol + rounded(y, wy))


def run_fwd(torch, rng, t, p, seed, first, stats=True, h=True):
    rows, cols = t["x"].shape
    y = torch.empty_like(t["x"])
    h = torch.empty_like(t["x"]) if h else None
    mean, rstd = (torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")) if stats else (None, None)
    rng.rng_dropout_layer_norm_fwd(t["x"], t["gamma"], t["beta"], y, mean, rstd, bias=t["bias"],
                                   residual=t["residual"], h=h, p=p, seed=seed, first_counter=first, eps=EPS)
    return y, h, mean, rstd


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_forward(torch, rng, orc, cols, dtype, wtype):
    for rows, p in ((1, 0.0), (11, 0.3), (300 if cols < 1000 else 37, 0.1)):
        t = make(torch, rows, cols, dtype, wtype, 7 * cols + rows)
        first = (1 << 32) - 5
        check_fwd(torch, orc, t, p, 42, first, *run_fwd(torch, rng, t, p, 42, first))


@pytest.mark.gpu
@pytest.mark.parametrize("weights,bias,residual,stats,h", [
    (False, False, False, False, False), (True, False, False, True, False), (False, True, False, False, True),
    (True, False, True, False, True), (False, True, True, True, True)])
@pytest.mark.parametrize("cols", (40, 769, 2048, 33000))
def test_forward_without_its_options(torch, rng, orc, cols, weights, bias, residual, stats, h):
    t = make(torch, 9, cols, "bfloat16", "float32", cols, weights, bias, residual)
    check_fwd(torch, orc, t, 0.5, 3, 0, *run_fwd(torch, rng, t, 0.5, 3, 0, stats, h))


def check_bwd(torch, orc, t, p, seed, first, h, mean, rstd, out):
    import layer_reference as ref
    rows, cols = h.shape
    keep = ref.keep_mask(orc, p, seed, first, (rows, cols), "cuda")
    wdx, wdz, wg, wb, wbias = ref.norm_bwd(t["dy"], h, t["dh"], t["gamma"], mean, rstd, keep)
    c = 48 + cols / 1024
    r = rstd.double()[:, None]
    m = (h.double().abs() + mean.double().abs()[:, None]) * r
    dy = t["dy"].double().abs()
    g = dy if t["gamma"] is None else dy * t["gamma"].double().abs()
    dh = 0.0 if t["dh"] is None else t["dh"].double().abs()
    mean_g, mean_gm = g.mean(1, keepdim=True), (g * m).mean(1, keepdim=True)
    tol = r * U * (4 * g + (c + 4) * mean_g + m * (c + 10) * mean_gm) + 4 * U * (wdz.abs() + dh)
    assert_within("dx", out["dx"], wdx, tol * keep + rounded(out["dx"], wdx))
    if out.get("dresidual") is not None:
        assert_within("dresidual", out["dresidual"], wdz, tol + rounded(out["dresidual"], wdz))
    chain = (min(rows, 4096) + 20) * U
    for name, want, terms, own in (("dgamma", wg, dy * m, 4 * U * dy * m), ("dbeta", wb, dy, 0 * dy),
                                   ("dbias", wbias, wdx.abs() + tol * keep, tol * keep)):
        if out.get(name) is not None:
            assert_within(name, out[name], want, chain * terms.sum(0) + own.sum(0) + rounded(out[name], want))


def run_bwd(torch, rng, t, p, seed, first, dresidual=True, grads=True, **more):
    import layer_reference as ref
    h, rows, cols = t["residual"] if t["residual"] is not None else t["x"], *t["dy"].shape
    mean = h.double().mean(1)
    rstd = (((h.double() - mean[:, None]) ** 2).mean(1) + EPS) ** -0.5
    mean, rstd = mean.float(), rstd.float()
    wt = t["gamma"].dtype if t["gamma"] is not None else t["dy"].dtype
    out = {"dx": torch.empty_like(t["dy"]), "dresidual": torch.empty_like(t["dy"]) if dresidual else None}
    for name in ("dgamma", "dbeta", "dbias"):
        out[name] = torch.full((cols,), float("nan"), dtype=wt, device="cuda") if grads else None
    rng.rng_dropout_layer_norm_bwd(t["dy"], h, t["gamma"], mean, rstd, out["dx"], out["dgamma"], out["dbeta"],
                                   dh=t["dh"], dresidual=out["dresidual"], dbias=out["dbias"], p=p, seed=seed,
                                   first_counter=first, **more)
    return h, mean, rstd, out


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_backward(torch, rng, orc, cols, dtype, wtype):
    for rows, p in ((1, 0.0), (11, 0.3), (1300 if cols < 1000 else 341, 0.1)):
        t = make(torch, rows, cols, dtype, wtype, 5 * cols + rows)
        first = (1 << 32) - 9
        check_bwd(torch, orc, t, p, 77, first, *run_bwd(torch, rng, t, p, 77, first))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", (40, 769, 2048, 8208))
def test_backward_without_its_options(torch, rng, orc, cols):
    for weights, dh, dresidual, grads in ((False, False, False, False), (True, False, True, True),
                                          (False, True, False, True)):
        t = make(torch, 19, cols, "float16", "float32", cols, weights)
        t["dh"] = t["dh"] if dh else None
        check_bwd(torch, orc, t, 0.5, 3, 0, *run_bwd(torch, rng, t, 0.5, 3, 0, dresidual, grads))


@pytest.mark.gpu
def test_backward_of_many_rows_and_twice_the_same_bits(torch, rng, orc):
    t = make(torch, 20011, 136, "bfloat16", "float32", 3)
    h, mean, rstd, out = run_bwd(torch, rng, t, 0.2, 9, 1)
    check_bwd(torch, orc, t, 0.2, 9, 1, h, mean, rstd, out)
    again = run_bwd(torch, rng, t, 0.2, 9, 1)[3]
    assert all(torch.equal(out[n], again[n]) for n in out)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,dtype,wtype", ((9001, 256, "float32", "float32"), (5003, 520, "bfloat16", "float32"),
                                                   (3001, 1000, "float16", "float16"), (1201, 8192, "float32", "float32"),
                                                   (801, 8184, "bfloat16", "bfloat16"), (7001, 24, "bfloat16", "bfloat16"),
                                                   (2001, 777, "float16", "float32")))
def test_many_rows_a_block(torch, rng, orc, rows, cols, dtype, wtype):
    t = make(torch, rows, cols, dtype, wtype, seed=cols)
    check_fwd(torch, orc, t, 0.1, 3, 1, *run_fwd(torch, rng, t, 0.1, 3, 1))
    check_bwd(torch, orc, t, 0.1, 3, 1, *run_bwd(torch, rng, t, 0.1, 3, 1))
    t["dh"] = None
    check_bwd(torch, orc, t, 0.0, 3, 1, *run_bwd(torch, rng, t, 0.0, 3, 1, dresidual=False))


@pytest.mark.gpu
def test_no_rows_give_zero_gradients(torch, rng):
    z = torch.empty(0, 48, device="cuda")
    stat = torch.empty(0, device="cuda")
    gamma = torch.ones(48, device="cuda")
    grads = [torch.full((48,), float("nan"), device="cuda") for _ in range(3)]
    rng.rng_dropout_layer_norm_bwd(z, z.clone(), gamma, stat, stat.clone(), z.clone(), grads[0], grads[1],
                                   dbias=grads[2], p=0.1)
    assert all(bool((g == 0).all()) for g in grads)
    rng.rng_dropout_layer_norm_fwd(z, gamma, gamma, z.clone(), stat, stat.clone())
    empty = torch.empty(5, 0, device="cuda")
    rng.rng_dropout_layer_norm_fwd(empty, None, None, torch.empty(5, 0, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("offset,pad", ((0, 8), (1, 3), (8, 16), (4, 5)))
@pytest.mark.parametrize("dtype", ("float32", "bfloat16"))
def test_strided_rows_and_nothing_written_beside_them(torch, rng, orc, dtype, offset, pad):
    rows, cols = 21, 520
    t = make(torch, rows, cols, dtype, "float32", 5)
    wide = {}
    for name in ("x", "residual", "y", "h", "dy", "dh", "dx", "dresidual"):
        buf = torch.full((rows, offset + cols + pad), 7.0, dtype=t["x"].dtype, device="cuda")
        view = buf[:, offset:offset + cols]
        if name in t:
            view.copy_(t[name])
        wide[name] = (buf, view)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    rng.rng_dropout_layer_norm_fwd(wide["x"][1], t["gamma"], t["beta"], wide["y"][1], mean, rstd, bias=t["bias"],
                                   residual=wide["residual"][1], h=wide["h"][1], p=0.25, seed=8, first_counter=2,
                                   eps=EPS)
    check_fwd(torch, orc, t, 0.25, 8, 2, wide["y"][1], wide["h"][1], mean, rstd)
    grads = {n: torch.empty(cols, device="cuda") for n in ("dgamma", "dbeta", "dbias")}
    rng.rng_dropout_layer_norm_bwd(wide["dy"][1], wide["h"][1], t["gamma"], mean, rstd, wide["dx"][1],
                                   grads["dgamma"], grads["dbeta"], dh=wide["dh"][1],
                                   dresidual=wide["dresidual"][1], dbias=grads["dbias"], p=0.25, seed=8,
                                   first_counter=2)
    check_bwd(torch, orc, t, 0.25, 8, 2, wide["h"][1], mean, rstd,
              {**grads, "dx": wide["dx"][1], "dresidual": wide["dresidual"][1]})
    for name, (buf, _) in wide.items():
        assert bool((buf[:, :offset] == 7).all()) and bool((buf[:, offset + cols:] == 7).all()), name


@pytest.mark.gpu
@pytest.mark.parametrize("cols", (24, 769, 4096, 9000, 33000))
def test_in_place(torch, rng, cols):
    t = make(torch, 13, cols, "bfloat16", "bfloat16", 9)
    y, h, mean, rstd = run_fwd(torch, rng, t, 0.1, 4, 0)
    x, residual = t["x"].clone(), t["residual"].clone()
    rng.rng_dropout_layer_norm_fwd(x, t["gamma"], t["beta"], x, bias=t["bias"], residual=residual, h=residual, p=0.1,
                                   seed=4, eps=EPS)
    assert torch.equal(x, y) and torch.equal(residual, h)
    out = [torch.empty_like(y), torch.empty_like(y)]
    grads = [torch.empty_like(t["gamma"]) for _ in range(6)]
    rng.rng_dropout_layer_norm_bwd(t["dy"], h, t["gamma"], mean, rstd, out[0], grads[0], grads[1], dh=t["dh"],
                                   dresidual=out[1], dbias=grads[2], p=0.1, seed=4)
    dy, dh = t["dy"].clone(), t["dh"].clone()
    rng.rng_dropout_layer_norm_bwd(dy, h, t["gamma"], mean, rstd, dy, grads[3], grads[4], dh=dh, dresidual=dh,
                                   dbias=grads[5], p=0.1, seed=4)
    assert torch.equal(dy, out[0]) and torch.equal(dh, out[1])
    assert all(torch.equal(grads[i], grads[i + 3]) for i in range(3))


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_row(torch, rng):
    t = make(torch, 6, 1000, "float32", "float32", 2)
    clean = run_fwd(torch, rng, t, 0.1, 4, 0)
    t["x"][2, 5], t["residual"][4, 7] = float("nan"), float("inf")
    dirty = run_fwd(torch, rng, t, 0.0, 4, 0)
    assert bool(dirty[0][2].isnan().all()) and bool(dirty[0][4].isnan().all())
    dirty = run_fwd(torch, rng, t, 0.1, 4, 0)
    for row in (0, 1, 3, 5):
        assert all(torch.equal(a[row], b[row]) for a, b in zip(clean, dirty))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", (96, 1000))
def test_gradient_against_differences(torch, rng, orc, cols):
    """The kernel's gradient along a direction against central differences of
    the 64-bit forward: loss = <dy, y> + <dh, h>, f32 inputs.  The difference
    quotient at step 1e-5 is good to about 1e-8 of the loss's scale; the
    kernel's gradient to its f32 sums, 1e-5 of the sum of its terms."""
    import layer_reference as ref
    t = make(torch, 7, cols, "float32", "float32", 12)
    p, seed, first = 0.3, 6, 11
    y, h, mean, rstd = run_fwd(torch, rng, t, p, seed, first)
    out = {n: torch.empty_like(t["x"]) for n in ("dx", "dresidual")}
    out |= {n: torch.empty_like(t["gamma"]) for n in ("dgamma", "dbeta", "dbias")}
    rng.rng_dropout_layer_norm_bwd(t["dy"], h, t["gamma"], mean, rstd, out["dx"], out["dgamma"], out["dbeta"],
                                   dh=t["dh"], dresidual=out["dresidual"], dbias=out["dbias"], p=p, seed=seed,
                                   first_counter=first)
    keep = ref.keep_mask(orc, p, seed, first, t["x"].shape, "cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    names = {"x": "dx", "residual": "dresidual", "gamma": "dgamma", "beta": "dbeta", "bias": "dbias"}
    for name, grad in names.items():
        d = torch.randn(t[name].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(step):
            v = {k: t[k].double() for k in names}
            v[name] = v[name] + step * d
            y, h, _, _ = ref.norm_fwd(v["x"], v["bias"], v["residual"], v["gamma"], v["beta"], keep, EPS)
            return (y * t["dy"]).sum() + (h * t["dh"]).sum()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = out[grad].double() * d
        assert abs(terms.sum() - want) <= 1e-5 * terms.abs().sum() + 1e-5, name


@pytest.mark.gpu
def test_more_than_2_to_32_elements(torch, rng, orc):
    """Offsets past 32 bits and counters that wrap: the last rows of 2^18 + 3."""
    rows, cols = (1 << 18) + 3, 16392
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.empty_like(x)
    rng.rng_dropout_layer_norm_fwd(x, None, None, y, p=0.25, seed=8, first_counter=7, eps=EPS)
    t = {"x": x[-3:].clone(), "bias": None, "residual": None, "gamma": None, "beta": None}
    check_fwd(torch, orc, t, 0.25, 8, 7 + (rows - 3) * cols, y[-3:], None, None, None)
    del x, y
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_another_stream_and_a_captured_graph(torch, rng):
    t = make(torch, 40, 1024, "bfloat16", "bfloat16", 21)
    want_y, h, mean, rstd = run_fwd(torch, rng, t, 0.1, 4, 0)
    _, _, _, want = run_bwd(torch, rng, t, 0.1, 4, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(want_y)
    rng.rng_dropout_layer_norm_fwd(t["x"], t["gamma"], t["beta"], y, bias=t["bias"], residual=t["residual"], p=0.1,
                                   seed=4, eps=EPS, stream=side)
    _, _, _, out = run_bwd(torch, rng, t, 0.1, 4, 0, stream=side)
    side.synchronize()
    assert torch.equal(y, want_y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, *_ = run_fwd(torch, rng, t, 0.1, 4, 0)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want_y)


# ---- refusals (nothing below reaches the GPU) -----------------------------------

A = 0x10000000  # an address that is never dereferenced


def fwd(rng, x=A, x_stride=64, bias=None, res=None, res_stride=0, gamma=None, beta=None, y=2 * A, y_stride=64, h=None,
        h_stride=0, mean=None, rstd=None, rows=4, cols=64, dtype=2, wtype=2, p=0.1, eps=1e-5):
    return rng.raw("rng_dropout_layer_norm_fwd")(x, x_stride, bias, res, res_stride, gamma, beta, y, y_stride, h,
                                                 h_stride, mean, rstd, rows, cols, dtype, wtype, p, 1, 0, eps, None)


def bwd(rng, dy=A, h=2 * A, dh=None, gamma=None, mean=3 * A, rstd=4 * A, dx=5 * A, dres=None, dgamma=6 * A, rows=4,
        cols=64, dtype=2, wtype=2, p=0.1, ws=7 * A, ws_bytes=1 << 20, stride=64):
    return rng.raw("rng_dropout_layer_norm_bwd")(dy, stride, h, stride, dh, stride, gamma, mean, rstd, dx, stride,
                                                 dres, stride, dgamma, None, None, rows, cols, dtype, wtype, p, 1, 0,
                                                 ws, ws_bytes, None)


@pytest.mark.parametrize("bad,says", [
    ({"x": None}, "NULL"), ({"y": None}, "NULL"), ({"x": A + 1}, "aligned"), ({"gamma": A + 1}, "aligned"),
    ({"mean": A + 2}, "aligned"), ({"x_stride": 63}, "stride"), ({"dtype": 3}, "dtype"),
    ({"dtype": 0, "wtype": 2}, "param_dtype"), ({"dtype": 2, "wtype": 1}, "param_dtype"), ({"p": 1.0}, "outside"),
    ({"p": float("nan")}, "outside"), ({"eps": -1.0}, "eps"), ({"eps": float("inf")}, "eps"),
    ({"y": A + 128}, "overlap"), ({"y": A, "y_stride": 128}, "overlap"), ({"h": 2 * A, "h_stride": 64}, "overlap"),
    ({"rows": 1 << 31}, "rows"), ({"cols": 1 << 31, "x_stride": 1 << 31, "y_stride": 1 << 31}, "columns"),
    ({"x_stride": 1 << 62}, "address space")])
def test_forward_refuses(rng, bad, says):
    assert fwd(rng, **bad) == rng.RNG_EINVAL
    assert says in rng.rng_last_error()


@pytest.mark.parametrize("bad,says", [
    ({"dy": None}, "NULL"), ({"mean": None}, "NULL"), ({"dx": None}, "NULL"), ({"dgamma": A + 1}, "aligned"),
    ({"p": -0.5}, "outside"), ({"dx": 2 * A}, "overlap"), ({"dx": A, "dres": A}, "overlap"), ({"dtype": 7}, "dtype"),
    ({"ws": None}, "workspace"), ({"ws_bytes": 16}, "workspace"), ({"ws": 7 * A + 4}, "workspace"),
    ({"stride": 60}, "stride")])
def test_backward_refuses(rng, bad, says):
    assert bwd(rng, **bad) == rng.RNG_EINVAL
    assert says in rng.rng_last_error()


def test_nothing_to_do_is_fine(rng):
    assert fwd(rng, x=None, y=None, rows=0) == rng.RNG_OK
    assert fwd(rng, x=None, y=None, cols=0) == rng.RNG_OK
    assert bwd(rng, cols=0) == rng.RNG_OK
    assert rng.rng_dropout_layer_norm_bwd_workspace(0, 64) == 0


@pytest.mark.gpu
def test_python_refusals(torch, rng):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    y, g = torch.empty_like(x), torch.ones(64, device="cuda", dtype=torch.bfloat16)
    call = rng.rng_dropout_layer_norm_fwd
    with pytest.raises(TypeError):
        call(x.cpu(), g, g, y)
    with pytest.raises(TypeError):
        call(x.double(), g, g, y)
    with pytest.raises(TypeError):
        call(x, g, g.float(), y)
    with pytest.raises(ValueError):
        call(x, g[:60], g, y)
    with pytest.raises(ValueError):
        call(x, g, g, y[:, :32])
    with pytest.raises(ValueError):
        call(x, g, g, torch.empty(64, 4, device="cuda", dtype=torch.bfloat16).t())
    with pytest.raises(ValueError):
        call(x, g.cpu(), g, y)
    with pytest.raises(rng.RngError):
        call(x, g, g, y, p=1.0)
    three = torch.zeros(2, 3, 8, device="cuda")
    with pytest.raises(ValueError):  # the leading dimensions do not lie one stride apart
        call(three, None, None, torch.zeros(2, 4, 8, device="cuda")[:, :3])

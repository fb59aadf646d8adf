"""How the layer operators are called: the stream and the workspace of a call,
sizes at the ends of what it accepts."""
import contextlib
import ctypes as C
import subprocess
import sys

import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def rng():
    import dropout_lowbias32_hash32_gb300 as rng
    return rng


# ---- the workspace's stream ----------------------------------------------------------


class FakeTorch:
    """As much of torch as takes a workspace; `allocated` lists the streams that
    were current when it was."""

    uint8 = "uint8"

    def __init__(self):
        self.current, self.allocated = "current", []
        fake = self

        class Stream:
            def __init__(self, handle):
                self.cuda_stream = handle

        class Cuda:
            pass

        @contextlib.contextmanager
        def stream(s):
            before, fake.current = fake.current, s.cuda_stream
            yield
            fake.current = before

        self.cuda = Cuda()
        self.cuda.Stream, self.cuda.stream = Stream, stream
        self.cuda.ExternalStream = lambda handle, device=None: Stream(handle)
        self.cuda.default_stream = lambda device=None: Stream(0)

    def empty(self, n, dtype, device):
        self.allocated.append(self.current)

        class Tensor:
            record_stream = staticmethod(lambda s: None)
            data_ptr, numel, element_size = (staticmethod(lambda: 1 << 20), staticmethod(lambda: n),
                                             staticmethod(lambda: 1))
        return Tensor()


def test_a_workspace_is_taken_from_the_stream_that_the_kernels_run_on(rng, monkeypatch):
    """The allocator hands a block of the current stream's pool out again while
    the current stream's earlier work still uses it: right for that stream
    alone."""
    fake = FakeTorch()
    monkeypatch.setattr(rng, "_torch", fake)
    like = type("Like", (), {"device": "cuda:0"})()

    class Handle:  # a stream of another library
        cuda_stream = 77

    for stream, want in ((None, "current"), (fake.cuda.Stream(55), 55), (66, 66), (Handle(), 77), (0, 0),
                         (fake.cuda.Stream(0), 0)):
        pointer, size, hold = rng._scratch(None, 4096, like, stream)
        assert (fake.allocated.pop(), fake.current) == (want, "current") and pointer and size == 4096 and hold
    assert rng._scratch(None, 0, like, 55) == (None, 0, None) and not fake.allocated


def busy(torch):
    """Work that the current stream is at for some milliseconds."""
    a = torch.randn(8192, 8192, device="cuda")
    for _ in range(6):
        a = a @ a * 1e-3
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("operator", ("attention_bwd", "attention_fwd", "norm_bwd"))
def test_a_call_on_another_stream_keeps_off_the_current_ones_workspace(torch, rng, operator):
    """Two calls of one size, the second on another stream while the first, and
    the workspace that it has given back, are still to be used: each gives what
    it gives alone."""
    g = torch.Generator(device="cuda").manual_seed(4)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    def call():
        if operator == "norm_bwd":
            dy, h, gamma, mean, rstd = (normal(4096, 1024), normal(4096, 1024), normal(1024),
                                        normal(4096, dtype=torch.float32), normal(4096, dtype=torch.float32))
            out = [torch.empty_like(t) for t in (dy, gamma, gamma)]
            return out, lambda **o: rng.rng_dropout_layer_norm_bwd(dy, h, gamma, mean, rstd, out[0], out[1], out[2],
                                                                   p=0.1, seed=3, **o)
        lq, lk = (1, 8192) if operator == "attention_fwd" else (512, 512)
        q, do = normal(2, lq, 8, 64), normal(2, lq, 8, 64)
        k, v = normal(2, lk, 8, 64), normal(2, lk, 8, 64)
        o, lse = torch.empty_like(q), torch.empty(2, 8, lq, device="cuda")
        if operator == "attention_fwd":
            return [o, lse], lambda **s: rng.rng_attention_fwd(q, k, v, o, lse=lse, **s)
        rng.rng_attention_fwd(q, k, v, o, lse=lse, p=0.1, seed=3)
        out = [torch.empty_like(t) for t in (q, k, v)]
        return out, lambda **s: rng.rng_attention_bwd(do, q, k, v, o, lse, *out, p=0.1, seed=3, **s)

    calls = [call() for _ in range(2)]
    want = []
    for out, run in calls:
        run()
        want.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        torch.cuda.synchronize()
        busy(torch)
        calls[0][1]()
        calls[1][1](stream=stream)
        torch.cuda.synchronize()
        for (out, _), w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
            for t in out:
                t.zero_()


# ---- the caller's workspace ------------------------------------------------------------


def guarded(torch, size):
    """A workspace of that many bytes, all of them NaN in every type, and what lies around it."""
    store = torch.full((size + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    return store[256:256 + size], lambda: bool((store[:256] == 0xFF).all() and (store[256 + size:] == 0xFF).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,h,hk,d,dtype,buckets", ((1, 9000, 8, 2, 128, "bfloat16", 0), (3, 4000, 4, 4, 64, "float16", 32),
                                                        (130, 700, 6, 3, 72, "bfloat16", 16), (257, 257, 4, 1, 64, "float16", 0)))
def test_attention_in_a_workspace_of_the_callers(torch, rng, lq, lk, h, hk, d, dtype, buckets):
    g = torch.Generator(device="cuda").manual_seed(lq)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(getattr(torch, dtype))

    q, do, k, v = normal(2, lq, h, d), normal(2, lq, h, d), normal(2, lk, hk, d), normal(2, lk, hk, d)
    table = normal(buckets, h) if buckets else None
    options = dict(bias_table=table, max_distance=100)
    results = []
    for own in (False, True):
        o, lse = torch.full_like(q, float("nan")), torch.full((2, h, lq), float("nan"), device="cuda")
        out = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        dtable = None if table is None else torch.full_like(table, float("nan"))
        fwd, bwd, beside = {}, {}, []
        if own:
            sizes = (rng.rng_attention_fwd_workspace(q, k, **options),
                     rng.rng_attention_bwd_workspace(q, k, dbias_table=dtable, **options))
            assert sizes[1] > 0 and (sizes[0] > 0) == (lq < 5)
            (fwd["workspace"], a), (bwd["workspace"], b) = (guarded(torch, n) for n in sizes)
            beside = [a, b]
            if sizes[0]:
                with pytest.raises(rng.RngError, match="workspace"):
                    rng.rng_attention_fwd(q, k, v, o, lse=lse, workspace=fwd["workspace"][:-4], **options)
            with pytest.raises(rng.RngError, match="workspace"):
                rng.rng_attention_bwd(do, q, k, v, o, lse, *out, dbias_table=dtable, workspace=bwd["workspace"][:-4], **options)
        common = dict(causal=True, queries_last=True, p=0.1, seed=5, **options)
        rng.rng_attention_fwd(q, k, v, o, lse=lse, **common, **fwd)
        rng.rng_attention_bwd(do, q, k, v, o, lse, *out, dbias_table=dtable, **common, **bwd)
        assert all(untouched() for untouched in beside)
        results.append([o, lse, *out] + ([] if table is None else [dtable]))
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*results))


@pytest.mark.gpu
def test_workspace_sizes_of_tensors_and_of_the_struct(torch, rng):
    q = torch.empty(2, 300, 4, 64, device="cuda", dtype=torch.float16)
    k = torch.empty(2, 77, 2, 64, device="cuda", dtype=torch.float16)
    table = torch.empty(32, 4, device="cuda", dtype=torch.float16)
    a = rng.AttentionArgs(dtype=rng.RNG_F16, batch=2, len_q=300, len_k=77, heads_q=4, heads_kv=2, head_dim=64, scale=0.125)
    assert rng.rng_attention_bwd_workspace(q, k) == rng.rng_attention_bwd_workspace(a)
    assert rng.rng_attention_fwd_workspace(q, k) == rng.rng_attention_fwd_workspace(a)
    a.bias_table, a.num_buckets, a.max_distance, a.bidirectional = table.data_ptr(), 32, 64, 1
    assert rng.rng_attention_bwd_workspace(q, k, bias_table=table, max_distance=64) == rng.rng_attention_bwd_workspace(a)
    a.dbias_table = table.data_ptr()
    size = rng.rng_attention_bwd_workspace(q, k, bias_table=table, dbias_table=table, max_distance=64)
    assert size == rng.rng_attention_bwd_workspace(a) > 0
    with pytest.raises(ValueError):
        rng.rng_attention_fwd_workspace(q)
    with pytest.raises(TypeError):
        rng.rng_attention_fwd_workspace(q.cpu(), k.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,dtype", ((700, 1024, "bfloat16"), (70, 769, "float16"), (40, 9000, "float32"),
                                             (3000, 64, "bfloat16")))
def test_norm_backward_in_a_workspace_of_the_callers(torch, rng, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy, h = (torch.randn(rows, cols, generator=g, device="cuda").to(getattr(torch, dtype)) for _ in range(2))
    mean, rstd = torch.randn(rows, generator=g, device="cuda"), torch.rand(rows, generator=g, device="cuda") + 0.5
    size = rng.rng_dropout_layer_norm_bwd_workspace(rows, cols)
    workspace, untouched = guarded(torch, size)
    results = []
    for more in ({}, {"workspace": workspace}):
        dx = torch.full_like(dy, float("nan"))
        grads = [torch.full((cols,), float("nan"), device="cuda", dtype=dy.dtype) for _ in range(3)]
        rng.rng_dropout_layer_norm_bwd(dy, h, None, mean, rstd, dx, *grads[:2], dbias=grads[2], p=0.2, seed=8, **more)
        results.append([dx, *grads])
    assert untouched() and all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*results))
    with pytest.raises(rng.RngError, match="workspace"):
        rng.rng_dropout_layer_norm_bwd(dy, h, None, mean, rstd, dx, *grads[:2], workspace=workspace[:-4])


# ---- sizes ---------------------------------------------------------------------------


def test_workspaces_without_query_heads():
    """In a process of its own: what it guards against ends the process."""
    code = """
import ctypes as C
import dropout_lowbias32_hash32_gb300 as rng
for causal in (0, 1):
    for scale in (0.125, 0.0):
        a = rng.AttentionArgs(dtype=rng.RNG_BF16, batch=2, len_q=4, len_k=4, heads_q=0, heads_kv=2, head_dim=64, scale=scale,
                              causal=causal)
        assert rng.rng_attention_fwd_workspace(a) == 0 and rng.rng_attention_bwd_workspace(a) == 0
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=120)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", (64, 128))
def test_without_query_heads_the_keys_gradients_are_zeros(torch, rng, dim):
    q = torch.empty(2, 5, 0, dim, device="cuda", dtype=torch.bfloat16)
    k, v, dk, dv = (torch.full((2, 150, 2, dim), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(4))
    lse = torch.empty(2, 0, 5, device="cuda")
    rng.rng_attention_fwd(q, k, v, q.clone(), lse=lse)
    rng.rng_attention_bwd(q, q, k, v, q, lse, q.clone(), dk, dv, causal=True, p=0.1)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dim", (64, 128))
def test_without_keys_or_queries_the_gradients_are_zeros(torch, rng, dim):
    some, none = (torch.randn(2, n, 2, dim, device="cuda").bfloat16() for n in (150, 0))
    table = torch.randn(8, 2, device="cuda").bfloat16()
    for q, k, lse in ((some, none, torch.full((2, 2, 150), -float("inf"), device="cuda")),
                      (none, some, torch.empty(2, 2, 0, device="cuda"))):
        dq, dk, dv, dtable = (torch.full_like(t, float("nan")) for t in (q, k, k, table))
        rng.rng_attention_bwd(q, q, k, k, torch.zeros_like(q), lse, dq, dk, dv, bias_table=table, dbias_table=dtable,
                              causal=True, p=0.1)
        assert all(bool((t == 0).all()) for t in (dq, dk, dv, dtable))


@pytest.mark.gpu
def test_rows_whose_three_sums_pass_2_to_32(torch, rng):
    """One row: dbias is dx, dbeta is dy and, as the statistics are 0 and 1, dgamma dy h, each rounded once."""
    cols = 1_440_000_007
    g = torch.Generator(device="cuda").manual_seed(6)
    dy, h = (torch.empty(1, cols, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    dx = torch.empty_like(dy)
    dgamma, dbeta, dbias = (torch.full((cols,), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(3))
    rng.rng_dropout_layer_norm_bwd(dy, h, None, mean, rstd, dx, dgamma, dbeta, dbias=dbias)
    assert torch.equal(dbias, dx[0]) and torch.equal(dbeta, dy[0]) and torch.equal(dgamma, dy[0] * h[0])
    del dy, h, dx, dgamma, dbeta, dbias
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_more_heads_than_a_grids_second_dimension(torch, rng):
    """The table's gradient of 70000 heads: the same bits as of two halves."""
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v, do = (torch.randn(1, 2, 70000, 8, generator=g, device="cuda").bfloat16() for _ in range(4))
    table = torch.randn(4, 70000, generator=g, device="cuda").bfloat16()

    def gradient(heads):
        part = [t[:, :, heads].contiguous() for t in (q, k, v, do)]
        bias = table[:, heads].contiguous()
        o, lse = torch.empty_like(part[0]), torch.empty(1, part[0].shape[2], 2, device="cuda")
        rng.rng_attention_fwd(*part[:3], o, lse=lse, bias_table=bias, max_distance=2)
        out = [torch.full_like(t, float("nan")) for t in (*part[:3], bias)]
        rng.rng_attention_bwd(part[3], *part[:3], o, lse, *out[:3], bias_table=bias, dbias_table=out[3], max_distance=2)
        return out[3]

    whole = gradient(slice(0, 70000))
    assert bool(whole.isfinite().all()) and float(whole.abs().max()) > 0.1
    assert torch.equal(whole, torch.cat([gradient(slice(0, 35000)), gradient(slice(35000, 70000))], 1))


@pytest.mark.gpu
def test_a_table_without_buckets_is_refused(torch, rng):
    q = torch.randn(1, 4, 2, 64, device="cuda").bfloat16()
    o, lse = torch.empty_like(q), torch.empty(1, 2, 4, device="cuda")
    none = torch.empty(0, 2, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="no buckets"):
        rng.rng_attention_fwd(q, q, q, o, bias_table=none)
    rng.rng_attention_fwd(q, q, q, o, lse=lse)
    with pytest.raises(ValueError, match="no buckets"):
        rng.rng_attention_bwd(q, q, q, q, o, lse, *(torch.empty_like(q) for _ in range(3)), bias_table=none)


# ---- what a request is batched with -----------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,h,hk,d,p,buckets", (
    (1, 300, 8, 8, 64, 0.0, 32), (1, 512, 16, 2, 128, 0.0, 0), (40, 40, 8, 8, 64, 0.1, 32), (77, 115, 6, 3, 40, 0.1, 0),
    (300, 20, 8, 8, 64, 0.0, 0), (150, 200, 4, 2, 128, 0.1, 16)))
def test_a_request_gets_the_same_bits_in_any_batch(torch, rng, lq, lk, h, hk, d, p, buckets):
    """Entry 0 alone, of 9 and of 65 (few enough keys that their axis is not split, whose parts go by the batch)."""
    g = torch.Generator(device="cuda").manual_seed(lq + lk)
    q, do = (torch.randn(65, lq, h, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn(65, lk, hk, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randn(buckets, h, generator=g, device="cuda").bfloat16() if buckets else None
    results = []
    for batch in (1, 9, 65):
        part = [t[:batch] for t in (q, k, v)]
        o, lse = torch.empty_like(part[0]), torch.empty(batch, h, lq, device="cuda")
        options = dict(bias_table=table, causal=True, queries_last=lq < lk, p=p, seed=2)
        rng.rng_attention_fwd(*part, o, lse=lse, **options)
        out = [torch.empty_like(t) for t in part]
        rng.rng_attention_bwd(do[:batch], *part, o, lse, *out, **options)
        results.append([t[0].clone() for t in (o, lse, *out)])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


# ---- overlaps (nothing below reaches the GPU) -----------------------------------------

A = 0x10000000  # an address that is never dereferenced


def norm_fwd(rng, x=A, bias=2 * A, residual=3 * A, gamma=4 * A, beta=5 * A, y=6 * A, h=7 * A, mean=8 * A, rstd=9 * A,
             stride=100, rows=4, cols=64):
    return rng.raw("rng_dropout_layer_norm_fwd")(x, stride, bias, residual, stride, gamma, beta, y, stride, h, stride,
                                                 mean, rstd, rows, cols, rng.RNG_BF16, rng.RNG_F32, 0.1, 1, 0, 1e-5,
                                                 None)


def norm_bwd(rng, dy=A, h=2 * A, dh=3 * A, gamma=4 * A, mean=5 * A, rstd=6 * A, dx=7 * A, dresidual=8 * A,
             dgamma=9 * A, dbeta=10 * A, dbias=11 * A, ws=12 * A, stride=100, rows=4, cols=64):
    need = rng.rng_dropout_layer_norm_bwd_workspace(rows, cols)
    return rng.raw("rng_dropout_layer_norm_bwd")(dy, stride, h, stride, dh, stride, gamma, mean, rstd, dx, stride,
                                                 dresidual, stride, dgamma, dbeta, dbias, rows, cols, rng.RNG_BF16,
                                                 rng.RNG_F32, 0.1, 1, 0, ws, need, None)


# rows of 128 bytes, 200 apart; weights of 256 bytes, statistics of 16
@pytest.mark.parametrize("bad,says", [
    ({"gamma": 6 * A}, "y and gamma"), ({"beta": 6 * A - 252}, "y and beta"), ({"bias": 7 * A + 600 + 124}, "h and bias"),
    ({"mean": 6 * A}, "y and mean"), ({"rstd": A}, "x and rstd"), ({"mean": 3 * A + 200}, "residual and mean"),
    ({"rstd": 8 * A + 12}, "mean and rstd"), ({"mean": 4 * A + 252}, "gamma and mean"),
    ({"mean": 6 * A, "rows": 1}, "y and mean"), ({"gamma": 6 * A + 124, "rows": 1}, "y and gamma")])
def test_norm_forward_refuses_overlaps(rng, bad, says):
    assert norm_fwd(rng, **bad) == rng.RNG_EINVAL
    assert says in rng.rng_last_error() and "overlap" in rng.rng_last_error()


@pytest.mark.parametrize("bad,says", [
    ({"dgamma": 4 * A}, "gamma and dgamma"), ({"dbeta": 9 * A + 252}, "dgamma and dbeta"),
    ({"dbias": 2 * A + 200}, "h and dbias"), ({"dx": 5 * A}, "dx and mean"), ({"dresidual": 6 * A + 8}, "dresidual and rstd"),
    ({"ws": A}, "dy and workspace"), ({"ws": 9 * A}, "dgamma and workspace"), ({"ws": 5 * A}, "mean and workspace"),
    ({"ws": 7 * A}, "dx and workspace"), ({"dgamma": 10 * A, "rows": 0}, "dgamma and dbeta")])
def test_norm_backward_refuses_overlaps(rng, bad, says):
    assert norm_bwd(rng, **bad) == rng.RNG_EINVAL
    assert says in rng.rng_last_error() and "overlap" in rng.rng_last_error()


@pytest.mark.gpu
def test_norm_beside_its_rows_is_fine(torch, rng):
    """Statistics and weights in the gaps of a wider array, and one after the
    other in one allocation."""
    rows, cols = 3, 64
    store = torch.zeros(rows, 512, device="cuda")
    x = torch.randn(rows, cols, device="cuda")
    y, gamma, mean, rstd = store[:, :cols], store[0, 64:128], store[1, 64:64 + rows], store[1, 64 + rows:64 + 2 * rows]
    gamma.fill_(2.0)
    rng.rng_dropout_layer_norm_fwd(x, gamma, None, y, mean, rstd)
    want = torch.empty_like(x)
    rng.rng_dropout_layer_norm_fwd(x, gamma.clone(), None, want)
    assert torch.equal(y, want) and bool((gamma == 2.0).all()) and bool((mean - x.mean(1)).abs().max() < 1e-6)


def attention_args(rng, strides=(1024, 256, 64), **change):
    """[2, 4, 2, 64] arrays, a position's two heads side by side and a gap of 128 elements after them."""
    a = rng.AttentionArgs(dtype=rng.RNG_BF16, batch=2, len_q=4, len_k=4, heads_q=2, heads_kv=2, head_dim=64, scale=0.125,
                          num_buckets=32, max_distance=128, bidirectional=1, workspace_bytes=1 << 20)
    names = ("q", "k", "v", "o", "d_o", "dq", "dk", "dv", "lse", "key_lengths", "bias_table", "dbias_table", "workspace")
    for i, n in enumerate(names):
        setattr(a, n, (i + 1) * A)
        if i < 8:
            setattr(a, "do_stride" if n == "d_o" else n + "_stride", strides)
    for n, v in change.items():
        setattr(a, n, v)
    return C.byref(a)


# lse: 64 bytes, key_lengths 8, tables 128; a position's heads use 256 of 512 bytes
@pytest.mark.parametrize("bad,says", [
    ({"lse": A}, "q and lse"), ({"lse": 4 * A + 128}, "o and lse"), ({"lse": 2 * A + 2048 + 512 * 3 + 252}, "k and lse"),
    ({"lse": 4 * A - 60}, "o and lse"), ({"bias_table": 4 * A + 1024}, "o and bias_table"),
    ({"key_lengths": 4 * A + 512 + 252}, "o and key_lengths"), ({"lse": 11 * A + 124}, "bias_table and lse"),
    ({"lse": 10 * A}, "key_lengths and lse"), ({"lse": 4 * A + 208}, "o and lse")])
def test_attention_forward_refuses_overlaps(rng, bad, says):
    assert rng.raw("rng_attention_fwd")(attention_args(rng, **bad), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error() and "overlap" in rng.rng_last_error()


@pytest.mark.gpu
def test_attention_forward_refuses_a_workspace_that_overlaps(torch, rng):
    """(How the key axis is split, and so whether there is a workspace, goes by the device.)"""
    q = torch.randn(1, 1, 8, 64, device="cuda").bfloat16()
    k = torch.randn(1, 8192, 8, 64, device="cuda").bfloat16()
    o, lse = torch.empty_like(q), torch.empty(1, 8, 1, device="cuda")
    with pytest.raises(rng.RngError, match="k and workspace overlap"):
        rng.rng_attention_fwd(q, k, k, o, lse=lse, workspace=k.view(-1))


@pytest.mark.parametrize("bad,says", [
    ({"lse": 6 * A}, "dq and lse"), ({"dbias_table": 6 * A}, "dq and dbias_table"), ({"dbias_table": 11 * A}, "bias_table and dbias_table"),
    ({"dbias_table": 4 * A + 256 - 16}, "o and dbias_table"), ({"bias_table": 8 * A}, "dv and bias_table"),
    ({"key_lengths": 7 * A}, "dk and key_lengths"), ({"dbias_table": 9 * A + 60}, "lse and dbias_table"),
    ({"workspace": 6 * A}, "dq and workspace"), ({"workspace": A - 64}, "q and workspace"),
    ({"workspace": 9 * A}, "lse and workspace"), ({"workspace": 12 * A + 112}, "dbias_table and workspace")])
def test_attention_backward_refuses_overlaps(rng, bad, says):
    assert rng.raw("rng_attention_bwd")(attention_args(rng, **bad), None) == rng.RNG_EINVAL
    assert says in rng.rng_last_error() and "overlap" in rng.rng_last_error()


@pytest.mark.gpu
def test_attention_beside_its_heads_is_fine(torch, rng):
    """lse, lengths, the table and its gradient in the gaps of the arrays."""
    g = torch.Generator(device="cuda").manual_seed(9)
    wide = {n: torch.zeros(2, 4, 4, 64, device="cuda").bfloat16() for n in ("q", "k", "v", "o", "do", "dq", "dk", "dv")}
    part = {n: t[:, :, 1:3] for n, t in wide.items()}
    for n in ("q", "k", "v", "do"):
        part[n].copy_(torch.randn(2, 4, 2, 64, generator=g, device="cuda"))
    lse = wide["o"][0, 1, 0].view(torch.float32)[:16].view(2, 2, 4)
    lengths = wide["dk"][1, 2, 3].view(torch.int32)[:2]
    lengths.copy_(torch.tensor([4, 3]))
    table, dtable = wide["dv"][0, 0, 3].view(32, 2), wide["dq"][1, 3, 0].view(32, 2)
    table.copy_(torch.randn(32, 2, generator=g, device="cuda"))
    options = dict(key_lengths=lengths, bias_table=table, p=0.1, seed=3)
    rng.rng_attention_fwd(part["q"], part["k"], part["v"], part["o"], lse=lse, **options)
    rng.rng_attention_bwd(part["do"], part["q"], part["k"], part["v"], part["o"], lse, part["dq"], part["dk"], part["dv"],
                          dbias_table=dtable, **options)
    own = {n: t.contiguous() for n, t in part.items()}
    options.update(key_lengths=lengths.clone(), bias_table=table.clone())
    lse2, dtable2 = torch.empty(2, 2, 4, device="cuda"), torch.empty(32, 2, device="cuda").bfloat16()
    out = {n: torch.empty_like(own[n]) for n in ("o", "dq", "dk", "dv")}
    rng.rng_attention_fwd(own["q"], own["k"], own["v"], out["o"], lse=lse2, **options)
    rng.rng_attention_bwd(own["do"], own["q"], own["k"], own["v"], out["o"], lse2, out["dq"], out["dk"], out["dv"],
                          dbias_table=dtable2, **options)
    assert all(torch.equal(out[n], part[n]) for n in out)
    assert torch.equal(lse, lse2) and torch.equal(dtable, dtable2)


# ---- biases that a score is lost beside -------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("value", (-3.3895313892515355e38, -1e9, 3e38))
@pytest.mark.parametrize("lq,lk,hk,d,causal,p", ((90, 90, 3, 64, False, 0.0), (200, 150, 3, 128, True, 0.1),
                                                 (150, 700, 1, 64, True, 0.0), (9, 70, 1, 64, False, 0.0),
                                                 (300, 270, 1, 72, False, 0.1)))
def test_gradients_of_rows_whose_biases_are_all_as_large(torch, rng, orc, lq, lk, hk, d, causal, p, value):
    """Head 0 has such an entry in every bucket, head 1 in the first few alone
    (so some of its rows see nothing else), head 2 has none.  An f32 score keeps
    nothing (or, beside 1e9, some) of q and k; a row's probabilities still add up
    to 1.  Where nothing is left they are one over the number of keys with the
    entry that wins, and the gradients are the formulas' with them."""
    import layer_reference as ref
    g = torch.Generator(device="cuda").manual_seed(lq)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    q, do = normal(2, lq, 3, d), normal(2, lq, 3, d)
    k, v, table = normal(2, lk, hk, d), normal(2, lk, hk, d), normal(16, 3)
    table[:, 0] = value
    table[:5, 1] = value
    o, lse = torch.empty_like(q), torch.empty(2, 3, lq, device="cuda")
    options = dict(bias_table=table, max_distance=64, bidirectional=False, causal=causal, p=p, seed=4)
    rng.rng_attention_fwd(q, k, v, o, lse=lse, **options)
    out = [torch.full_like(t, float("nan")) for t in (q, k, v, table)]
    rng.rng_attention_bwd(do, q, k, v, o, lse, *out[:3], dbias_table=out[3], **options)
    pairs = ref.Pairs(orc, q, k, None, causal, False, 16, 64, False, p, 4, 0)
    if p == 0.0:  # sum over j of dv = sum over i of (sum over j of P) do, with P rounded to 2^-8 of itself
        heads = do.double().unflatten(2, (hk, -1))
        assert bool(((out[2].double().sum(1) - heads.sum((1, 3))).abs() <= 2.0 ** -7 * heads.abs().sum((1, 3))).all())
    if abs(value) < 1e30:
        return
    # (64 bits would lose the sum's logarithm beside such a score as well)
    prob = ref.scores(q, k, table, pairs, d ** -0.5).softmax(-1)
    want = ((prob * pairs.keep) @ ref.heads_first(v, 3 // hk)).transpose(1, 2)
    ut, av = 2.0 ** -8, ref.heads_first(v, 3 // hk).abs()
    # two roundings of P, 2^-19 for its exponential (whose argument is exact here, or a score's), and one of o
    tol = ((2 * ut + 2.0 ** -17) * (prob * pairs.keep) @ av).transpose(1, 2) + ut * want.abs() + 2.0 ** -20
    assert bool(((o.double() - want).abs() <= tol).all())
    dq, dk, dv, dtable, ds = ref.attention_bwd(do, q, k, v, o, table, pairs, prob, d ** -0.5)
    # dS and P rounded once, the f32 sums behind dP - delta, the result rounded once
    ado, ao, aq, ak = *(ref.heads_first(t).abs() for t in (do, o, q)), ref.heads_first(k, 3 // hk).abs()
    err = (d + 8) * 2.0 ** -23 * (ado @ av.transpose(2, 3) / (1 - p) + (ado * ao).sum(-1, keepdim=True))
    w = (ut + 2.0 ** -17) * ds.abs() + 2 * prob * err
    assert bool(((out[0].double() - dq).abs() <= (w @ ak * d ** -0.5).transpose(1, 2) + ut * dq.abs() + 1e-30).all())
    assert bool(((out[1].double() - dk).abs() <= ref.shared(w.transpose(2, 3) @ aq * d ** -0.5, hk) + ut * dk.abs() + 1e-30).all())
    wv = (ut + 2.0 ** -17) * prob * pairs.keep
    assert bool(((out[2].double() - dv).abs() <= ref.shared(wv.transpose(2, 3) @ ado, hk) + ut * dv.abs() + 1e-30).all())
    tol = ref.by_bucket((2.0 ** -17 + 2.0 ** -12) * ds.abs() + 2 * prob * err, table, pairs)
    assert bool(((out[3].double() - dtable).abs() <= tol + ut * dtable.abs() + 1e-30).all())


# ---- captured, and again -----------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,buckets", ((150, 150, 32), (1, 5000, 0), (600, 600, 0)))
def test_a_captured_training_step(torch, rng, lq, lk, buckets):
    """Forward and backward of both operators in one graph, replayed with new inputs, against plain calls."""
    g = torch.Generator(device="cuda").manual_seed(lq)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    q, x, do = normal(2, lq, 4, 64), normal(2, lq, 256), normal(2, lq, 256)
    k, v, gamma = normal(2, lk, 2, 64), normal(2, lk, 2, 64), normal(256)
    table = normal(buckets, 4) if buckets else None
    options = dict(bias_table=table, causal=True, queries_last=True, p=0.1, seed=7)

    def step():
        o, lse, y, h = torch.empty_like(q), torch.empty(2, 4, lq, device="cuda"), torch.empty_like(x), torch.empty_like(x)
        mean, rstd = (torch.empty(2, lq, device="cuda") for _ in range(2))
        rng.rng_attention_fwd(q, k, v, o, lse=lse, **options)
        rng.rng_dropout_layer_norm_fwd(o.view(2, lq, 256), gamma, None, y, mean, rstd, residual=x, h=h, p=0.1, seed=8)
        dx, dres, dgamma = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gamma)
        rng.rng_dropout_layer_norm_bwd(do, h, gamma, mean, rstd, dx, dgamma, dresidual=dres, p=0.1, seed=8)
        out = [torch.empty_like(t) for t in (q, k, v)]
        dtable = torch.empty_like(table) if buckets else None
        rng.rng_attention_bwd(dx.view(2, lq, 4, 64), q, k, v, o, lse, *out, dbias_table=dtable, **options)
        return [o, lse, y, h, dx, dres, dgamma, *out] + ([dtable] if buckets else [])

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        for t in (q, k, v, x, do):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        for t in captured:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(captured, step()))


# ---- queries that see nothing --------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ("bfloat16", "float16"))
@pytest.mark.parametrize("lq,lk,h,hk,d,buckets,p", ((300, 200, 4, 2, 64, 0, 0.1), (200, 180, 2, 1, 128, 16, 0.0),
                                                    (70, 30, 2, 2, 64, 32, 0.1), (150, 149, 6, 2, 72, 0, 0.0)))
def test_queries_that_see_nothing_pass_no_gradient_whatever_they_hold(torch, rng, dtype, lq, lk, h, hk, d, buckets, p):
    """The last queries of caches that are shorter than they: those before the
    first key hold NaN and infinities, or zeros; the rest has the same bits."""
    g = torch.Generator(device="cuda").manual_seed(lq)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(getattr(torch, dtype))

    q, do, k, v = normal(4, lq, h, d), normal(4, lq, h, d), normal(4, lk, hk, d), normal(4, lk, hk, d)
    table = normal(buckets, h) if buckets else None
    lengths = torch.tensor([lk, 0, lk // 2, 1], dtype=torch.int32, device="cuda")
    unseen = (torch.arange(lq, device="cuda")[None, :] < lq - lengths[:, None])[:, :, None, None]
    results = []
    for fill in (0.0, float("nan"), float("inf")):
        a, b = q.masked_fill(unseen, fill), do.masked_fill(unseen, fill)
        o, lse = torch.empty_like(q), torch.empty(4, h, lq, device="cuda")
        options = dict(key_lengths=lengths, causal=True, queries_last=True, bias_table=table, p=p, seed=6)
        rng.rng_attention_fwd(a, k, v, o, lse=lse, **options)
        out = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        dtable = torch.full_like(table, float("nan")) if buckets else None
        rng.rng_attention_bwd(b, a, k, v, o, lse, *out, dbias_table=dtable, **options)
        results.append([o, lse, *out] + ([dtable] if buckets else []))
    assert all(bool(t.isfinite().all()) for t in results[0][2:])
    assert bool((results[0][2].masked_select(unseen) == 0).all())
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))

"""Stateless counter-based random fills (lowbias32 hash32) for GB300.

A thin ctypes binding of the C ABI in include/rng.h: every function here
carries the C entry point's name, marshals a CUDA tensor's pointer, length
and the current stream, and raises on a non-OK status.  All work runs in the
library's sm_103a kernels; there is no fallback: if the library has not been
built, importing this package fails.

    import torch, dropout_lowbias32_hash32_gb300 as rng
    out = torch.empty(1 << 28, dtype=torch.float32, device="cuda")
    rng.rng_fill_f32(seed=1, first_counter=0, out=out)
"""
from __future__ import annotations

import ctypes as C
import os
import struct

from . import sharding  # noqa: F401  (counter ranges for multi-process fills)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_PKG, "_lib", "librng_lowbias32.so")

if not os.path.exists(LIBRARY_PATH):
    raise ImportError(
        f"{LIBRARY_PATH} is missing: build the CUDA library first "
        "(python dropout_lowbias32_hash32_gb300/build.py, or __graft_entry__.build())")

_lib = C.CDLL(LIBRARY_PATH)

_u32, _u64, _i32, _i64, _sz = C.c_uint32, C.c_uint64, C.c_int32, C.c_int64, C.c_size_t
_p, _f32, _int = C.c_void_p, C.c_float, C.c_int

# name -> argument types (every entry point returns rng_status = int)
_FILL_SIGS = {
    "rng_fill_u32": [_u32, _u32, _sz, _p, _p],
    "rng_fill_u64": [_u32, _u32, _sz, _p, _p],
    "rng_fill_f32": [_u32, _u32, _sz, _p, _p],
    "rng_fill_f64": [_u32, _u32, _sz, _p, _p],
    "rng_fill_u8": [_u32, _u32, _sz, _p, _p],
    "rng_fill_u16": [_u32, _u32, _sz, _p, _p],
    "rng_fill_f16": [_u32, _u32, _sz, _p, _p],
    "rng_fill_bool": [_u32, _u32, _sz, _p, _p],
    "rng_fill_u32_below": [_u32, _u32, _sz, _u32, _p, _p],
    "rng_fill_u64_below": [_u32, _u32, _sz, _u64, _p, _p],
    "rng_fill_i32_range": [_u32, _u32, _sz, _i32, _u32, _p, _p],
    "rng_fill_i64_range32": [_u32, _u32, _sz, _i64, _u32, _p, _p],
    "rng_fill_i64_range": [_u32, _u32, _sz, _i64, _u64, _p, _p],
    "rng_fill_normal_f32": [_u32, _u32, _sz, _p, _p],
    "rng_fill_normal_f32_pairs": [_u32, _u32, _sz, _p, _p],
    "rng_fill_normal_f32_precise": [_u32, _u32, _sz, _p, _p],
    "rng_fill_exponential_f32": [_u32, _u32, _sz, _p, _p],
    "rng_fill_exponential_f64": [_u32, _u32, _sz, _p, _p],
    "rng_fill_normal_f64": [_u32, _u32, _sz, _p, _p],
    "rng_fill_normal_f64_noalloc": [_u32, _u32, _sz, _p, _p],
    "rng_dropout_fwd": [_p, _p, _f32, _u32, _u32, _sz, _p],
    "rng_dropout_bwd": [_p, _p, _f32, _u32, _u32, _sz, _p],
    "rng_dropout_layer_norm_fwd": [_p, _sz, _p, _p, _sz, _p, _p, _p, _sz, _p, _sz, _p, _p, _sz, _sz, _int, _int, _f32,
                                   _u32, _u32, _f32, _p],
    "rng_dropout_layer_norm_bwd": [_p, _sz, _p, _sz, _p, _sz, _p, _p, _p, _p, _sz, _p, _sz, _p, _p, _p, _sz, _sz, _int,
                                   _int, _f32, _u32, _u32, _p, _sz, _p],
    "rng_attention_fwd": [_p, _p],
    "rng_attention_bwd": [_p, _p],
    "rng_relative_bucket": [_i64, _i32, _i32, _i32, C.POINTER(_i32)],
    "rng_debug_set_miss_capacity": [_sz],
    "rng_debug_last_miss_count": [C.POINTER(_u64)],
    "rng_debug_stalled_waits": [C.POINTER(_u64)],
    "rng_debug_eval_f64": [_int, _p, _p, _sz, _p],
    "rng_debug_write_ceiling": [_int, _p, _sz, _p],
}
for _name, _args in _FILL_SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _int
for _name, _args in {"rng_dropout_layer_norm_bwd_workspace": [_sz, _sz], "rng_attention_fwd_workspace": [_p],
                     "rng_attention_bwd_workspace": [_p]}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _sz
_lib.rng_status_string.argtypes = [_int]
_lib.rng_status_string.restype = C.c_char_p
_lib.rng_last_error.argtypes = []
_lib.rng_last_error.restype = C.c_char_p
_lib.rng_debug_launch_count.argtypes = []
_lib.rng_debug_launch_count.restype = _u64

RNG_OK, RNG_EINVAL, RNG_ECUDA, RNG_ENOMEM = 0, 1, 2, 3


class RngError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.rng_status_string(status).decode()
        detail = _lib.rng_last_error().decode()
        super().__init__(f"{where}: {msg}" + (f" ({detail})" if detail else ""))


def _check(status: int, where: str) -> None:
    if status != RNG_OK:
        raise RngError(status, where)


def raw(name: str):
    """The ctypes function of a C entry point (plain pointers and sizes)."""
    return getattr(_lib, name)


# ---- tensor marshalling -------------------------------------------------------
_ALLOWED = {
    "u32": ("uint32", "int32"), "u64": ("uint64", "int64"), "i32": ("int32",), "i64": ("int64",),
    "f32": ("float32",), "f64": ("float64",), "u8": ("uint8", "int8", "bool"), "u16": ("uint16", "int16"),
    "f16": ("float16", "uint16", "int16"),
}


def _ptr(t, kind: str, name: str = "out") -> tuple[int, int]:
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    if str(t.dtype).replace("torch.", "") not in _ALLOWED[kind]:
        raise TypeError(f"{name} must have dtype {' or '.join(_ALLOWED[kind])}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), t.numel()


def _stream(stream, t) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream(t.device).cuda_stream or None
    return int(getattr(stream, "cuda_stream", stream)) or None


def _on_device(t):
    """The library launches on the CUDA runtime's current device: make it the
    tensor's for the duration of a call."""
    import torch
    return torch.cuda.device(t.device)


def _fill(name, kind, seed, first_counter, out, stream, *extra):
    p, n = _ptr(out, kind)
    with _on_device(out):
        _check(getattr(_lib, name)(seed & 0xFFFFFFFF, first_counter & 0xFFFFFFFF, n, *extra, p,
                                   _stream(stream, out)), name)
    return out


def rng_fill_u32(seed, first_counter, out, stream=None):
    return _fill("rng_fill_u32", "u32", seed, first_counter, out, stream)


def rng_fill_u64(seed, first_counter, out, stream=None):
    return _fill("rng_fill_u64", "u64", seed, first_counter, out, stream)


def rng_fill_f32(seed, first_counter, out, stream=None):
    return _fill("rng_fill_f32", "f32", seed, first_counter, out, stream)


def rng_fill_f64(seed, first_counter, out, stream=None):
    return _fill("rng_fill_f64", "f64", seed, first_counter, out, stream)


def rng_fill_u8(seed, first_counter, out, stream=None):
    return _fill("rng_fill_u8", "u8", seed, first_counter, out, stream)


def rng_fill_u16(seed, first_counter, out, stream=None):
    return _fill("rng_fill_u16", "u16", seed, first_counter, out, stream)


def rng_fill_f16(seed, first_counter, out, stream=None):
    return _fill("rng_fill_f16", "f16", seed, first_counter, out, stream)


def rng_fill_bool(seed, first_counter, out, stream=None):
    return _fill("rng_fill_bool", "u8", seed, first_counter, out, stream)


def rng_fill_u32_below(seed, first_counter, bound, out, stream=None):
    return _fill("rng_fill_u32_below", "u32", seed, first_counter, out, stream, bound)


def rng_fill_u64_below(seed, first_counter, bound, out, stream=None):
    return _fill("rng_fill_u64_below", "u64", seed, first_counter, out, stream, bound)


def rng_fill_i32_range(seed, first_counter, low, bound, out, stream=None):
    return _fill("rng_fill_i32_range", "i32", seed, first_counter, out, stream, low, bound)


def rng_fill_i64_range32(seed, first_counter, low, bound, out, stream=None):
    return _fill("rng_fill_i64_range32", "i64", seed, first_counter, out, stream, low, bound)


def rng_fill_i64_range(seed, first_counter, low, bound, out, stream=None):
    return _fill("rng_fill_i64_range", "i64", seed, first_counter, out, stream, low, bound)


def rng_fill_normal_f32(seed, first_counter, out, stream=None):
    return _fill("rng_fill_normal_f32", "f32", seed, first_counter, out, stream)


def rng_fill_normal_f32_pairs(seed, first_counter, out, stream=None):
    return _fill("rng_fill_normal_f32_pairs", "f32", seed, first_counter, out, stream)


def rng_fill_normal_f32_precise(seed, first_counter, out, stream=None):
    return _fill("rng_fill_normal_f32_precise", "f32", seed, first_counter, out, stream)


def rng_fill_exponential_f32(seed, first_counter, out, stream=None):
    return _fill("rng_fill_exponential_f32", "f32", seed, first_counter, out, stream)


def rng_fill_exponential_f64(seed, first_counter, out, stream=None):
    return _fill("rng_fill_exponential_f64", "f64", seed, first_counter, out, stream)


def rng_fill_normal_f64(seed, first_counter, out, stream=None):
    return _fill("rng_fill_normal_f64", "f64", seed, first_counter, out, stream)


def rng_fill_normal_f64_noalloc(seed, first_counter, out, stream=None):
    """rng_fill_normal_f64 without any device allocation (n <= 2^28); see rng.h."""
    return _fill("rng_fill_normal_f64_noalloc", "f64", seed, first_counter, out, stream)


def _dropout(name, x, y, p, seed, first_counter, stream):
    px, n = _ptr(x, "f32", "x")
    py, ny = _ptr(y, "f32", "y")
    if n != ny:
        raise ValueError(f"{name}: x has {n} elements, y has {ny}")
    if x.device != y.device:
        raise ValueError(f"{name}: x is on {x.device}, y on {y.device}")
    with _on_device(y):
        _check(getattr(_lib, name)(px, py, float(p), seed & 0xFFFFFFFF, first_counter & 0xFFFFFFFF, n,
                                   _stream(stream, y)), name)
    return y


def rng_dropout_fwd(x, y, p, seed, first_counter, stream=None):
    return _dropout("rng_dropout_fwd", x, y, p, seed, first_counter, stream)


def rng_dropout_bwd(dy, dx, p, seed, first_counter, stream=None):
    return _dropout("rng_dropout_bwd", dy, dx, p, seed, first_counter, stream)


# ---- a transformer layer's dropout ----------------------------------------------
RNG_F32, RNG_F16, RNG_BF16 = 0, 1, 2


class AttentionArgs(C.Structure):
    """rng_attention_args of include/rng.h."""
    _fields_ = [("dtype", _int), ("batch", _i32), ("len_q", _i32), ("len_k", _i32), ("heads_q", _i32),
                ("heads_kv", _i32), ("head_dim", _i32), ("q", _p), ("k", _p), ("v", _p), ("q_stride", _i64 * 3),
                ("k_stride", _i64 * 3), ("v_stride", _i64 * 3), ("o", _p), ("o_stride", _i64 * 3), ("lse", _p),
                ("key_lengths", _p), ("causal", _i32), ("queries_last", _i32), ("scale", _f32), ("bias_table", _p),
                ("num_buckets", _i32), ("max_distance", _i32), ("bidirectional", _i32), ("p", _f32), ("seed", _u32),
                ("first_counter", _u32), ("d_o", _p), ("dq", _p), ("dk", _p), ("dv", _p), ("do_stride", _i64 * 3),
                ("dq_stride", _i64 * 3), ("dk_stride", _i64 * 3), ("dv_stride", _i64 * 3), ("dbias_table", _p),
                ("workspace", _p), ("workspace_bytes", _sz)]


# The same struct as bytes, which a small call fills in less time than the
# struct's fields one by one (native alignment, as the C struct's).
_pack_attention = struct.Struct("@7i3P9qP3q2P2if1P3if2I4P12q2PN").pack
assert struct.calcsize("@7i3P9qP3q2P2if1P3if2I4P12q2PN") == C.sizeof(AttentionArgs)

_torch = None  # torch, from the first call on (importing this package does not import it)
_codes: dict = {}  # torch dtype -> rng_dtype
_raw_stream = None  # device index -> the current stream's handle


def _load_torch():
    global _torch, _raw_stream
    import torch
    _codes.update({torch.float32: RNG_F32, torch.float16: RNG_F16, torch.bfloat16: RNG_BF16})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch


def _first(t, name: str) -> int:
    """The rng_dtype of the tensor whose device and dtype the others follow."""
    if _torch is None:
        _load_torch()
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must have dtype float32, float16 or bfloat16, not {t.dtype}")
    return code


def _same(t, name: str, like, like_name: str, dtype) -> None:
    """t lies on like's device and has the dtype."""
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, {like_name} on {like.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, not {t.dtype}")


def _rows(t, name: str, like, like_name: str) -> tuple:
    """(pointer, elements between rows) of a [..., cols] tensor of like's shape
    whose leading dimensions lie one row stride apart; (None, 0) for None."""
    if t is None:
        return None, 0
    if t is not like:
        if t.dtype is not like.dtype or t.device != like.device:
            _same(t, name, like, like_name, like.dtype)
        if t.shape != like.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, {like_name} {tuple(like.shape)}")
    if t.is_contiguous() or t.numel() == 0:
        return t.data_ptr(), t.shape[-1]
    stride, rows = None, 1  # from the last leading dimension out
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride = s
        elif s != stride * rows:
            raise ValueError(f"{name}'s rows must lie one stride apart")
        rows *= n
    if t.shape[-1] != 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), t.shape[-1] if stride is None else stride


def _flat(t, name: str, n: int, like, like_name: str, dtype) -> int | None:
    """Pointer of a contiguous tensor of n elements; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != like.device:
        _same(t, name, like, like_name, dtype)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} elements")
    return t.data_ptr()


def _size(t, name: str) -> tuple:
    """(rows, columns) of a [..., cols] tensor."""
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    cols = t.shape[-1]
    return (t.numel() // cols if cols else 0), cols


def _weight_dtype(like, *weights):
    """The weights' common dtype (the activations' when there are none)."""
    for w in weights:
        if w is not None:
            if w.dtype not in _codes:
                raise TypeError(f"a weight must have dtype float32, float16 or bfloat16, not {w.dtype}")
            return w.dtype, _codes[w.dtype]
    return like.dtype, _codes[like.dtype]


def _scratch(workspace, need: int, like, stream):
    """(pointer, bytes, tensor) of the caller's workspace, or of one of the
    caching allocator's; (None, 0, None) where none is needed."""
    if need == 0:
        return None, 0, None
    if workspace is None:
        # From the pool of the stream that the kernels run on: a block that another stream has given back may still
        # be used by that stream's queued work.
        if stream is None:
            workspace = _torch.empty(need, dtype=_torch.uint8, device=like.device)
        else:
            if not isinstance(stream, _torch.cuda.Stream):
                handle = int(getattr(stream, "cuda_stream", stream))
                stream = (_torch.cuda.ExternalStream(handle, device=like.device) if handle
                          else _torch.cuda.default_stream(like.device))
            with _torch.cuda.stream(stream):
                workspace = _torch.empty(need, dtype=_torch.uint8, device=like.device)
    elif workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _handle(stream, index: int) -> int | None:
    return (_raw_stream(index) if stream is None else int(getattr(stream, "cuda_stream", stream))) or None


class _Current:
    """Makes a device the current one, where it is not."""
    __slots__ = ("index", "before")

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.before = _torch.cuda.current_device()
        if self.before != self.index:
            _torch.cuda.set_device(self.index)

    def __exit__(self, *_):
        if self.before != self.index:
            _torch.cuda.set_device(self.before)


def rng_dropout_layer_norm_fwd(x, gamma, beta, y, mean=None, rstd=None, *, bias=None, residual=None, h=None, p=0.0,
                               seed=0, first_counter=0, eps=1e-5, stream=None):
    """h = residual + dropout(x + bias); y = (h - mean) * rstd * gamma + beta
    over the last dimension; see rng.h.  Writes y and, where given, h, mean
    and rstd; returns y."""
    code = _first(x, "x")
    rows, cols = _size(x, "x")
    wd, wcode = _weight_dtype(x, gamma, beta, bias)
    f32, index = _torch.float32, x.get_device()
    px, sx = _rows(x, "x", x, "x")
    pr, sr = _rows(residual, "residual", x, "x")
    py, sy = _rows(y, "y", x, "x")
    ph, sh = _rows(h, "h", x, "x")
    pb = _flat(bias, "bias", cols, x, "x", wd)
    pg, pe = _flat(gamma, "gamma", cols, x, "x", wd), _flat(beta, "beta", cols, x, "x", wd)
    pm, ps = _flat(mean, "mean", rows, x, "x", f32), _flat(rstd, "rstd", rows, x, "x", f32)
    with _Current(index):
        status = _lib.rng_dropout_layer_norm_fwd(px, sx, pb, pr, sr, pg, pe, py, sy, ph, sh, pm, ps, rows, cols, code,
                                                 wcode, p, seed & 0xFFFFFFFF, first_counter & 0xFFFFFFFF, eps,
                                                 _handle(stream, index))
    if status:
        _check(status, "rng_dropout_layer_norm_fwd")
    return y


def rng_dropout_layer_norm_bwd_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of rng_dropout_layer_norm_bwd on the current device."""
    return _lib.rng_dropout_layer_norm_bwd_workspace(rows, cols)


def rng_dropout_layer_norm_bwd(dy, h, gamma, mean, rstd, dx, dgamma=None, dbeta=None, *, dh=None, dresidual=None,
                               dbias=None, p=0.0, seed=0, first_counter=0, workspace=None, stream=None):
    """The gradient of rng_dropout_layer_norm_fwd from its h, mean and rstd;
    dh is the gradient that reaches h past the norm.  Writes dx and, where
    given, dresidual, dgamma, dbeta and dbias; returns dx."""
    code = _first(dy, "dy")
    rows, cols = _size(dy, "dy")
    wd, wcode = _weight_dtype(dy, gamma, dgamma, dbeta, dbias)
    f32, index = _torch.float32, dy.get_device()
    py, sy = _rows(dy, "dy", dy, "dy")
    ph, sh = _rows(h, "h", dy, "dy")
    pd, sd = _rows(dh, "dh", dy, "dy")
    px, sx = _rows(dx, "dx", dy, "dy")
    pr, sr = _rows(dresidual, "dresidual", dy, "dy")
    pg, pm = _flat(gamma, "gamma", cols, dy, "dy", wd), _flat(mean, "mean", rows, dy, "dy", f32)
    ps, pdg = _flat(rstd, "rstd", rows, dy, "dy", f32), _flat(dgamma, "dgamma", cols, dy, "dy", wd)
    pde, pdb = _flat(dbeta, "dbeta", cols, dy, "dy", wd), _flat(dbias, "dbias", cols, dy, "dy", wd)
    with _Current(index):
        ws, ws_bytes, hold = _scratch(workspace, _lib.rng_dropout_layer_norm_bwd_workspace(rows, cols), dy, stream)
        status = _lib.rng_dropout_layer_norm_bwd(py, sy, ph, sh, pd, sd, pg, pm, ps, px, sx, pr, sr, pdg, pde, pdb,
                                                 rows, cols, code, wcode, p, seed & 0xFFFFFFFF,
                                                 first_counter & 0xFFFFFFFF, ws, ws_bytes, _handle(stream, index))
    if status:
        _check(status, "rng_dropout_layer_norm_bwd")
    del hold
    return dx


def _heads(t, name: str, shape, like) -> tuple:
    """Pointer and strides of a [batch, length, heads, head_dim] tensor."""
    if t.dtype is not like.dtype or t.device != like.device:
        _same(t, name, like, "q", like.dtype)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    b, l, h, d = t.stride()
    if d != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), b, l, h


_NO_GRADIENT = (0, 0, 0, 0)  # pointer, strides


def _attention(name, q, k, v, o, lse, key_lengths, causal, queries_last, scale, bias_table, max_distance,
               bidirectional, p, seed, first_counter, gradients, dbias_table, workspace, stream):
    code = _first(q, "q")
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be [batch, length, heads, head_dim]")
    shape = q.shape
    batch, len_q, heads, dim = shape
    key_shape = (batch, k.shape[1], k.shape[2], dim)
    pq, qb, ql, qh = _heads(q, "q", shape, q)
    pk, kb, kl, kh = _heads(k, "k", key_shape, q)
    pv, vb, vl, vh = _heads(v, "v", key_shape, q)
    po, ob, ol, oh = _heads(o, "o", shape, q)
    if lse is not None and lse.shape != (batch, heads, len_q):
        raise ValueError(f"lse has shape {tuple(lse.shape)}, not [batch, heads, len_q]")
    plse = _flat(lse, "lse", batch * heads * len_q, q, "q", _torch.float32)
    plen = _flat(key_lengths, "key_lengths", batch, q, "q", _torch.int32)
    buckets = 0
    if bias_table is not None:
        if bias_table.dim() != 2 or bias_table.shape[1] != heads:
            raise ValueError(f"bias_table has shape {tuple(bias_table.shape)}, not [num_buckets, heads]")
        buckets = bias_table.shape[0]
        if buckets == 0:  # whose null pointer would say that there is no table
            raise ValueError("bias_table has no buckets")
    elif dbias_table is not None:
        raise ValueError("dbias_table without a bias_table")
    pt = _flat(bias_table, "bias_table", buckets * heads, q, "q", q.dtype)
    pdt = _flat(dbias_table, "dbias_table", buckets * heads, q, "q", q.dtype)
    do, dq, dk, dv = _NO_GRADIENT, _NO_GRADIENT, _NO_GRADIENT, _NO_GRADIENT
    if gradients is not None:
        do, dq = _heads(gradients[0], "do", shape, q), _heads(gradients[1], "dq", shape, q)
        dk, dv = _heads(gradients[2], "dk", key_shape, q), _heads(gradients[3], "dv", key_shape, q)
    fields = (code, batch, len_q, key_shape[1], heads, key_shape[2], dim, pq, pk, pv, qb, ql, qh, kb, kl, kh, vb, vl,
              vh, po, ob, ol, oh, plse or 0, plen or 0, bool(causal), bool(queries_last),
              dim ** -0.5 if scale is None else scale, pt or 0, buckets, max_distance if buckets else 0,
              bool(bidirectional), p, seed & 0xFFFFFFFF, first_counter & 0xFFFFFFFF, do[0], dq[0], dk[0], dv[0],
              *do[1:], *dq[1:], *dk[1:], *dv[1:], pdt or 0)
    index = q.get_device()
    with _Current(index):
        args = _pack_attention(*fields, 0, 0)
        ws, ws_bytes, hold = _scratch(workspace, getattr(_lib, name + "_workspace")(args), q, stream)
        if ws_bytes:
            args = _pack_attention(*fields, ws, ws_bytes)
        status = getattr(_lib, name)(args, _handle(stream, index))
    if status:
        _check(status, name)
    del hold


def _attention_workspace(name, q, k, scale, bias_table, dbias_table, max_distance, bidirectional) -> int:
    if isinstance(q, AttentionArgs):
        return getattr(_lib, name)(C.byref(q))
    code = _first(q, "q")
    if q.dim() != 4 or k is None or k.dim() != 4:
        raise ValueError("q and k must be [batch, length, heads, head_dim]")
    batch, len_q, heads, dim = q.shape
    table = 0 if bias_table is None else bias_table.data_ptr()
    buckets = bias_table.shape[0] if table else 0
    args = _pack_attention(code, batch, len_q, k.shape[1], heads, k.shape[2], dim, 0, 0, 0, *(0,) * 9, 0, 0, 0, 0, 0, 0,
                           False, False, dim ** -0.5 if scale is None else scale, table, buckets,
                           max_distance if buckets else 0, bool(bidirectional), 0.0, 0, 0, *(0,) * 16,
                           0 if dbias_table is None else dbias_table.data_ptr(), 0, 0)
    with _Current(q.get_device()):
        return getattr(_lib, name)(args)


def rng_attention_fwd_workspace(q, k=None, *, scale=None, bias_table=None, max_distance=128, bidirectional=True) -> int:
    """Bytes of workspace of rng_attention_fwd for q and k on their device (or
    of an AttentionArgs on the current one); 0 also where the call itself would
    be refused."""
    return _attention_workspace("rng_attention_fwd_workspace", q, k, scale, bias_table, None, max_distance,
                                bidirectional)


def rng_attention_bwd_workspace(q, k=None, *, scale=None, bias_table=None, dbias_table=None, max_distance=128,
                                bidirectional=True) -> int:
    """Bytes of workspace of rng_attention_bwd, likewise."""
    return _attention_workspace("rng_attention_bwd_workspace", q, k, scale, bias_table, dbias_table, max_distance,
                                bidirectional)


def rng_attention_fwd(q, k, v, o, *, lse=None, key_lengths=None, causal=False, queries_last=False, scale=None,
                      bias_table=None, max_distance=128, bidirectional=True, p=0.0, seed=0, first_counter=0,
                      workspace=None, stream=None):
    """Attention with a bucketed relative position bias and dropout on its
    probabilities; q and o are [batch, len_q, heads, head_dim], k and v
    [batch, len_k, key heads, head_dim] (any strides, the last dimension
    contiguous); scale None: head_dim ** -0.5; see rng.h.  Writes o and, where
    given, lse [batch, heads, len_q]; returns o."""
    _attention("rng_attention_fwd", q, k, v, o, lse, key_lengths, causal, queries_last, scale, bias_table,
               max_distance, bidirectional, p, seed, first_counter, None, None, workspace, stream)
    return o


def rng_attention_bwd(do, q, k, v, o, lse, dq, dk, dv, *, dbias_table=None, key_lengths=None, causal=False,
                      queries_last=False, scale=None, bias_table=None, max_distance=128, bidirectional=True, p=0.0,
                      seed=0, first_counter=0, workspace=None, stream=None):
    """The gradient of rng_attention_fwd from its o and lse and the same
    options.  Writes dq, dk, dv and, where given, dbias_table; returns dq, dk, dv."""
    _attention("rng_attention_bwd", q, k, v, o, lse, key_lengths, causal, queries_last, scale, bias_table,
               max_distance, bidirectional, p, seed, first_counter, (do, dq, dk, dv), dbias_table, workspace, stream)
    return dq, dk, dv


def rng_relative_bucket(relative_position: int, num_buckets: int, max_distance: int = 128,
                        bidirectional: bool = True) -> int:
    """The bucket of a relative position (the key's minus the query's)."""
    bucket = _i32()
    _check(_lib.rng_relative_bucket(relative_position, num_buckets, max_distance, bool(bidirectional),
                                    C.byref(bucket)), "rng_relative_bucket")
    return bucket.value


def rng_status_string(status: int) -> str:
    return _lib.rng_status_string(status).decode()


def rng_last_error() -> str:
    return _lib.rng_last_error().decode()


def rng_debug_set_miss_capacity(capacity: int | None) -> None:
    _check(_lib.rng_debug_set_miss_capacity((1 << 64) - 1 if capacity is None else capacity),
           "rng_debug_set_miss_capacity")


def rng_debug_last_miss_count() -> int:
    c = _u64()
    _check(_lib.rng_debug_last_miss_count(C.byref(c)), "rng_debug_last_miss_count")
    return c.value


def rng_debug_stalled_waits() -> int:
    c = _u64()
    _check(_lib.rng_debug_stalled_waits(C.byref(c)), "rng_debug_stalled_waits")
    return c.value


def rng_debug_launch_count() -> int:
    return _lib.rng_debug_launch_count()


def rng_debug_write_ceiling(which: int, buf, stream=None):
    """which = 0: cudaMemsetAsync over buf; 1: the plain 16-byte store kernel."""
    if not buf.is_contiguous():
        raise ValueError("rng_debug_write_ceiling: buf must be contiguous")
    nbytes = buf.numel() * buf.element_size()
    with _on_device(buf):
        _check(_lib.rng_debug_write_ceiling(which, buf.data_ptr(), nbytes, _stream(stream, buf)),
               "rng_debug_write_ceiling")
    return buf


def rng_debug_eval_f64(which: int, inp, out, stream=None):
    pi, n = _ptr(inp, "f64", "in")
    po, no = _ptr(out, "f64", "out")
    if n != no:
        raise ValueError("in and out differ in length")
    if inp.device != out.device:
        raise ValueError(f"rng_debug_eval_f64: in is on {inp.device}, out on {out.device}")
    with _on_device(out):
        _check(_lib.rng_debug_eval_f64(which, pi, po, n, _stream(stream, out)), "rng_debug_eval_f64")
    return out

"""Binding of the attention block (``include/puro_attention.h``): rotary positions,
query/key norms with the rotation, attention.

Argument marshalling only, as in the package's ``__init__``.  The raw C calls keep
their names and take integer device pointers; the tensor helpers check shapes,
types and devices, allocate outputs with torch and run on the current stream (or
on ``stream``).  Head tensors are [tokens][heads][head_dim] bf16 with densely packed
heads and any distance between tokens, so that slices of a projection's output are
passed as they lie.
"""
from __future__ import annotations

import ctypes

import torch

import blockwise_fp8_gemm_act_amd as _puro

_lib = _puro._lib
_P, _I64, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float

ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3
_LAYOUTS = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED}
_SCALINGS = {"none": ROPE_PLAIN, "linear": ROPE_LINEAR, "ntk": ROPE_NTK, "yarn": ROPE_YARN}


class Rotation(ctypes.Structure):
    """puro_rotation."""
    _fields_ = [("table", _P), ("positions", _I64), ("rot", _I64), ("layout", ctypes.c_int), ("pos", _P)]


class AttentionShape(ctypes.Structure):
    """puro_attention_shape."""
    _fields_ = [(n, _I64) for n in ("q_tokens", "k_tokens", "sequences", "q_heads", "k_heads", "head_dim", "q_stride",
                                    "k_stride", "v_stride", "o_stride", "dq_stride", "dk_stride", "dv_stride", "max_k",
                                    "window", "sinks")] + [("scale", _F)]


_R, _S = ctypes.POINTER(Rotation), ctypes.POINTER(AttentionShape)
_int, _size = ctypes.c_int, ctypes.c_size_t
for _name, _args, _res in (
        ("puro_rope_table", [_I64, _I64, ctypes.c_double, _int, ctypes.c_double, _I64, _P, _P], _int),
        ("puro_rope", [_R, _int, _P, _I64, _I64, _I64, _I64, _P, _I64, _P], _int),
        ("puro_qk_norm_rope", [_R, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _F, _P, _I64, _P, _I64, _P], _int),
        ("puro_qk_norm_rope_append", [_R, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _F, _P, _I64, _P, _I64, _P, _I64, _P,
                                      _I64, _P], _int),
        ("puro_qk_norm_rope_backward_workspace_bytes", [_I64, _I64], _size),
        ("puro_qk_norm_rope_backward", [_R, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _I64, _P, _P, _F, _P, _I64,
                                        _P, _P, _P, _size, _P], _int),
        ("puro_attention_workspace_bytes", [_S], _size),
        ("puro_attention_backward_workspace_bytes", [_S], _size),
        ("puro_attention", [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _size, _P], _int),
        ("puro_attention_backward", [_S, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _size, _P], _int)):
    _fn = getattr(_lib, _name)
    _fn.argtypes, _fn.restype = _args, _res
    globals()[_name] = _fn


# ---------------------------------------------------------------- argument checks
# The handle of a device's current stream, without the torch.cuda.Stream object that
# torch.cuda.current_stream builds (3 us of a call whose kernel may take 3).
_current = torch._C._cuda_getCurrentRawStream


def _stream(stream, device):
    return _current(device.index) if stream is None else getattr(stream, "cuda_stream", stream)


def _heads_tensor(t, name, heads=None, head_dim=None, tokens=None, device=None):
    """A [tokens][heads][head_dim] bf16 CUDA tensor with packed heads; returns its token stride."""
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or not t.is_cuda or t.dim() != 3:
        raise TypeError("%s must be a bfloat16 CUDA tensor [tokens][heads][head_dim]" % name)
    n, h, d = t.shape
    if (heads is not None and h != heads) or (head_dim is not None and d != head_dim) or (tokens is not None and n != tokens):
        raise ValueError("%s must have shape %s, got %s" % (name, (tokens, heads, head_dim), tuple(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    s, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (h > 1 and sh != d):
        raise ValueError("%s must have densely packed heads" % name)
    return s if n > 1 else -(-h * d // 8) * 8          # one token's stride means nothing


def _ints(t, name, n, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_cuda:
        raise TypeError("%s must be an int32 CUDA tensor" % name)
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be contiguous with shape (%d,)" % (name, n))
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    return t.data_ptr()


def _rotation(table, pos, layout, tokens, head_dim, device):
    if not isinstance(table, torch.Tensor) or table.dtype != torch.float32 or not table.is_cuda or table.dim() != 3 \
            or table.shape[1] != 2 or not table.is_contiguous():
        raise TypeError("table must be a contiguous float32 CUDA tensor [positions][2][rot/2], as rope_table makes it")
    if table.device != device:
        raise ValueError("table is on %s, expected %s" % (table.device, device))
    if layout not in _LAYOUTS:
        raise ValueError("layout must be one of %s" % sorted(_LAYOUTS))
    return Rotation(table.data_ptr(), table.shape[0], 2 * table.shape[2], _LAYOUTS[layout], _ints(pos, "pos", tokens, device))


def _weight(w, name, head_dim, device):
    _puro._tensor(w, name, torch.bfloat16, (head_dim,), device)
    return w.data_ptr()


def _rows2d(x, name, width):
    """A 2-D bf16 CUDA tensor with contiguous rows of at least `width`; returns its row stride."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or not x.is_cuda or x.dim() != 2:
        raise TypeError("%s must be a 2-D bfloat16 CUDA tensor" % name)
    if x.shape[1] < width:
        raise ValueError("%s needs at least %d columns, got %d" % (name, width, x.shape[1]))
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    return x.stride(0) if x.shape[0] > 1 else -(-width // 8) * 8


def _out(t, name, shape, device):
    """The caller's output tensor, or a new one; and its token stride."""
    if t is None:
        t = _puro.empty(shape, dtype=torch.bfloat16, device=device)
        return t, shape[1] * shape[2]
    return t, _heads_tensor(t, name, shape[1], shape[2], shape[0], device)


# ---------------------------------------------------------------- rotary positions
@_puro._on_stream
def rope_table(positions: int, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               trained: int = 0, device="cuda", stream=None):
    """Cosines and sines of positions 0 .. positions-1 for `rot` rotated dimensions: fp32
    [positions][2][rot/2].  scaling: "none", "linear", "ntk" or "yarn" (which also reads `trained`, the
    positions of the trained context); factor: how far the context is stretched."""
    if scaling not in _SCALINGS:
        raise ValueError("scaling must be one of %s" % sorted(_SCALINGS))
    if positions < 0 or rot < 0:
        raise ValueError("positions and rot must not be negative")
    table = _puro.empty((positions, 2, rot // 2), dtype=torch.float32, device=device)
    with torch.cuda.device(table.device):
        _puro._check(_lib.puro_rope_table(positions, rot, base, _SCALINGS[scaling], factor, trained, table.data_ptr(),
                                          _stream(stream, table.device)), "puro_rope_table")
    return table


@_puro._on_stream
def rope(x, table, pos=None, layout: str = "half", inverse: bool = False, out=None, stream=None):
    """x [tokens][heads][head_dim] turned by its positions (pos int32 [tokens]; None: token t at position t).
    inverse: by the opposite angles, which is the gradient.  Returns a new tensor, or `out`."""
    xs = _heads_tensor(x, "x")
    n, h, d = x.shape
    r = _rotation(table, pos, layout, n, d, x.device)
    y, ys = _out(out, "out", (n, h, d), x.device)
    _puro._check(_lib.puro_rope(r, inverse, x.data_ptr(), xs, n, h, d, y.data_ptr(), ys, _stream(stream, x.device)),
                 "puro_rope")
    return y


# ---------------------------------------------------------------- norms and rotation
@_puro._on_stream
def qk_norm_rope(x, wq, wk, table, pos=None, *, q_heads: int, k_heads: int, eps: float = 1e-6, layout: str = "half",
                 q=None, k=None, stream=None):
    """The QKV projection's output x [tokens][>= (q_heads + k_heads) head_dim] to normed and rotated queries and
    keys: (q [tokens][q_heads][head_dim], k [tokens][k_heads][head_dim]).  head_dim is that of the weights."""
    d = wq.shape[0]
    xs = _rows2d(x, "x", (q_heads + k_heads) * d)
    n, dev = x.shape[0], x.device
    r = _rotation(table, pos, layout, n, d, dev)
    pq, pk = _weight(wq, "wq", d, dev), _weight(wk, "wk", d, dev)
    q, qs = _out(q, "q", (n, q_heads, d), dev)
    k, ks = _out(k, "k", (n, k_heads, d), dev)
    _puro._check(_lib.puro_qk_norm_rope(r, x.data_ptr(), xs, n, q_heads, k_heads, d, pq, pk, eps, q.data_ptr(), qs,
                                        k.data_ptr(), ks, _stream(stream, dev)), "puro_qk_norm_rope")
    return q, k


@_puro._on_stream
def qk_norm_rope_append(x, wq, wk, table, pos, cache_k, cache_v, rows, *, q_heads: int, eps: float = 1e-6,
                        layout: str = "half", q=None, stream=None):
    """The same for serving: keys and values of token t go into row rows[t] (int32) of cache_k and cache_v
    [rows][k_heads][head_dim]; returns the queries.  x holds q_heads query, then key, then value heads."""
    d = wq.shape[0]
    ks = _heads_tensor(cache_k, "cache_k", head_dim=d, device=x.device)
    kh = cache_k.shape[1]
    vs = _heads_tensor(cache_v, "cache_v", kh, d, cache_k.shape[0], x.device)
    xs = _rows2d(x, "x", (q_heads + 2 * kh) * d)
    n, dev = x.shape[0], x.device
    r = _rotation(table, pos, layout, n, d, dev)
    pq, pk = _weight(wq, "wq", d, dev), _weight(wk, "wk", d, dev)
    pr = _ints(rows, "rows", n, dev)
    q, qs = _out(q, "q", (n, q_heads, d), dev)
    _puro._check(_lib.puro_qk_norm_rope_append(r, x.data_ptr(), xs, n, q_heads, kh, d, pq, pk, eps, q.data_ptr(), qs,
                                               cache_k.data_ptr(), ks, cache_v.data_ptr(), vs, pr, cache_k.shape[0],
                                               _stream(stream, dev)), "puro_qk_norm_rope_append")
    return q


@_puro._on_stream
def qk_norm_rope_backward(dq, dk, x, wq, wk, table, pos=None, *, eps: float = 1e-6, layout: str = "half", dx=None,
                          workspace=None, stream=None):
    """Gradients of qk_norm_rope: (dx [tokens][q_heads + k_heads][head_dim], dwq, dwk fp32 [head_dim]).  dx may be the
    first columns of the projection output's gradient, as a [tokens][heads][head_dim] view."""
    dqs, d = _heads_tensor(dq, "dq"), dq.shape[2]
    n, qh, _ = dq.shape
    dev = dq.device
    dks = _heads_tensor(dk, "dk", head_dim=d, tokens=n, device=dev)
    kh = dk.shape[1]
    xs = _rows2d(x, "x", (qh + kh) * d)
    if x.shape[0] != n or x.device != dev:
        raise ValueError("x must have %d rows on %s" % (n, dev))
    r = _rotation(table, pos, layout, n, d, dev)
    pq, pk = _weight(wq, "wq", d, dev), _weight(wk, "wk", d, dev)
    dx, dxs = _out(dx, "dx", (n, qh + kh, d), dev)
    dw = _puro.empty((2, d), dtype=torch.float32, device=dev)
    ws = _workspace(workspace, _lib.puro_qk_norm_rope_backward_workspace_bytes(n, d), dev)
    _puro._check(_lib.puro_qk_norm_rope_backward(r, dq.data_ptr(), dqs, dk.data_ptr(), dks, x.data_ptr(), xs, n, qh, kh,
                                                 d, pq, pk, eps, dx.data_ptr(), dxs, dw.data_ptr(),
                                                 dw.data_ptr() + 4 * d, *_span(ws), _stream(stream, dev)),
                 "puro_qk_norm_rope_backward")
    return dx, dw[0], dw[1]


# ---------------------------------------------------------------- attention
def _workspace(ws, need, device):
    """The caller's workspace, or a new one where one is needed, else None.  The call holds the tensor until it has
    enqueued its kernels: only then is a released block's memory safe, as the caching allocator gives it to later work
    of the same stream."""
    if ws is None:
        return _puro.empty((need,), dtype=torch.uint8, device=device) if need else None
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous() or ws.device != device:
        raise ValueError("workspace must be a contiguous CUDA tensor on %s" % device)
    return ws


def _span(ws):
    """(pointer, bytes) of a workspace."""
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _attention_shape(q, k, v, q_start, k_start, k_len, window, sinks, scale, max_k):
    """The call's shape and the pointers of its sequences."""
    qs = _heads_tensor(q, "q")
    n, qh, d = q.shape
    dev = q.device
    ks = _heads_tensor(k, "k", head_dim=d, device=dev)
    kn, kh, _ = k.shape
    vs = _heads_tensor(v, "v", kh, d, kn, dev)
    seqs = 1
    if (q_start is None) != (k_start is None):
        raise ValueError("q_start and k_start go together")
    if q_start is not None:
        if not isinstance(q_start, torch.Tensor) or q_start.dim() != 1 or q_start.shape[0] < 2:
            raise ValueError("q_start must be a 1-D tensor of sequences + 1 starts")
        seqs = q_start.shape[0] - 1
    a = AttentionShape(n, kn, seqs, qh, kh, d, qs, ks, vs, qh * d, qh * d, kh * d, kh * d, max_k, window, sinks,
                       d ** -0.5 if scale is None else scale)
    return a, _ints(q_start, "q_start", seqs + 1, dev), _ints(k_start, "k_start", seqs + 1, dev), \
        _ints(k_len, "k_len", seqs, dev)


@_puro._on_stream
def attention(q, k, v, q_start=None, k_start=None, k_len=None, *, window: int = 0, sinks: int = 0, scale=None,
              max_k: int = 0, out=None, workspace=None, stream=None):
    """Causal attention of q [q_tokens][q_heads][head_dim] over k, v [k_tokens][k_heads][head_dim]: (o like q, lse fp32
    [q_heads][q_tokens]).

    q_start, k_start: int32 [sequences + 1] first rows of each sequence (None: one sequence).  k_len: int32 [sequences]
    keys in use of each sequence's rows (a cache).  A sequence's queries are its last positions; each sees the last
    `window` keys up to its own (0: all) and the first `sinks`.  scale: head_dim ** -0.5 unless given.  max_k: the
    longest sequence's keys, for planning only."""
    a, pqs, pks, pkl = _attention_shape(q, k, v, q_start, k_start, k_len, window, sinks, scale, max_k)
    o, a.o_stride = _out(out, "out", tuple(q.shape), q.device)
    lse = _puro.empty((a.q_heads, a.q_tokens), dtype=torch.float32, device=q.device)
    ws = _workspace(workspace, _lib.puro_attention_workspace_bytes(a), q.device)
    _puro._check(_lib.puro_attention(a, q.data_ptr(), k.data_ptr(), v.data_ptr(), pqs, pks, pkl, o.data_ptr(),
                                     lse.data_ptr(), *_span(ws), _stream(stream, q.device)), "puro_attention")
    return o, lse


@_puro._on_stream
def attention_backward(do, q, k, v, o, lse, q_start=None, k_start=None, *, window: int = 0, sinks: int = 0, scale=None,
                       dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of attention (without k_len): (dq, dk, dv), new or the caller's tensors (dv may be the value columns of
    the projection output's gradient).  o, lse: as attention returned them; do: the gradient of o."""
    a, pqs, pks, _ = _attention_shape(q, k, v, q_start, k_start, None, window, sinks, scale, 0)
    n, qh, d = q.shape
    dev = q.device
    a.o_stride = _heads_tensor(o, "o", qh, d, n, dev)
    if _heads_tensor(do, "do", qh, d, n, dev) != a.o_stride:
        raise ValueError("do must be laid out as o")
    _puro._tensor(lse, "lse", torch.float32, (qh, n), dev)
    dq, a.dq_stride = _out(dq, "dq", tuple(q.shape), dev)
    dk, a.dk_stride = _out(dk, "dk", tuple(k.shape), dev)
    dv, a.dv_stride = _out(dv, "dv", tuple(v.shape), dev)
    ws = _workspace(workspace, _lib.puro_attention_backward_workspace_bytes(a), dev)
    _puro._check(_lib.puro_attention_backward(a, do.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                              lse.data_ptr(), pqs, pks, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                              *_span(ws), _stream(stream, dev)), "puro_attention_backward")
    return dq, dk, dv

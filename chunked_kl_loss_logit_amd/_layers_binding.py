"""ctypes binding of include/kdlayers.h: the layers on the model's side of the output head.

The rules are those of _binding.py: every tensor's shape, type and device is
checked before a pointer is taken, nothing is converted, and there is no
fallback.  Calls go to the tensors' own device, on its current stream unless
one is given.
"""
from __future__ import annotations

import ctypes

import torch

from . import _policy_binding as P
from ._binding import _F32, _I32, _MASK, _matrix, _need, _one_device, _ptr, _ws_bytes, lib
from ._policy_binding import GRAD_TYPES, _choice

TYPES = tuple(GRAD_TYPES)
_I8 = (torch.int8,)
ROWS_KINDS = {"int8": 1, "e4m3": 2}
ROWS_TYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
GROUPS = (0, 32, 64, 128, 256, 512)

LAYERS_EXPORTS = (
    "kd_embedding_fwd", "kd_embedding_workspace_size", "kd_embedding_bwd", "kd_rows_quantize", "kd_rows_dequantize",
    "kd_layer_norm_fwd", "kd_layer_norm_workspace_size", "kd_layer_norm_bwd", "kd_int8_matmul_workspace_size",
    "kd_int8_matmul",
)

_llib = None


def llib() -> ctypes.CDLL:
    global _llib
    if _llib is not None:
        return _llib
    L = lib()
    i64, i32, vp, f32, f64, sz, st = (ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float, ctypes.c_double,
                                      ctypes.c_size_t, ctypes.c_int)
    psz = ctypes.POINTER(sz)
    L.kd_embedding_fwd.argtypes = [vp, vp, vp, f32, i64, i64, i64, st, i32, vp, vp]
    L.kd_embedding_workspace_size.argtypes = [i64, i64, i64, psz]
    L.kd_embedding_bwd.argtypes = [vp, vp, vp, f32, i64, i64, i64, st, st, i32, i32, vp, vp, sz, vp]
    L.kd_rows_quantize.argtypes = [vp, i64, i64, st, st, i64, vp, vp, vp]
    L.kd_rows_dequantize.argtypes = [vp, vp, i64, i64, st, i64, st, vp, vp]
    L.kd_layer_norm_fwd.argtypes = [vp, vp, vp, vp, f64, i64, i64, st, st, vp, vp, vp, st, i64, vp, vp, vp]
    L.kd_layer_norm_workspace_size.argtypes = [i64, i64, psz]
    L.kd_layer_norm_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, st, st, st, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.kd_int8_matmul_workspace_size.argtypes = [i64, i64, i64, psz]
    L.kd_int8_matmul.argtypes = [vp, vp, vp, vp, i64, i64, i64, st, vp, vp, sz, vp]
    for f in LAYERS_EXPORTS:
        getattr(L, f).restype = st
    _llib = L
    return L


def _size(fn, *args) -> int:
    llib()
    return P._size(fn, *args)


def _run(name, t, stream, *args):
    llib()
    P._run(name, t, stream, *args)


def _kind(kind, group):
    """The code of a kind of 8-bit rows; group checked."""
    code = _choice("kind", kind, ROWS_KINDS)
    if group not in GROUPS:
        raise ValueError(f"group must be one of {', '.join(map(str, GROUPS))}, got {group!r}")
    return code


def _groups(d, group):
    return -(-d // group) if group else 1


# ---------------------------------------------------------------- token embeddings
def kd_embedding_workspace_size(T, V, d) -> int:
    return _size("kd_embedding_workspace_size", T, V, d)


def _tokens(tokens, mask):
    _need("tokens", tokens, None, _I32)
    if tokens.dim() != 1:
        raise ValueError(f"tokens must be 1-D, got shape {tuple(tokens.shape)}")
    T = int(tokens.shape[0])
    _need("mask", mask, (T,), _MASK, optional=True)
    return T


def kd_embedding_fwd(tokens, table, mask, scale, tied, out, stream=None):
    """Enqueue the lookup; out [T,d] in place."""
    T = _tokens(tokens, mask)
    n, m = _matrix("table", table, None, TYPES)
    V, d = (m, n) if tied else (n, m)
    _need("out", out, (T, d), (table.dtype,))
    _one_device(tokens, table, mask, out)
    _run("kd_embedding_fwd", table, stream, _ptr(tokens), _ptr(table), _ptr(mask), float(scale), T, V, d,
         GRAD_TYPES[table.dtype], int(bool(tied)), _ptr(out))


def kd_embedding_bwd(grad, tokens, mask, scale, V, tied, accumulate, grad_table, workspace, stream=None):
    """Enqueue the gradient; grad_table ([V,d], or [d,V] if tied) in place."""
    T = _tokens(tokens, mask)
    _, d = _matrix("grad", grad, T, TYPES)
    _need("grad_table", grad_table, (d, V) if tied else (V, d), TYPES)
    nb = _ws_bytes(workspace)
    _one_device(grad, tokens, mask, grad_table, workspace)
    _run("kd_embedding_bwd", grad_table, stream, _ptr(grad), _ptr(tokens), _ptr(mask), float(scale), T, int(V), d,
         GRAD_TYPES[grad.dtype], GRAD_TYPES[grad_table.dtype], int(bool(tied)), int(bool(accumulate)),
         _ptr(grad_table), _ptr(workspace), nb)


# ---------------------------------------------------------------- rows in 8 bits
def _quantized(q, scale, group, T=None, d=None, kind=None):
    """Rows in 8 bits: q's type says of which kind.  Returns the kind, T and d."""
    n, m = _matrix("q", q, T, (ROWS_TYPES[kind],) if kind else tuple(ROWS_TYPES.values()))
    if d is not None and m != d:
        raise ValueError(f"q must have {d} columns, got shape {tuple(q.shape)}")
    kind = "int8" if q.dtype == torch.int8 else "e4m3"
    _kind(kind, group)
    _need("scale", scale, (n, _groups(m, group)), _F32)
    return kind, n, m


def kd_rows_quantize(x, kind, group, q, scale, stream=None):
    """Enqueue the rounding to 8 bits; q [T,d] and scale [T, groups] in place."""
    T, d = _matrix("x", x, None, TYPES)
    code = _kind(kind, group)
    _quantized(q, scale, group, T, d, kind)
    _one_device(x, q, scale)
    _run("kd_rows_quantize", x, stream, _ptr(x), T, d, GRAD_TYPES[x.dtype], code, int(group), _ptr(q), _ptr(scale))


def kd_rows_dequantize(q, scale, group, out, stream=None):
    kind, T, d = _quantized(q, scale, group)
    _need("out", out, (T, d), TYPES)
    _one_device(q, scale, out)
    _run("kd_rows_dequantize", out, stream, _ptr(q), _ptr(scale), T, d, ROWS_KINDS[kind], int(group),
         GRAD_TYPES[out.dtype], _ptr(out))


# ---------------------------------------------------------------- layer norm
def kd_layer_norm_workspace_size(T, d) -> int:
    return _size("kd_layer_norm_workspace_size", T, d)


def _norm_in(x, weight, bias, mask, name="x"):
    T, d = _matrix(name, x, None, TYPES)
    for n, t in (("weight", weight), ("bias", bias)):
        _need(n, t, (d,), (x.dtype, torch.float32), optional=True)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight and bias must have one type, got {weight.dtype} and {bias.dtype}")
    _need("mask", mask, (T,), _MASK, optional=True)
    return T, d


def _norm_type(x, weight, bias):
    given = weight if weight is not None else bias
    return GRAD_TYPES[x.dtype if given is None else given.dtype]


def kd_layer_norm_fwd(x, weight, bias, mask, eps, y, mean, rstd, kind=None, group=0, q=None, scale=None, stream=None):
    """Enqueue the forward; y, mean, rstd (None: not kept) and, of a kind, q and scale in place."""
    T, d = _norm_in(x, weight, bias, mask)
    _need("y", y, (T, d), (x.dtype,))
    for n, t in (("mean", mean), ("rstd", rstd)):
        _need(n, t, (T,), _F32, optional=True)
    code = 0
    if kind is not None:
        code = _kind(kind, group)
        _quantized(q, scale, group, T, d, kind)
    elif q is not None or scale is not None:
        raise ValueError("q and scale need a kind")
    _one_device(x, weight, bias, mask, y, mean, rstd, q, scale)
    _run("kd_layer_norm_fwd", x, stream, _ptr(x), _ptr(weight), _ptr(bias), _ptr(mask), float(eps), T, d,
         GRAD_TYPES[x.dtype], _norm_type(x, weight, bias), _ptr(y), _ptr(mean), _ptr(rstd), code, int(group), _ptr(q),
         _ptr(scale))


def kd_layer_norm_bwd(grad, x, weight, mask, mean, rstd, dx, dweight, dbias, workspace, group=0, q=None, scale=None,
                      stream=None):
    """Enqueue the backward; dx, dweight and dbias (None: not wanted) in place.  x, or q and scale in its place."""
    T, d = _norm_in(grad, weight, None, mask, "grad")
    code = 0
    if q is None:
        _need("x", x, (T, d), (grad.dtype,))
        if scale is not None:
            raise ValueError("scale needs q")
    else:
        if x is not None:
            raise ValueError("x must be None where q and scale stand for it")
        code = ROWS_KINDS[_quantized(q, scale, group, T, d)[0]]
    for n, t in (("mean", mean), ("rstd", rstd)):
        _need(n, t, (T,), _F32)
    _need("dx", dx, (T, d), (grad.dtype,), optional=True)
    wtypes = (grad.dtype, torch.float32) if weight is None else (weight.dtype,)
    for n, t in (("dweight", dweight), ("dbias", dbias)):
        _need(n, t, (d,), wtypes, optional=True)
    if dweight is not None and dbias is not None and dweight.dtype != dbias.dtype:
        raise TypeError(f"dweight and dbias must have one type, got {dweight.dtype} and {dbias.dtype}")
    if dx is None and dweight is None and dbias is None:
        raise ValueError("dx, dweight and dbias are all None")
    wt = next((t.dtype for t in (weight, dweight, dbias) if t is not None), grad.dtype)
    nb = _ws_bytes(workspace)
    _one_device(grad, x, weight, mask, mean, rstd, q, scale, dx, dweight, dbias, workspace)
    _run("kd_layer_norm_bwd", grad, stream, _ptr(grad), _ptr(x), _ptr(weight), _ptr(mask), _ptr(mean), _ptr(rstd), T, d,
         GRAD_TYPES[grad.dtype], GRAD_TYPES[wt], code, int(group), _ptr(q), _ptr(scale), _ptr(dx), _ptr(dweight),
         _ptr(dbias), _ptr(workspace), nb)


# ---------------------------------------------------------------- product of 8-bit integers
def kd_int8_matmul_workspace_size(T, d, V) -> int:
    return _size("kd_int8_matmul_workspace_size", T, d, V)


def _scales(name, t, n):
    """One scale a row: [n], or [n,1] as whole rows in 8 bits have them."""
    _need(name, t, None, _F32)
    if tuple(t.shape) not in ((n,), (n, 1)):
        raise ValueError(f"{name} must have shape {(n,)} or {(n, 1)}, got {tuple(t.shape)}")


def kd_int8_matmul(x, x_scale, w, w_scale, out, workspace, stream=None):
    """Enqueue the product; out [T,V] in place."""
    T, d = _matrix("x", x, None, _I8)
    V, dw = _matrix("w", w, None, _I8)
    if dw != d:
        raise ValueError(f"w must have {d} columns, got shape {tuple(w.shape)}")
    _scales("x_scale", x_scale, T)
    _scales("w_scale", w_scale, V)
    _need("out", out, (T, V), TYPES)
    nb = _ws_bytes(workspace)
    _one_device(x, x_scale, w, w_scale, out, workspace)
    _run("kd_int8_matmul", x, stream, _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), T, d, V, GRAD_TYPES[out.dtype],
         _ptr(out), _ptr(workspace), nb)

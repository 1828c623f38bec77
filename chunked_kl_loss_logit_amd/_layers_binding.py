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
from ._binding import _F32, _I32, _MASK, _check, _matrix, _need, _one_device, _ptr, _ws_bytes, lib
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
    L.kd_embedding_workspace_size.argtypes = [i64, i64, i64, i32, psz]
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


def _place(*tensors):
    """The tensors' device index and their pointers (None stays None): all on one GPU, all contiguous.  One pass, as
    small calls take no longer on the GPU than on the host."""
    index, ptrs = None, []
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        i = t.get_device()
        if i != index:
            if index is not None or i < 0:
                _one_device(*tensors)
                _ptr(t)  # not on a GPU
            index = i
        if not t.is_contiguous():
            _ptr(t)
        ptrs.append(t.data_ptr())
    return index, ptrs


_entries = {}


def _run(name, index, stream, *args):
    """Calls a library function on a device, on its current stream unless one is given."""
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(llib(), name)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != 0:
        _check(status, name)


def _kind(kind, group):
    """The code of a kind of 8-bit rows; group checked."""
    code = _choice("kind", kind, ROWS_KINDS)
    if group not in GROUPS:
        raise ValueError(f"group must be one of {', '.join(map(str, GROUPS))}, got {group!r}")
    return code


def _groups(d, group):
    return -(-d // group) if group else 1


# ---------------------------------------------------------------- token embeddings
def kd_embedding_workspace_size(T, V, d, tied=False) -> int:
    return _size("kd_embedding_workspace_size", T, V, d, int(bool(tied)))


def _tokens(tokens, mask):
    _need("tokens", tokens, None, _I32)
    if tokens.dim() != 1:
        raise ValueError(f"tokens must be 1-D, got shape {tuple(tokens.shape)}")
    T = int(tokens.shape[0])
    _need("mask", mask, (T,), _MASK, optional=True)
    return T


def _embedding_in(tokens, table, mask, tied):
    """T, V and d."""
    T = _tokens(tokens, mask)
    n, m = _matrix("table", table, None, TYPES)
    return (T, m, n) if tied else (T, n, m)


def _embedding_fwd(T, V, d, tokens, table, mask, scale, tied, out, stream=None):
    index, (tokens, src, mask, out) = _place(tokens, table, mask, out)
    _run("kd_embedding_fwd", index, stream, tokens, src, mask, float(scale), T, V, d, GRAD_TYPES[table.dtype],
         bool(tied), out)


def kd_embedding_fwd(tokens, table, mask, scale, tied, out, stream=None):
    """Enqueue the lookup; out [T,d] in place."""
    T, V, d = _embedding_in(tokens, table, mask, tied)
    _need("out", out, (T, d), (table.dtype,))
    _embedding_fwd(T, V, d, tokens, table, mask, scale, tied, out, stream)


def _embedding_bwd(T, V, d, grad, tokens, mask, scale, tied, accumulate, grad_table, workspace, stream=None):
    nb = _ws_bytes(workspace)
    index, (g, tokens, mask, out, ws) = _place(grad, tokens, mask, grad_table, workspace)
    _run("kd_embedding_bwd", index, stream, g, tokens, mask, float(scale), T, int(V), d, GRAD_TYPES[grad.dtype],
         GRAD_TYPES[grad_table.dtype], bool(tied), bool(accumulate), out, ws, nb)


def kd_embedding_bwd(grad, tokens, mask, scale, V, tied, accumulate, grad_table, workspace, stream=None):
    """Enqueue the gradient; grad_table ([V,d], or [d,V] if tied) in place."""
    T = _tokens(tokens, mask)
    _, d = _matrix("grad", grad, T, TYPES)
    _need("grad_table", grad_table, (d, V) if tied else (V, d), TYPES)
    _embedding_bwd(T, V, d, grad, tokens, mask, scale, tied, accumulate, grad_table, workspace, stream)


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


def _rows_quantize(T, d, x, code, group, q, scale, stream=None):
    index, (src, q, scale) = _place(x, q, scale)
    _run("kd_rows_quantize", index, stream, src, T, d, GRAD_TYPES[x.dtype], code, group, q, scale)


def kd_rows_quantize(x, kind, group, q, scale, stream=None):
    """Enqueue the rounding to 8 bits; q [T,d] and scale [T, groups] in place."""
    T, d = _matrix("x", x, None, TYPES)
    code = _kind(kind, group)
    _quantized(q, scale, group, T, d, kind)
    _rows_quantize(T, d, x, code, group, q, scale, stream)


def kd_rows_dequantize(q, scale, group, out, stream=None):
    kind, T, d = _quantized(q, scale, group)
    _need("out", out, (T, d), TYPES)
    index, (q, scale, to) = _place(q, scale, out)
    _run("kd_rows_dequantize", index, stream, q, scale, T, d, ROWS_KINDS[kind], group, GRAD_TYPES[out.dtype], to)


# ---------------------------------------------------------------- layer norm
def kd_layer_norm_workspace_size(T, d) -> int:
    return _size("kd_layer_norm_workspace_size", T, d)


def _norm_in(x, weight, bias, mask, name="x"):
    """T and d.  What a right call needs is looked at first, in one go; a wrong one is told what is wrong after that."""
    try:
        dtype, (T, d) = x.dtype, x.shape
        if dtype in GRAD_TYPES:
            row, wide = (d,), True
            if weight is not None:
                wide = weight.shape == row and weight.dtype in (dtype, torch.float32)
                if bias is not None:
                    wide = wide and bias.dtype == weight.dtype
            if bias is not None:
                wide = wide and bias.shape == row and bias.dtype in (dtype, torch.float32)
            if wide and (mask is None or (mask.shape == (T,) and mask.dtype in _MASK)):
                return T, d
    except (AttributeError, TypeError, ValueError):
        pass
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


def _layer_norm_fwd(T, d, x, weight, bias, mask, eps, y, mean, rstd, code=0, group=0, q=None, scale=None, stream=None):
    index, (src, w, b, mask, y, mean, rstd, q, scale) = _place(x, weight, bias, mask, y, mean, rstd, q, scale)
    _run("kd_layer_norm_fwd", index, stream, src, w, b, mask, float(eps), T, d, GRAD_TYPES[x.dtype],
         _norm_type(x, weight, bias), y, mean, rstd, code, group, q, scale)


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
    _layer_norm_fwd(T, d, x, weight, bias, mask, eps, y, mean, rstd, code, group, q, scale, stream)


def _norm_bwd_in(grad, x, weight, mask, mean, rstd, group, q, scale):
    """T, d and the code of the kind of 8-bit rows that stand for x."""
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
    return T, d, code


def _layer_norm_bwd(T, d, code, wtype, grad, x, weight, mask, mean, rstd, dx, dweight, dbias, workspace, group, q, scale,
                    stream=None):
    nb = _ws_bytes(workspace)
    index, (g, x, w, mask, mean, rstd, q, scale, dx, dw, db, ws) = _place(
        grad, x, weight, mask, mean, rstd, q, scale, dx, dweight, dbias, workspace)
    _run("kd_layer_norm_bwd", index, stream, g, x, w, mask, mean, rstd, T, d, GRAD_TYPES[grad.dtype], GRAD_TYPES[wtype],
         code, group, q, scale, dx, dw, db, ws, nb)


def kd_layer_norm_bwd(grad, x, weight, mask, mean, rstd, dx, dweight, dbias, workspace, group=0, q=None, scale=None,
                      stream=None):
    """Enqueue the backward; dx, dweight and dbias (None: not wanted) in place.  x, or q and scale in its place."""
    T, d, code = _norm_bwd_in(grad, x, weight, mask, mean, rstd, group, q, scale)
    _need("dx", dx, (T, d), (grad.dtype,), optional=True)
    wtypes = (grad.dtype, torch.float32) if weight is None else (weight.dtype,)
    for n, t in (("dweight", dweight), ("dbias", dbias)):
        _need(n, t, (d,), wtypes, optional=True)
    if dweight is not None and dbias is not None and dweight.dtype != dbias.dtype:
        raise TypeError(f"dweight and dbias must have one type, got {dweight.dtype} and {dbias.dtype}")
    if dx is None and dweight is None and dbias is None:
        raise ValueError("dx, dweight and dbias are all None")
    wtype = next((t.dtype for t in (weight, dweight, dbias) if t is not None), grad.dtype)
    _layer_norm_bwd(T, d, code, wtype, grad, x, weight, mask, mean, rstd, dx, dweight, dbias, workspace, group, q, scale,
                    stream)


# ---------------------------------------------------------------- product of 8-bit integers
def kd_int8_matmul_workspace_size(T, d, V) -> int:
    return _size("kd_int8_matmul_workspace_size", T, d, V)


def _scales(name, t, n):
    """One scale a row: [n], or [n,1] as whole rows in 8 bits have them."""
    _need(name, t, None, _F32)
    if tuple(t.shape) not in ((n,), (n, 1)):
        raise ValueError(f"{name} must have shape {(n,)} or {(n, 1)}, got {tuple(t.shape)}")


def _int8_in(x, x_scale, w, w_scale):
    """T, d and V."""
    T, d = _matrix("x", x, None, _I8)
    V, dw = _matrix("w", w, None, _I8)
    if dw != d:
        raise ValueError(f"w must have {d} columns, got shape {tuple(w.shape)}")
    _scales("x_scale", x_scale, T)
    _scales("w_scale", w_scale, V)
    return T, d, V


def _int8_matmul(T, d, V, x, x_scale, w, w_scale, out, workspace, stream=None):
    nb = _ws_bytes(workspace)
    index, (x, sx, w, sw, to, ws) = _place(x, x_scale, w, w_scale, out, workspace)
    _run("kd_int8_matmul", index, stream, x, sx, w, sw, T, d, V, GRAD_TYPES[out.dtype], to, ws, nb)


def kd_int8_matmul(x, x_scale, w, w_scale, out, workspace, stream=None):
    """Enqueue the product; out [T,V] in place."""
    T, d, V = _int8_in(x, x_scale, w, w_scale)
    _need("out", out, (T, V), TYPES)
    _int8_matmul(T, d, V, x, x_scale, w, w_scale, out, workspace, stream)

"""ctypes binding of include/kdpolicy.h: policy and preference training over the output head.

The rules are those of _binding.py: every tensor's shape, type and device is
checked before a pointer is taken, nothing is converted, and there is no
fallback.  Calls go to the tensors' own device, on its current stream unless
one is given.
"""
from __future__ import annotations

import array
import ctypes
import functools

import torch

from ._binding import (KD_BF16, KD_F32, _F32, _HEAD, _I32, _MASK, _check, _dtype_code, _matrix, _need, _one_device,
                       _ptr, _ws_bytes, lib)

KD_F16 = 2
REDUCTIONS = {"sum": 0, "token": 1, "sequence": 2}
KL_KINDS = {"k1": 1, "k2": 2, "k3": 3}
PREFERENCES = {"sigmoid": 0, "hinge": 1, "ipo": 2}
GRAD_TYPES = {torch.float32: KD_F32, torch.bfloat16: KD_BF16, torch.float16: KD_F16}
_F64 = (torch.float64,)

POLICY_EXPORTS = (
    "kd_token_logp_logits_size", "kd_token_logp_fwd_workspace_size", "kd_token_logp_workspace_size", "kd_token_logp_fwd",
    "kd_token_logp_bwd",
    "kd_token_logp_fwd_shard", "kd_token_logp_shard_combine", "kd_token_logp_bwd_shard",
    "kd_policy_loss_workspace_size", "kd_policy_loss_fwd", "kd_policy_loss_bwd", "kd_policy_loss_fwd_bwd",
    "kd_preference_loss_workspace_size", "kd_preference_loss_fwd", "kd_preference_loss_bwd",
    "kd_preference_loss_fwd_bwd",
    "kd_grad_norm_workspace_size", "kd_grad_sumsq", "kd_grad_clip", "kd_grad_clip_norm",
)


class KdPolicyOpts(ctypes.Structure):
    """kd_policy_opts of kdpolicy.h."""
    _fields_ = [("ref_logp", ctypes.c_void_p), ("entropy", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
                ("S", ctypes.c_int64), ("per_sequence", ctypes.c_int32), ("reduction", ctypes.c_int32),
                ("kl_kind", ctypes.c_int32), ("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double),
                ("dual_clip", ctypes.c_double), ("kl_weight", ctypes.c_double), ("entropy_weight", ctypes.c_double)]


class KdPrefOpts(ctypes.Structure):
    """kd_pref_opts of kdpolicy.h."""
    _fields_ = [("ref_logp", ctypes.c_void_p), ("kind", ctypes.c_int32), ("average", ctypes.c_int32),
                ("beta", ctypes.c_double), ("label_smoothing", ctypes.c_double), ("margin", ctypes.c_double)]


_plib = None


def plib() -> ctypes.CDLL:
    global _plib
    if _plib is not None:
        return _plib
    L = lib()
    i64, vp, f32, f64, sz, st = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double, ctypes.c_size_t,
                                 ctypes.c_int)
    psz, po, fo = ctypes.POINTER(sz), ctypes.POINTER(KdPolicyOpts), ctypes.POINTER(KdPrefOpts)
    L.kd_token_logp_logits_size.argtypes = [i64, i64, psz]
    L.kd_token_logp_fwd_workspace_size.argtypes = [i64, i64, i64, st, psz]
    L.kd_token_logp_workspace_size.argtypes = [i64, i64, i64, st, st, i64, psz]
    L.kd_token_logp_fwd.argtypes = [vp, vp, vp, vp, f32, i64, i64, i64, st, vp, vp, vp, vp, vp, sz, vp]
    L.kd_token_logp_bwd.argtypes = [vp, vp, vp, vp, f32, i64, i64, i64, st, vp, vp, vp, vp, vp, vp, vp, st, i64, vp, sz,
                                    vp]
    L.kd_token_logp_fwd_shard.argtypes = [vp, vp, vp, vp, f32, i64, i64, i64, i64, st, vp, vp, vp, sz, vp]
    L.kd_token_logp_shard_combine.argtypes = [vp, i64, vp, f32, i64, vp, vp, vp, vp]
    L.kd_token_logp_bwd_shard.argtypes = [vp, vp, vp, vp, f32, i64, i64, i64, i64, st, vp, vp, vp, vp, vp, vp, vp, st,
                                          i64, vp, sz, vp]
    L.kd_policy_loss_workspace_size.argtypes = [i64, i64, psz]
    L.kd_policy_loss_fwd.argtypes = [vp, vp, vp, vp, po, i64, vp, vp, vp, vp, sz, vp]
    L.kd_policy_loss_bwd.argtypes = [vp, vp, vp, vp, po, i64, vp, vp, vp, vp, vp]
    L.kd_policy_loss_fwd_bwd.argtypes = [vp, vp, vp, vp, po, i64, vp, vp, vp, vp, vp, sz, vp]
    L.kd_preference_loss_workspace_size.argtypes = [i64, i64, psz]
    L.kd_preference_loss_fwd.argtypes = [vp, vp, vp, fo, i64, i64, vp, vp, vp, vp, sz, vp]
    L.kd_preference_loss_bwd.argtypes = [vp, vp, fo, i64, i64, vp, vp, vp, vp]
    L.kd_preference_loss_fwd_bwd.argtypes = [vp, vp, vp, fo, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.kd_grad_norm_workspace_size.argtypes = [vp, i64, psz]
    L.kd_grad_sumsq.argtypes = [vp, vp, vp, i64, vp, vp, sz, vp]
    L.kd_grad_clip.argtypes = [vp, vp, vp, i64, vp, vp, vp, f64, vp, vp]
    L.kd_grad_clip_norm.argtypes = [vp, vp, vp, i64, vp, vp, f64, vp, vp, vp, sz, vp]
    for f in POLICY_EXPORTS:
        getattr(L, f).restype = st
    _plib = L
    return L


@functools.lru_cache(maxsize=1024)  # a plain function of its arguments
def _size(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(getattr(plib(), fn)(*args, ctypes.byref(out)), fn)
    return out.value


def _run(name, t, stream, *args):
    """Calls a library function on t's device, on its current stream unless one is given."""
    fn = getattr(plib(), name)
    index = t.device.index
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status != 0:
        _check(status, name)


# ---------------------------------------------------------------- token log-probabilities
def kd_token_logp_logits_size(T, V) -> int:
    return _size("kd_token_logp_logits_size", T, V)


def kd_token_logp_fwd_workspace_size(T, d, V, dtype) -> int:
    return _size("kd_token_logp_fwd_workspace_size", T, d, V, _dtype_code(dtype))


def kd_token_logp_workspace_size(T, d, V, dtype, dw_dtype=torch.float32, chunk_rows=0) -> int:
    return _size("kd_token_logp_workspace_size", T, d, V, _dtype_code(dtype), _dtype_code(dw_dtype), chunk_rows)


def _logp_in(H, W, tokens, mask, logits=None):
    T, d = _matrix("H", H, None, _HEAD)
    _, V = _matrix("W", W, d, (H.dtype,))
    _need("tokens", tokens, (T,), _I32)
    _need("mask", mask, (T,), _MASK, optional=True)
    if logits is not None:
        _need("logits", logits, (T, -(-V // 256) * 256), _F32)
    return T, d, V


def kd_token_logp_fwd(H, W, tokens, mask, tau, logp, lse, entropy, logits, workspace, stream=None):
    """Enqueue the forward; outputs logp, lse (and entropy, logits if given) in place."""
    T, d, V = _logp_in(H, W, tokens, mask, logits)
    for n, t in (("logp", logp), ("lse", lse)):
        _need(n, t, (T,), _F32)
    _need("entropy", entropy, (T,), _F32, optional=True)
    nb = _ws_bytes(workspace)
    _one_device(H, W, tokens, mask, logp, lse, entropy, logits, workspace)
    _run("kd_token_logp_fwd", H, stream, _ptr(H), _ptr(W), _ptr(tokens), _ptr(mask), float(tau), T, d, V,
         _dtype_code(H.dtype), _ptr(logp), _ptr(lse), _ptr(entropy), _ptr(logits), _ptr(workspace), nb)


def _logp_bwd_in(H, W, tokens, mask, lse, entropy, logits, grad_logp, grad_entropy, dH, dW, dh_dtype):
    T, d, V = _logp_in(H, W, tokens, mask, logits)
    _need("lse", lse, (T,), _F32)
    for n, t in (("entropy", entropy), ("grad_logp", grad_logp), ("grad_entropy", grad_entropy)):
        _need(n, t, (T,), _F32, optional=True)
    _need("dH", dH, (T, d), (dh_dtype,), optional=True)
    _need("dW", dW, (d, V), _HEAD, optional=True)
    if dH is None and dW is None:
        raise ValueError("dH and dW are both None")
    return T, d, V


def kd_token_logp_bwd(H, W, tokens, mask, tau, lse, entropy, logits, grad_logp, grad_entropy, dH, dW, chunk_rows,
                      workspace, stream=None):
    """Enqueue the backward; dH and dW (float32 or bfloat16; None: not wanted) in place."""
    T, d, V = _logp_bwd_in(H, W, tokens, mask, lse, entropy, logits, grad_logp, grad_entropy, dH, dW, H.dtype)
    nb = _ws_bytes(workspace)
    _one_device(H, W, tokens, mask, lse, entropy, logits, grad_logp, grad_entropy, dH, dW, workspace)
    _run("kd_token_logp_bwd", H, stream, _ptr(H), _ptr(W), _ptr(tokens), _ptr(mask), float(tau), T, d, V,
         _dtype_code(H.dtype), _ptr(lse), _ptr(entropy), _ptr(logits), _ptr(grad_logp), _ptr(grad_entropy), _ptr(dH),
         _ptr(dW), KD_F32 if dW is None else _dtype_code(dW.dtype), int(chunk_rows), _ptr(workspace), nb)


def kd_token_logp_fwd_shard(H, W, v0, tokens, mask, tau, rec, logits, workspace, stream=None):
    """Enqueue a vocabulary shard's forward; rec [T,4] in place."""
    T, d, V = _logp_in(H, W, tokens, mask, logits)
    _need("rec", rec, (T, 4), _F32)
    nb = _ws_bytes(workspace)
    _one_device(H, W, tokens, mask, rec, logits, workspace)
    _run("kd_token_logp_fwd_shard", H, stream, _ptr(H), _ptr(W), _ptr(tokens), _ptr(mask), float(tau), T, d, V, int(v0),
         _dtype_code(H.dtype), _ptr(rec), _ptr(logits), _ptr(workspace), nb)


def kd_token_logp_shard_combine(rec, mask, tau, logp, lse, entropy, stream=None):
    _need("rec", rec, None, _F32)
    if rec.dim() != 3 or rec.shape[2] != 4:
        raise ValueError(f"rec must be [R, T, 4], got shape {tuple(rec.shape)}")
    R, T = int(rec.shape[0]), int(rec.shape[1])
    for n, t in (("logp", logp), ("lse", lse)):
        _need(n, t, (T,), _F32)
    _need("entropy", entropy, (T,), _F32, optional=True)
    _need("mask", mask, (T,), _MASK, optional=True)
    _one_device(rec, mask, logp, lse, entropy)
    _run("kd_token_logp_shard_combine", rec, stream, _ptr(rec), R, _ptr(mask), float(tau), T, _ptr(logp), _ptr(lse),
         _ptr(entropy))


def kd_token_logp_bwd_shard(H, W, v0, tokens, mask, tau, lse, entropy, logits, grad_logp, grad_entropy, dH, dW,
                            chunk_rows, workspace, stream=None):
    """Enqueue a shard's backward; the float32 partial dH and the shard's dW in place."""
    T, d, V = _logp_bwd_in(H, W, tokens, mask, lse, entropy, logits, grad_logp, grad_entropy, dH, dW, torch.float32)
    nb = _ws_bytes(workspace)
    _one_device(H, W, tokens, mask, lse, entropy, logits, grad_logp, grad_entropy, dH, dW, workspace)
    _run("kd_token_logp_bwd_shard", H, stream, _ptr(H), _ptr(W), _ptr(tokens), _ptr(mask), float(tau), T, d, V, int(v0),
         _dtype_code(H.dtype), _ptr(lse), _ptr(entropy), _ptr(logits), _ptr(grad_logp), _ptr(grad_entropy), _ptr(dH),
         _ptr(dW), KD_F32 if dW is None else _dtype_code(dW.dtype), int(chunk_rows), _ptr(workspace), nb)


# ---------------------------------------------------------------- clipped policy loss
def _choice(name, value, table):
    if value not in table:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {value!r}")
    return table[value]


def _cu(cu_seqlens, name="cu_seqlens"):
    """cu_seqlens [S+1]; returns S."""
    _need(name, cu_seqlens, None, _I32)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError(f"{name} must be 1-D with at least two entries, got shape {tuple(cu_seqlens.shape)}")
    return int(cu_seqlens.shape[0]) - 1


class _Options:
    """What a loss's backward needs of its forward's options, without their tensors: autograd saves those, and gives
    them back where they were, unless hooks moved them in between."""

    def keep(self):
        self.places, self.tensors = _places(self.tensors), (None,) * len(self.tensors)

    def hold(self, tensors):
        """Whether the saved tensors lie where these options point to."""
        return _places(tensors) == self.places


def _places(tensors):
    return [t if t is None else (t.data_ptr(), t.numel()) for t in tensors]


class PolicyOptions(_Options):
    """The loss's parameters and optional tensors, checked once against T tokens."""

    def __init__(self, logp, old_logp, advantages, mask, ref_logp=None, entropy=None, cu_seqlens=None, clip_low=0.2,
                 clip_high=0.2, dual_clip=0.0, kl_weight=0.0, kl_kind="k3", entropy_weight=0.0, reduction="token",
                 per_sequence=None):
        _need("logp", logp, None, _F32)
        if logp.dim() != 1:
            raise ValueError(f"logp must be 1-D, got shape {tuple(logp.shape)}")
        T = self.T = int(logp.shape[0])
        S = self.S = 0 if cu_seqlens is None else _cu(cu_seqlens)
        _need("old_logp", old_logp, (T,), _F32)
        _need("advantages", advantages, None, _F32)
        if per_sequence is None:  # by its length
            if cu_seqlens is not None and S == T:
                raise ValueError("per_sequence must be given where there are as many sequences as tokens")
            per_sequence = cu_seqlens is not None and tuple(advantages.shape) == (S,)
        if per_sequence and cu_seqlens is None:
            raise ValueError("per_sequence needs cu_seqlens")
        _need("advantages", advantages, (S if per_sequence else T,))
        _need("mask", mask, (T,), _MASK, optional=True)
        _need("ref_logp", ref_logp, (T,), _F32, optional=True)
        _need("entropy", entropy, (T,), _F32, optional=True)
        self.tensors = (logp, old_logp, advantages, mask, ref_logp, entropy, cu_seqlens)
        _one_device(*self.tensors)
        self.head = tuple(_ptr(t) for t in self.tensors[:4])
        self.c = KdPolicyOpts(_ptr(ref_logp), _ptr(entropy), _ptr(cu_seqlens), S, int(bool(per_sequence)),
                              _choice("reduction", reduction, REDUCTIONS), _choice("kl_kind", kl_kind, KL_KINDS),
                              float(clip_low), float(clip_high), float(dual_clip), float(kl_weight),
                              float(entropy_weight))


def kd_policy_loss_workspace_size(T, S) -> int:
    return _size("kd_policy_loss_workspace_size", T, S)


def _policy_out(o, stats, weights, workspace=None):
    _need("stats", stats, (6,), _F32)
    _need("weights", weights, (max(o.S, 1),), _F64)
    _one_device(o.tensors[0], stats, weights, workspace)
    return _ws_bytes(workspace)


def _policy_grads(o, grad_logp, grad_entropy):
    _need("grad_logp", grad_logp, (o.T,), _F32)
    _need("grad_entropy", grad_entropy, (o.T,), _F32, optional=True)
    _one_device(o.tensors[0], grad_logp, grad_entropy)


def kd_policy_loss_fwd(o, total, stats, weights, workspace, stream=None):
    """Enqueue the forward of PolicyOptions o; total (one float32, or None), stats [6] and weights in place."""
    nb = _policy_out(o, stats, weights, workspace)
    if total is not None:
        _need("total", total, (), _F32)
        _one_device(stats, total)
    _run("kd_policy_loss_fwd", stats, stream, *o.head, ctypes.byref(o.c), o.T, _ptr(total), _ptr(stats), _ptr(weights),
         _ptr(workspace), nb)


def kd_policy_loss_bwd(o, weights, grad_total, grad_logp, grad_entropy, stream=None):
    _need("weights", weights, (max(o.S, 1),), _F64)
    _need("grad_total", grad_total, None, _F32)
    if grad_total.numel() != 1:
        raise ValueError("grad_total must have one element")
    _policy_grads(o, grad_logp, grad_entropy)
    _one_device(grad_logp, weights, grad_total)
    _run("kd_policy_loss_bwd", grad_logp, stream, *o.head, ctypes.byref(o.c), o.T, _ptr(weights), _ptr(grad_total),
         _ptr(grad_logp), _ptr(grad_entropy))


def kd_policy_loss_fwd_bwd(o, stats, weights, grad_logp, grad_entropy, workspace, stream=None):
    nb = _policy_out(o, stats, weights, workspace)
    _policy_grads(o, grad_logp, grad_entropy)
    _run("kd_policy_loss_fwd_bwd", stats, stream, *o.head, ctypes.byref(o.c), o.T, _ptr(stats), _ptr(weights),
         _ptr(grad_logp), _ptr(grad_entropy), _ptr(workspace), nb)


# ---------------------------------------------------------------- preference loss
class PreferenceOptions(_Options):
    """The loss's parameters and optional tensors, checked once."""

    def __init__(self, T, device_of, cu_seqlens, mask, ref_logp=None, beta=0.1, kind="sigmoid", label_smoothing=0.0,
                 margin=0.0, average=False):
        self.T = T
        n = _cu(cu_seqlens)
        if n % 2:
            raise ValueError(f"cu_seqlens must hold an even number of sequences (P chosen, then P rejected), got {n}")
        self.P = n // 2
        _need("mask", mask, (T,), _MASK, optional=True)
        _need("ref_logp", ref_logp, (T,), _F32, optional=True)
        self.tensors = (cu_seqlens, mask, ref_logp)
        _one_device(device_of, *self.tensors)
        self.cu, self.mask = _ptr(cu_seqlens), _ptr(mask)
        self.c = KdPrefOpts(_ptr(ref_logp), _choice("kind", kind, PREFERENCES), int(bool(average)), float(beta),
                            float(label_smoothing), float(margin))


def kd_preference_loss_workspace_size(T, P) -> int:
    return _size("kd_preference_loss_workspace_size", T, P)


def _pref_out(o, logp, loss, rewards, sums, workspace=None):
    _need("logp", logp, (o.T,), _F32)
    _need("loss", loss, (o.P,), _F32)
    _need("rewards", rewards, (2 * o.P,), _F32)
    _need("sums", sums, (2 * o.P, 2), _F64)
    _one_device(logp, loss, rewards, sums, workspace, *o.tensors)
    return _ws_bytes(workspace)


def kd_preference_loss_fwd(o, logp, loss, rewards, sums, workspace, stream=None):
    nb = _pref_out(o, logp, loss, rewards, sums, workspace)
    _run("kd_preference_loss_fwd", loss, stream, _ptr(logp), o.cu, o.mask, ctypes.byref(o.c), o.T, o.P, _ptr(loss),
         _ptr(rewards), _ptr(sums), _ptr(workspace), nb)


def _pref_grad(o, sums, grad_loss, grad_logp):
    _need("sums", sums, (2 * o.P, 2), _F64)
    _need("grad_loss", grad_loss, (o.P,), _F32)
    _need("grad_logp", grad_logp, (o.T,), _F32)
    _one_device(sums, grad_loss, grad_logp, *o.tensors)


def kd_preference_loss_bwd(o, sums, grad_loss, grad_logp, stream=None):
    _pref_grad(o, sums, grad_loss, grad_logp)
    _run("kd_preference_loss_bwd", grad_logp, stream, o.cu, o.mask, ctypes.byref(o.c), o.T, o.P, _ptr(sums),
         _ptr(grad_loss), _ptr(grad_logp))


def kd_preference_loss_fwd_bwd(o, logp, grad_loss, loss, rewards, sums, grad_logp, workspace, stream=None):
    nb = _pref_out(o, logp, loss, rewards, sums, workspace)
    _pref_grad(o, sums, grad_loss, grad_logp)
    _run("kd_preference_loss_fwd_bwd", loss, stream, _ptr(logp), o.cu, o.mask, ctypes.byref(o.c), o.T, o.P,
         _ptr(grad_loss), _ptr(loss), _ptr(rewards), _ptr(sums), _ptr(grad_logp), _ptr(workspace), nb)


# ---------------------------------------------------------------- gradient norm and clipping
def _dense(t):
    """Whether t's elements fill its memory without gaps or overlap, in any order of its axes."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != want:
            return False
        want *= n
    return True


def _writable(name, tensors):
    """Refuses what a write past autograd would falsify: parameters (it is their gradients that are clipped), and in
    grad mode every tensor that autograd follows."""
    for t in tensors:
        if t.requires_grad and (t.is_leaf or torch.is_grad_enabled()):
            raise ValueError(f"{name} must not require a gradient where they are written to: pass the parameters' .grad "
                             "(a tensor whose own values are meant: its .detach())")


class TensorTable:
    """Host arrays of pointers, element counts and types of a list of tensors on one device.  One pass per attribute:
    a few hundred tensors are checked in less time than their kernels take.  written: they are to be written to."""

    def __init__(self, name, tensors, written=False):
        try:
            types = [GRAD_TYPES[t.dtype] for t in tensors]
        except (KeyError, AttributeError):
            for t in tensors:
                if not isinstance(t, torch.Tensor):
                    raise TypeError(f"{name} must hold torch.Tensors, got {type(t).__name__}") from None
                if t.dtype not in GRAD_TYPES:
                    raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}") from None
            raise
        if written and any([t.requires_grad for t in tensors]):
            _writable(name, tensors)
        devices = {t.get_device() for t in tensors}
        if -1 in devices:
            raise ValueError("libkdloss tensors must be on the GPU")
        if len(devices) > 1:
            _one_device(*tensors)
        self.contiguous = all([t.is_contiguous() for t in tensors])
        if not self.contiguous:
            for t in tensors:
                if not _dense(t):
                    raise ValueError(f"{name} must be dense in memory, got shape {tuple(t.shape)} with strides {t.stride()}")
        self.n = len(tensors)
        self.tensors = tensors
        self._arrays = (array.array("Q", [t.data_ptr() for t in tensors]),
                        array.array("q", [t.numel() for t in tensors]), array.array("i", types))
        self.ptrs, self.numel, self.types = (a.buffer_info()[0] for a in self._arrays)

    def same_layout(self, other):
        """Whether the two tables' tensors pair up element by element in memory."""
        if self._arrays[1] != other._arrays[1]:
            return False
        if self.contiguous and other.contiguous:
            return True
        return all(t.shape == o.shape and t.stride() == o.stride() for t, o in zip(self.tensors, other.tensors))


def kd_grad_norm_workspace_size(table) -> int:
    out = ctypes.c_size_t(0)
    _check(plib().kd_grad_norm_workspace_size(table.numel, table.n, ctypes.byref(out)), "kd_grad_norm_workspace_size")
    return out.value


def kd_grad_sumsq(table, sumsq, workspace, stream=None):
    """Enqueue the sum of squares of a TensorTable; sumsq (one float64) in place."""
    _need("sumsq", sumsq, (1,), _F64)
    _one_device(sumsq, workspace, *table.tensors[:1])
    _run("kd_grad_sumsq", sumsq, stream, table.ptrs, table.numel, table.types, table.n, _ptr(sumsq), _ptr(workspace),
         _ws_bytes(workspace))


def _clip_in(table, outs, sumsq, norm):
    _need("sumsq", sumsq, (1,), _F64)
    _need("norm", norm, (), _F32)
    if outs is not table and not table.same_layout(outs):
        raise ValueError("out must match the tensors' number, sizes and strides")
    _one_device(sumsq, norm, *table.tensors[:1], *outs.tensors[:1])


def _written(outs):
    """Tells autograd that the tensors changed: tensors saved for a backward pass are refused there, not used."""
    torch.autograd.graph.increment_version(outs.tensors)


def kd_grad_clip(table, outs, sumsq, max_norm, norm, stream=None):
    """Enqueue the scaling of a TensorTable into another (or itself); norm (one float32) in place."""
    _clip_in(table, outs, sumsq, norm)
    _run("kd_grad_clip", sumsq, stream, table.ptrs, table.numel, table.types, table.n, outs.ptrs, outs.types, _ptr(sumsq),
         float(max_norm), _ptr(norm))
    _written(outs)


def kd_grad_clip_norm(table, outs, max_norm, sumsq, norm, workspace, stream=None):
    """Enqueue the sum of squares and the scaling; sumsq and norm in place."""
    _clip_in(table, outs, sumsq, norm)
    _one_device(sumsq, workspace)
    _run("kd_grad_clip_norm", sumsq, stream, table.ptrs, table.numel, table.types, table.n, outs.ptrs, outs.types,
         float(max_norm), _ptr(sumsq), _ptr(norm), _ptr(workspace), _ws_bytes(workspace))
    _written(outs)

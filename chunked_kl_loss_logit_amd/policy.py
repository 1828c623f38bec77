"""Policy and preference training over the output head (include/kdpolicy.h).

    logp, ent = token_logp(H, W, tokens, mask, want_entropy=True)      # autograd, through the head
    loss, stats = policy_loss(logp, old_logp, advantages, mask, entropy=ent, entropy_weight=0.01)
    loss.backward()
    norm = clip_grad_norm_([H.grad, W.grad], 1.0)

    loss, rewards = preference_loss(logp, cu_seqlens, mask, ref_logp=ref)   # P pairs, autograd

In a captured graph the _forward and _backward functions are the safe form:
torch ends the process where a backward of its autograd is captured while an
uncaptured graph of the same leaves is alive, whatever functions are in it.

As for the distillation losses, all arithmetic runs in the HIP kernels of
libkdloss.so; this module allocates outputs and workspaces with torch.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _policy_binding as B


def _workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _f32(like, *shape):
    return torch.empty(*shape, dtype=torch.float32, device=like.device)


def _grad(g):
    """An upstream gradient as the kernels take it."""
    return None if g is None else g.float().contiguous()


# ---------------------------------------------------------------- token log-probabilities
def token_logp_forward(H, W, tokens, mask=None, tau=1.0, want_entropy=False, keep_logits=False, workspace=None):
    """logp [T], lse [T], entropy [T] (or None) and, with keep_logits, the logits that spare the backward its
    projection (T x roundup(V, 256) float32; else None)."""
    T, d, V = B._logp_in(H, W, tokens, mask)
    logp, lse = _f32(H, T), _f32(H, T)
    entropy = _f32(H, T) if want_entropy else None
    logits = _f32(H, T, -(-V // 256) * 256) if keep_logits else None
    if workspace is None:
        workspace = _workspace(B.kd_token_logp_fwd_workspace_size(T, d, V, H.dtype), H.device)
    B.kd_token_logp_fwd(H, W, tokens, mask, tau, logp, lse, entropy, logits, workspace)
    return logp, lse, entropy, logits


def token_logp_backward(H, W, tokens, mask, tau, lse, grad_logp, entropy=None, grad_entropy=None, logits=None,
                        chunk_rows=0, dw_dtype=torch.float32, workspace=None, want=(True, True)):
    """dH (dtype of H) and dW (dw_dtype) for the upstream gradients of logp and of the entropy (either may be None).
    want: whether dH and dW are wanted; the other is None and costs nothing."""
    T, d, V = B._logp_in(H, W, tokens, mask)
    dH = torch.empty_like(H) if want[0] else None
    dW = torch.empty(d, V, dtype=dw_dtype, device=H.device) if want[1] else None
    if workspace is None:
        workspace = _workspace(B.kd_token_logp_workspace_size(T, d, V, H.dtype, dw_dtype, chunk_rows), H.device)
    B.kd_token_logp_bwd(H, W, tokens, mask, tau, lse, entropy, logits, _grad(grad_logp), _grad(grad_entropy), dH, dW,
                        chunk_rows, workspace)
    return dH, dW


def token_logp_shard_forward(H, W_shard, v0, tokens, mask=None, tau=1.0, keep_logits=False, workspace=None):
    """A vocabulary shard's records rec [T,4] (and its logits, or None): W_shard holds columns [v0, v0 + V) of the
    head, tokens are indices into all of it.  The caller all-gathers the records."""
    T, d, V = B._logp_in(H, W_shard, tokens, mask)
    rec = _f32(H, T, 4)
    logits = _f32(H, T, -(-V // 256) * 256) if keep_logits else None
    if workspace is None:
        workspace = _workspace(B.kd_token_logp_fwd_workspace_size(T, d, V, H.dtype), H.device)
    B.kd_token_logp_fwd_shard(H, W_shard, v0, tokens, mask, tau, rec, logits, workspace)
    return rec, logits


def token_logp_shard_combine(recs, mask=None, tau=1.0, want_entropy=False):
    """logp, lse and entropy (or None) of the whole head from the shards' records (a list in rank order, or [R,T,4])."""
    rec = recs if isinstance(recs, torch.Tensor) else torch.stack(list(recs))
    T = rec.shape[1]
    logp, lse = _f32(rec, T), _f32(rec, T)
    entropy = _f32(rec, T) if want_entropy else None
    B.kd_token_logp_shard_combine(rec.contiguous(), mask, tau, logp, lse, entropy)
    return logp, lse, entropy


def token_logp_shard_backward(H, W_shard, v0, tokens, mask, tau, lse, grad_logp, entropy=None, grad_entropy=None,
                              logits=None, chunk_rows=0, dw_dtype=torch.float32, workspace=None, want=(True, True)):
    """This shard's dH partial [T,d] float32 (the caller sums them over the ranks) and its columns of dW; want as for
    token_logp_backward."""
    T, d, V = B._logp_in(H, W_shard, tokens, mask)
    dH = _f32(H, T, d) if want[0] else None
    dW = torch.empty(d, V, dtype=dw_dtype, device=H.device) if want[1] else None
    if workspace is None:
        workspace = _workspace(B.kd_token_logp_workspace_size(T, d, V, H.dtype, dw_dtype, chunk_rows), H.device)
    B.kd_token_logp_bwd_shard(H, W_shard, v0, tokens, mask, tau, lse, entropy, logits, _grad(grad_logp),
                              _grad(grad_entropy), dH, dW, chunk_rows, workspace)
    return dH, dW


class _TokenLogp(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, tokens, mask, tau, want_entropy, keep_logits, chunk_rows):
        keep = keep_logits and any(ctx.needs_input_grad[:2])
        logp, lse, entropy, logits = token_logp_forward(H, W, tokens, mask, tau, want_entropy, keep)
        ctx.save_for_backward(H, W, tokens, mask, lse, entropy, logits)
        ctx.tau, ctx.chunk_rows = tau, chunk_rows
        ctx.set_materialize_grads(False)
        return (logp, entropy) if want_entropy else logp

    @staticmethod
    @once_differentiable
    def backward(ctx, g, ge=None):
        H, W, tokens, mask, lse, entropy, logits = ctx.saved_tensors
        if g is None and ge is None:
            return (None,) * 8
        dH, dW = token_logp_backward(H, W, tokens, mask, ctx.tau, lse, g, entropy, ge, logits, ctx.chunk_rows, W.dtype,
                                     want=ctx.needs_input_grad[:2])
        return dH, dW, None, None, None, None, None, None


def token_logp(H, W, tokens, mask=None, tau=1.0, want_entropy=False, keep_logits=False, chunk_rows=0):
    """Log-probability of tokens [T] under softmax(H.W / tau), 0 on masked rows (and with want_entropy each row's
    entropy); differentiable in H and W, whose gradients have their dtypes.  keep_logits holds the logits for the
    backward instead of computing the projection again."""
    return _TokenLogp.apply(H, W, tokens, mask, float(tau), bool(want_entropy), bool(keep_logits), int(chunk_rows))


# ---------------------------------------------------------------- clipped policy loss
# Options of the functions below (kd_policy_opts of kdpolicy.h): ref_logp [T] with kl_weight and kl_kind "k1", "k2" or
# "k3"; entropy [T] with entropy_weight; cu_seqlens [S+1]; clip_low, clip_high; dual_clip (0 = none); reduction "sum",
# "token" or "sequence".  advantages is [T], or [S] for one per sequence: told by its length, or by per_sequence (which
# has to be given where S = T).
def _policy_forward(o, grads, workspace, total=None):
    like = o.tensors[0]
    stats = _f32(like, 6)
    weights = torch.empty(max(o.S, 1), dtype=torch.float64, device=like.device)
    if workspace is None:
        workspace = _workspace(B.kd_policy_loss_workspace_size(o.T, o.S), like.device)
    if not grads:
        B.kd_policy_loss_fwd(o, total, stats, weights, workspace)
        return stats, weights, None, None
    g = _f32(like, o.T)
    ge = _f32(like, o.T) if o.tensors[5] is not None else None
    B.kd_policy_loss_fwd_bwd(o, stats, weights, g, ge, workspace)
    return stats, weights, g, ge


def policy_loss_forward(logp, old_logp, advantages, mask=None, workspace=None, **options):
    """stats [6] (total, policy, kl, entropy, clipped share, valid tokens) and the weights the backward takes."""
    o = B.PolicyOptions(logp, old_logp, advantages, mask, **options)
    stats, weights, _, _ = _policy_forward(o, False, workspace)
    return stats, weights


def _policy_backward(o, weights, grad_total):
    g = _f32(weights, o.T)
    ge = _f32(weights, o.T) if o.c.entropy is not None else None
    B.kd_policy_loss_bwd(o, weights, _grad(grad_total), g, ge)
    return g, ge


def policy_loss_backward(logp, old_logp, advantages, mask, weights, grad_total, **options):
    """grad_logp [T] and, with an entropy, grad_entropy [T] (else None) for the total's upstream gradient."""
    return _policy_backward(B.PolicyOptions(logp, old_logp, advantages, mask, **options), weights, grad_total)


def policy_loss_forward_backward(logp, old_logp, advantages, mask=None, workspace=None, **options):
    """stats [6], grad_logp [T] and grad_entropy [T] (or None) in one call, for an upstream gradient of 1."""
    o = B.PolicyOptions(logp, old_logp, advantages, mask, **options)
    stats, _, g, ge = _policy_forward(o, True, workspace)
    return stats, g, ge


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, entropy, old_logp, advantages, mask, ref_logp, cu_seqlens, options):
        o = B.PolicyOptions(logp, old_logp, advantages, mask, entropy=entropy, ref_logp=ref_logp,
                            cu_seqlens=cu_seqlens, **options)
        total = _f32(logp, ())  # a tensor of its own: a view of stats could not be changed in place by its user
        stats, weights, _, _ = _policy_forward(o, False, None, total)
        ctx.save_for_backward(*o.tensors, weights)
        o.keep()
        ctx.o, ctx.options = o, options
        ctx.mark_non_differentiable(stats)
        ctx.set_materialize_grads(False)
        return total, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        if g is None:
            return (None,) * 8
        *tensors, weights = ctx.saved_tensors  # refuses tensors changed in place since
        o = ctx.o
        if not o.hold(tensors):
            logp, old_logp, advantages, mask, ref_logp, entropy, cu_seqlens = tensors
            o = B.PolicyOptions(logp, old_logp, advantages, mask, ref_logp, entropy, cu_seqlens, **ctx.options)
        gl, ge = _policy_backward(o, weights, g)
        return gl, ge, None, None, None, None, None, None


def policy_loss(logp, old_logp, advantages, mask=None, ref_logp=None, entropy=None, cu_seqlens=None, **options):
    """The clipped policy loss (a scalar, differentiable in logp and entropy) and stats [6]."""
    return _PolicyLoss.apply(logp, entropy, old_logp, advantages, mask, ref_logp, cu_seqlens, options)


# ---------------------------------------------------------------- preference loss
# Options (kd_pref_opts of kdpolicy.h): ref_logp [T] (None: no reference), beta, kind "sigmoid", "hinge" or "ipo",
# label_smoothing (sigmoid), margin (not ipo), average.  cu_seqlens [2P+1]: P chosen sequences, then the P rejected.
def _pref_in(logp, cu_seqlens, mask, options):
    B._need("logp", logp, None, B._F32)
    if logp.dim() != 1:
        raise ValueError(f"logp must be 1-D, got shape {tuple(logp.shape)}")
    return B.PreferenceOptions(int(logp.shape[0]), logp, cu_seqlens, mask, **options)


def _pref_out(logp, o, workspace):
    if workspace is None:
        workspace = _workspace(B.kd_preference_loss_workspace_size(o.T, o.P), logp.device)
    return (_f32(logp, o.P), _f32(logp, 2 * o.P), torch.empty(2 * o.P, 2, dtype=torch.float64, device=logp.device),
            workspace)


def _pref_forward(o, logp, workspace):
    loss, rewards, sums, workspace = _pref_out(logp, o, workspace)
    B.kd_preference_loss_fwd(o, logp, loss, rewards, sums, workspace)
    return loss, rewards, sums


def _pref_backward(o, sums, grad_loss):
    g = _f32(sums, o.T)
    B.kd_preference_loss_bwd(o, sums, _grad(grad_loss), g)
    return g


def preference_loss_forward(logp, cu_seqlens, mask=None, workspace=None, **options):
    """loss [P], rewards [2P] and the sums the backward takes."""
    return _pref_forward(_pref_in(logp, cu_seqlens, mask, options), logp, workspace)


def preference_loss_backward(T, cu_seqlens, mask, sums, grad_loss, **options):
    """grad_logp [T] for the upstream gradient of the pair losses."""
    return _pref_backward(B.PreferenceOptions(int(T), sums, cu_seqlens, mask, **options), sums, grad_loss)


def preference_loss_forward_backward(logp, cu_seqlens, mask, grad_loss, workspace=None, **options):
    """loss [P], rewards [2P] and grad_logp [T] in one call, for a known upstream gradient [P]."""
    o = _pref_in(logp, cu_seqlens, mask, options)
    loss, rewards, sums, workspace = _pref_out(logp, o, workspace)
    g = _f32(logp, o.T)
    B.kd_preference_loss_fwd_bwd(o, logp, _grad(grad_loss), loss, rewards, sums, g, workspace)
    return loss, rewards, g


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, cu_seqlens, mask, ref_logp, options):
        o = _pref_in(logp, cu_seqlens, mask, dict(options, ref_logp=ref_logp))
        loss, rewards, sums = _pref_forward(o, logp, None)
        ctx.save_for_backward(*o.tensors, sums)
        o.keep()
        ctx.o, ctx.options = o, options
        ctx.mark_non_differentiable(rewards)
        ctx.set_materialize_grads(False)
        return loss, rewards

    @staticmethod
    @once_differentiable
    def backward(ctx, g, _):
        if g is None:
            return (None,) * 5
        *tensors, sums = ctx.saved_tensors  # refuses tensors changed in place since
        o = ctx.o
        if not o.hold(tensors):
            cu_seqlens, mask, ref_logp = tensors
            o = B.PreferenceOptions(o.T, sums, cu_seqlens, mask, ref_logp, **ctx.options)
        return _pref_backward(o, sums, g), None, None, None, None


def preference_loss(logp, cu_seqlens, mask=None, ref_logp=None, **options):
    """Per-pair preference loss [P] (differentiable in logp) and the sequences' rewards [2P]."""
    return _PreferenceLoss.apply(logp, cu_seqlens, mask, ref_logp, options)


# ---------------------------------------------------------------- gradient norm and clipping
def _tensors(tensors):
    tensors = [tensors] if isinstance(tensors, torch.Tensor) else [t for t in tensors if t is not None]
    if not tensors:
        raise ValueError("no tensors")
    return tensors


def grad_sumsq(tensors):
    """The sum of all elements' squares, [1] float64 on the device: what ranks that hold parts of the gradients add up
    before clip_grad_norm(..., sumsq=...)."""
    table = B.TensorTable("tensors", _tensors(tensors))
    device = table.tensors[0].device
    sumsq = torch.empty(1, dtype=torch.float64, device=device)
    B.kd_grad_sumsq(table, sumsq, _workspace(B.kd_grad_norm_workspace_size(table), device))
    return sumsq


def clip_grad_norm(tensors, max_norm, out=None, sumsq=None):
    """Writes tensors[i] * min(1, max_norm / (norm + 1e-6)) to out[i] (the same number of elements in the same order
    in memory; float32, bfloat16 or float16) and returns the global L2 norm, one float32 on the device.  out = None: in
    place, and None entries among the tensors are left out.  sumsq: the squared norm, if it is not that of these
    tensors alone.  The tensors are the gradients themselves: what is written to may not be a parameter (a leaf that
    requires a gradient), nor in grad mode any tensor that requires one."""
    if not isinstance(tensors, torch.Tensor):
        tensors = list(tensors)
    kept = _tensors(tensors)
    table = outs = B.TensorTable("tensors", kept, written=out is None)
    if out is not None:
        outs = B.TensorTable("out", [out] if isinstance(out, torch.Tensor) else list(out), written=True)
        if not isinstance(tensors, torch.Tensor) and len(kept) != len(tensors):
            raise ValueError("with out, no tensor may be None")
    device = kept[0].device
    norm = torch.empty((), dtype=torch.float32, device=device)
    if sumsq is not None:
        B.kd_grad_clip(table, outs, sumsq, max_norm, norm)
    else:
        B.kd_grad_clip_norm(table, outs, max_norm, torch.empty(1, dtype=torch.float64, device=device), norm,
                            _workspace(B.kd_grad_norm_workspace_size(table), device))
    return norm


def clip_grad_norm_(tensors, max_norm, sumsq=None):
    """clip_grad_norm in place, on the gradients (p.grad), not on the parameters that have them."""
    return clip_grad_norm(tensors, max_norm, None, sumsq)

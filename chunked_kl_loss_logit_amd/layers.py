"""The layers on the model's side of the output head (include/kdlayers.h).

    X = embedding(tokens, E, mask, scale)                  # or embedding(tokens, W, ..., tied=True): W [d,V], the head
    H = layer_norm(X, weight, bias, mask)                  # autograd; checkpoint="int8" keeps X in 8 bits
    logp = token_logp(H, W, tokens, mask)                  # any loss over the head

    y = checkpoint_8bit(block, x)                          # keeps x in 8 bits, runs block again in the backward pass

    q, scale = quantize_rows(H, "int8", 0)                 # one scale a row
    Z = int8_matmul(q, scale, wq, w_scale)                 # logits through a frozen 8-bit head

In a captured graph the _forward and _backward functions are the safe form:
torch ends the process where a backward of its autograd is captured while an
uncaptured graph of the same leaves is alive, whatever functions are in it.

All arithmetic runs in the HIP kernels of libkdloss.so; this module allocates
outputs and workspaces with torch.
"""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.function import once_differentiable
from torch.utils._python_dispatch import TorchDispatchMode

from . import _layers_binding as B
from .policy import _f32, _workspace


# ---------------------------------------------------------------- token embeddings
def embedding_forward(tokens, table, mask=None, scale=1.0, tied=False):
    """scale * table[tokens] [T,d] in the table's type: rows of table [V,d], or with tied the columns of the head
    W [d,V].  Masked rows are 0; a valid token outside the vocabulary gives a row of NaN."""
    T, V, d = B._embedding_in(tokens, table, mask, tied)
    out = torch.empty(T, d, dtype=table.dtype, device=table.device)
    B._embedding_fwd(T, V, d, tokens, table, mask, scale, tied, out)
    return out


def embedding_backward(grad, tokens, V, mask=None, scale=1.0, tied=False, grad_dtype=None, out=None, workspace=None):
    """The table's gradient [V,d] (or [d,V] if tied) of grad_dtype (None: grad's).  out: a tensor that takes it on
    top of what it holds and is returned, such as the gradient of the head that the embedding shares."""
    T = B._tokens(tokens, mask)
    _, d = B._matrix("grad", grad, T, B.TYPES)
    shape = (d, V) if tied else (V, d)
    if out is None:
        dtype = grad_dtype or grad.dtype
        if dtype not in B.TYPES:
            raise TypeError(f"grad_dtype must be one of {', '.join(map(str, B.TYPES))}, got {dtype}")
        table = torch.empty(shape, dtype=dtype, device=grad.device)
    else:
        B._need("out", out, shape, B.TYPES if grad_dtype is None else (grad_dtype,))
        B.P._writable("out", [out])
        table = out
    if workspace is None:
        workspace = _workspace(B.kd_embedding_workspace_size(T, V, d, tied), grad.device)
    B._embedding_bwd(T, V, d, grad, tokens, mask, scale, tied, out is not None, table, workspace)
    if out is not None:
        torch.autograd.graph.increment_version([out])
    return table


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, mask, scale, tied):
        out = embedding_forward(tokens, table, mask, scale, tied)
        ctx.save_for_backward(tokens, mask)
        ctx.V, ctx.scale, ctx.tied = table.shape[1 if tied else 0], scale, tied
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        tokens, mask = ctx.saved_tensors
        return (embedding_backward(g.contiguous(), tokens, ctx.V, mask, ctx.scale, ctx.tied), None, None, None, None)


def embedding(tokens, table, mask=None, scale=1.0, tied=False):
    """embedding_forward, differentiable in the table; its gradient has its type and layout."""
    return _Embedding.apply(table, tokens, mask, float(scale), bool(tied))


# ---------------------------------------------------------------- rows in 8 bits
def quantize_rows(x, kind="int8", group=0):
    """x [T,d] in 8 bits: q [T,d] (int8, or float8_e4m3fn for kind "e4m3") and scale [T, groups] float32, for groups
    of 32, 64, 128, 256 or 512 values of a row, or of whole rows (0)."""
    T, d = B._matrix("x", x, None, B.TYPES)
    code = B._kind(kind, group)
    q = torch.empty(T, d, dtype=B.ROWS_TYPES[kind], device=x.device)
    scale = _f32(x, T, B._groups(d, group))
    B._rows_quantize(T, d, x, code, group, q, scale)
    return q, scale


def dequantize_rows(q, scale, group=0, dtype=torch.bfloat16):
    """What rows in 8 bits stand for, rounded to dtype."""
    out = torch.empty(q.shape, dtype=dtype, device=q.device)
    B.kd_rows_dequantize(q, scale, group, out)
    return out


def _rows(x):
    return x.detach().contiguous().reshape(-1, x.shape[-1])


def _capturing():
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


class _NoDraws(TorchDispatchMode):
    """Refuses operations that draw random numbers."""

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        kwargs = kwargs or {}
        if torch.Tag.nondeterministic_seeded in func.tags:
            names = func._schema.arguments
            given = {a.name: a.default_value for a in names} | dict(zip((a.name for a in names), args)) | kwargs
            if given.get("dropout_p") != 0:  # (attention draws nothing then)
                raise RuntimeError(f"fn must not draw random numbers ({func}) in a captured graph: its random states can be "
                                   "neither read nor set, and the backward pass has to draw the same ones")
        return func(*args, **kwargs)


class _Surroundings:
    """What fn's result hangs on beside its arguments, as it is before the forward pass: autocast and the random
    states."""

    def __init__(self, x, others):
        self.autocast = [self._autocast(d) for d in {x.device.type, "cpu"}]
        self.states = [] if _capturing() else self._states(
            [torch.default_generator, *(torch.cuda.default_generators if torch.cuda.is_initialized() else ()),
             *(g for g in others if isinstance(g, torch.Generator))])

    @staticmethod
    def _autocast(device_type):
        return dict(device_type=device_type, dtype=torch.get_autocast_dtype(device_type),
                    enabled=torch.is_autocast_enabled(device_type), cache_enabled=torch.is_autocast_cache_enabled())

    @staticmethod
    def _states(generators):
        return [(g, g.get_state()) for g in generators]

    @staticmethod
    def _set(states):
        for g, state in states:
            g.set_state(state)

    @staticmethod
    @contextlib.contextmanager
    def first():
        try:
            with _NoDraws() if _capturing() else contextlib.nullcontext():
                yield
        finally:  # casts that autocast remembers from here, where nothing is recorded, would have no gradient elsewhere
            torch.clear_autocast_cache()

    @contextlib.contextmanager
    def again(self):
        """As it was then; afterwards as it is now."""
        with contextlib.ExitStack() as stack:
            for settings in self.autocast:
                if settings != self._autocast(settings["device_type"]):
                    stack.enter_context(torch.autocast(**settings))
            if _capturing():
                stack.enter_context(_NoDraws())
            else:
                stack.callback(self._set, self._states([g for g, _ in self.states]))
                self._set(self.states)
            yield


def _graph(nodes):
    """The nodes that lie behind some of autograd's."""
    stack, seen = list(nodes), set()
    while stack:
        node = stack.pop()
        if node is not None and node not in seen:
            seen.add(node)
            stack += [n for n, _ in node.next_functions]
    return seen


def _runs(node):
    """Whether the running backward pass comes to a node; None if torch.autograd.grad asks for that leaf's gradient."""
    try:
        return torch._C._will_engine_execute_node(node)
    except RuntimeError:
        return None


def _check_asked(ctx, out, own):
    """Under torch.autograd.grad and backward(inputs=...): fn's tensors from elsewhere must not be among those asked for,
    whose gradients would lack fn's share."""
    leaf = "torch::autograd::AccumulateGrad"
    edge = torch.autograd.graph.get_gradient_edge
    nodes = _graph(edge(o).node for o in out) - {edge(t).node for t in own}
    asked = any(_runs(n) is not False for n in nodes)
    if not asked and any(n.name() == leaf for n in nodes):
        # backward(inputs=...) does not say which leaves it is for unless its own graph leads to them
        asked = any(n.name() == leaf and _runs(n) for n in _graph([ctx]))
    if asked:
        raise RuntimeError("fn takes a tensor from elsewhere whose gradient may be asked for: torch.autograd.grad and "
                           "backward(inputs=...) reach x and the others alone, so it has to be among the others")


class _Checkpoint(torch.autograd.Function):
    @staticmethod
    def forward(ctx, fn, kind, group, form, x, *others):
        before = [t._version for t in (x, *others) if isinstance(t, torch.Tensor)]
        ctx.surroundings = _Surroundings(x, others)
        with ctx.surroundings.first():
            out = fn(x, *others)
        if before != [t._version for t in (x, *others) if isinstance(t, torch.Tensor)]:
            raise RuntimeError("fn must not change its arguments in place: the backward pass runs it again on them")
        if isinstance(out, (tuple, list)):
            form.append(tuple if isinstance(out, list) else getattr(out, "_make", type(out)))
            out = tuple(out)
        for o in out if form else (out,):
            if not isinstance(o, (torch.Tensor, int, float, complex, str, type(None))):  # whose tensors would have no gradient
                raise TypeError(f"fn must return a tensor, or a tuple or list of them, got a {type(o).__name__} in its place")
        # a tensor from elsewhere must not become this function's output itself
        given = [t for t in (x, *others) if isinstance(t, torch.Tensor)]
        own = [o.detach() if isinstance(o, torch.Tensor) and not any(o is t for t in given) else o
               for o in (out if form else (out,))]
        q, scale = quantize_rows(_rows(x), kind, group)
        tensors = [t if isinstance(t, torch.Tensor) else None for t in others]
        ctx.save_for_backward(q, scale, *tensors)
        ctx.fn, ctx.group, ctx.shape, ctx.dtype = fn, group, x.shape, x.dtype
        ctx.plain = [None if isinstance(t, torch.Tensor) else t for t in others]
        ctx.set_materialize_grads(False)
        return tuple(own) if form else own[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        q, scale, *others = ctx.saved_tensors
        x = dequantize_rows(q, scale, ctx.group, ctx.dtype).reshape(ctx.shape)
        need = ctx.needs_input_grad[4:]
        args = [t.detach().requires_grad_(n) if isinstance(t, torch.Tensor) else p
                for t, p, n in zip([x, *others], [None, *ctx.plain], need)]
        with torch.enable_grad(), ctx.surroundings.again():
            out = ctx.fn(*args)
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        pairs = [(o, g) for o, g in zip(out, grads) if g is not None and isinstance(o, torch.Tensor) and o.requires_grad]
        own = [a for a, n in zip(args, need) if n]
        got = [None] * len(own)
        if pairs:
            out, up = zip(*pairs)
            if torch.autograd.Variable._execution_engine.is_checkpoint_valid():  # backward() for all leaves
                torch.autograd.backward(out, up)
                got = [a.grad for a in own]
            else:
                _check_asked(ctx, out, own)
                got = torch.autograd.grad(out, own, up, allow_unused=True)
        got = iter(got)
        return (None, None, None, None, *(next(got) if n else None for n in need))


def checkpoint_8bit(fn, x, *others, kind="int8", group=128):
    """fn(x, *others), keeping x in 8 bits for the backward pass (any shape, groups along the last axis) and nothing
    of what fn computes: the backward pass runs fn again on what those 8 bits stand for, and its gradients are exactly
    the gradients there.  others (tensors or not) are kept as they are.

    Leaves that fn takes from elsewhere, such as a module's parameters, get their .grad from backward(); tensors that were
    computed with a gradient belong among the others.  torch.autograd.grad and backward(inputs=...) reach x and the others
    only, and are refused where they may have been asked for a tensor from elsewhere.  What fn takes from elsewhere must
    not change in between.

    fn has to compute the same both times: it runs under the autocast of the forward pass again, and random numbers of
    torch's own generators and of generators among the others are drawn again as they were (in a captured graph they are
    refused); others, such as numpy's, are not."""
    if not isinstance(x, torch.Tensor) or x.dim() == 0 or x.shape[-1] == 0:
        raise TypeError("x must be a tensor with a last axis of at least one element")
    if x.dtype not in B.TYPES:
        raise TypeError(f"x must be one of {', '.join(map(str, B.TYPES))}, got {x.dtype}")
    B._kind(kind, group)
    if not torch.is_grad_enabled() or not any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, *others)):
        return fn(x, *others)  # nothing of it is kept, or only what fn takes from elsewhere needs it
    form = []  # of a tuple that fn returns, a named one for instance
    out = _Checkpoint.apply(fn, kind, int(group), form, x, *others)
    return form[0](out) if form else out


# ---------------------------------------------------------------- layer norm
def layer_norm_forward(x, weight=None, bias=None, mask=None, eps=1e-5, checkpoint=None, group=128):
    """y [T,d], mean [T], rstd [T] and, with checkpoint "int8" or "e4m3", x in 8 bits (q, scale) for the backward
    (else None)."""
    T, d = B._norm_in(x, weight, bias, mask)
    y, mean, rstd = torch.empty_like(x), _f32(x, T), _f32(x, T)
    if checkpoint is None:
        B._layer_norm_fwd(T, d, x, weight, bias, mask, eps, y, mean, rstd)
        return y, mean, rstd, None
    code = B._kind(checkpoint, group)
    q = torch.empty(T, d, dtype=B.ROWS_TYPES[checkpoint], device=x.device)
    scale = _f32(x, T, B._groups(d, group))
    B._layer_norm_fwd(T, d, x, weight, bias, mask, eps, y, mean, rstd, code, group, q, scale)
    return y, mean, rstd, (q, scale)


def layer_norm_backward(grad, x, weight, mask, mean, rstd, kept=None, group=128, grad_dtype=None,
                        want=(True, True, True), workspace=None):
    """dx (grad's type), dweight and dbias (weight's type; without a weight grad_dtype, None: grad's), each None where
    `want` is false.  kept: the forward's (q, scale) in place of x, which is None then."""
    q, scale = (None, None) if kept is None else kept
    T, d, code = B._norm_bwd_in(grad, x, weight, mask, mean, rstd, group, q, scale)
    if not any(want):
        raise ValueError("dx, dweight and dbias are all not wanted")
    wt = weight.dtype if weight is not None else grad_dtype or grad.dtype
    if wt != grad.dtype and wt != torch.float32:
        raise TypeError(f"grad_dtype must be {grad.dtype} or torch.float32, got {wt}")
    dx = torch.empty_like(grad) if want[0] else None
    dw, db = (torch.empty(d, dtype=wt, device=grad.device) if w else None for w in want[1:])
    if workspace is None:
        workspace = _workspace(B.kd_layer_norm_workspace_size(T, d), grad.device)
    B._layer_norm_bwd(T, d, code, wt, grad, x, weight, mask, mean, rstd, dx, dw, db, workspace, group, q, scale)
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, mask, eps, checkpoint, group):
        y, mean, rstd, kept = layer_norm_forward(x, weight, bias, mask, eps, checkpoint, group)
        ctx.save_for_backward(x if kept is None else None, weight, mask, mean, rstd, *(kept or (None, None)))
        ctx.group, ctx.wtype = group, None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, mask, mean, rstd, q, scale = ctx.saved_tensors
        grads = layer_norm_backward(g.contiguous(), x, weight, mask, mean, rstd, None if q is None else (q, scale),
                                    ctx.group, ctx.wtype, ctx.needs_input_grad[:3])
        return (*grads, None, None, None, None)


def layer_norm(x, weight=None, bias=None, mask=None, eps=1e-5, checkpoint=None, group=128):
    """Layer norm of the rows of x [T,d], 0 on masked rows; differentiable in x, weight and bias, whose gradients have
    their types.  weight and bias are of x's type or float32.  checkpoint "int8" or "e4m3": the backward pass takes x
    from 8 bits, in groups of `group` values with a scale each, and x itself is not kept."""
    if checkpoint is not None:
        B._kind(checkpoint, group)
        # (within apply, gradients count as on, and as needed wherever an input has one)
        if not torch.is_grad_enabled() or not any(getattr(t, "requires_grad", False) for t in (x, weight, bias)):
            checkpoint = None
    return _LayerNorm.apply(x, weight, bias, mask, float(eps), checkpoint, int(group))


# ---------------------------------------------------------------- product of 8-bit integers
def int8_matmul(x, x_scale, w, w_scale, out_dtype=torch.bfloat16, workspace=None):
    """out [T,V] = x w^T with x_scale [T] and w_scale [V] (or [T,1], [V,1]): x [T,d] int8, w [V,d] int8 with a row for
    each channel, d a multiple of 16.  quantize_rows(H, "int8", 0) gives x, quantize_rows of a head's transpose w."""
    T, d, V = B._int8_in(x, x_scale, w, w_scale)
    if out_dtype not in B.TYPES:
        raise TypeError(f"out_dtype must be one of {', '.join(map(str, B.TYPES))}, got {out_dtype}")
    out = torch.empty(T, V, dtype=out_dtype, device=x.device)
    if workspace is None:
        n = B.kd_int8_matmul_workspace_size(T, d, V)
        workspace = _workspace(n, x.device) if n else None
    B._int8_matmul(T, d, V, x, x_scale, w, w_scale, out, workspace)
    return out

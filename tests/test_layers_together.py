"""The layers as a model has them around the head: captured, on other streams, with the losses."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests import layers_util as R
from tests.gpu_util import say
from tests.test_workspace_canary import Guarded

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def model(V=520, d=128, T=300, seed=0, masked=0.2):
    g = R.gen(seed)
    tokens, mask = R.make_tokens(T, V, seed, masked)
    s = dict(tokens=tokens, mask=mask, W=(torch.randn(d, V, generator=g) / d ** 0.5).to(bf),
             w=(1 + 0.1 * torch.randn(d, generator=g)).to(bf), b=(0.1 * torch.randn(d, generator=g)).to(bf),
             labels=torch.randint(0, V, (T,), generator=g, dtype=torch.int32), up=torch.randn(T, generator=g) / T)
    return {k: v if v is None else v.cuda() for k, v in s.items()}


def step(s, kept="int8"):
    """Tied embedding, norm with its input in 8 bits, token log-probabilities, and back: every gradient."""
    V = s["W"].shape[1]
    X = kd.embedding_forward(s["tokens"], s["W"], s["mask"], 4.0, tied=True)
    H, mean, rstd, k = kd.layer_norm_forward(X, s["w"], s["b"], s["mask"], checkpoint=kept, group=64)
    logp, lse, _, _ = kd.token_logp_forward(H, s["W"], s["labels"], s["mask"])
    dH, dW = kd.token_logp_backward(H, s["W"], s["labels"], s["mask"], 1.0, lse, s["up"])
    dX, dw, db = kd.layer_norm_backward(dH, None if k else X, s["w"], s["mask"], mean, rstd, k, 64)
    kd.embedding_backward(dX, s["tokens"], V, s["mask"], 4.0, tied=True, out=dW)
    return [X, H, logp, dH, dX, dw, db, dW]


def score(s):
    """Logits through the head in 8 bits, as a frozen teacher gives them, and the loss against its largest ones."""
    X = kd.embedding_forward(s["tokens"], s["W"], s["mask"], 4.0, tied=True)
    H = kd.layer_norm_forward(X, s["w"], s["b"], s["mask"])[0]
    q, sc = kd.quantize_rows(H, "int8", 0)
    Z = kd.int8_matmul(q, sc, s["wq"], s["ws"], torch.float32)
    return [H, q, sc, Z]


def test_training_step_is_the_autograd_one():
    s = model()
    got = step(s, kept=None)
    W, w, b = (s[k].clone().requires_grad_(True) for k in ("W", "w", "b"))
    X = kd.embedding(s["tokens"], W, s["mask"], 4.0, tied=True)
    X.retain_grad()
    H = kd.layer_norm(X, w, b, s["mask"])
    logp = kd.token_logp(H, W, s["labels"], s["mask"])
    logp.backward(s["up"])
    for a, c in zip(got[:3], (X, H, logp)):
        assert torch.equal(a, c)
    for a, c in zip(got[4:7], (X.grad, w.grad, b.grad)):
        assert torch.equal(a, c)
    # the head's gradient: here a float32 sum of the two shares p and q; in autograd each is rounded to bf16, and so is
    # their sum, which makes u |p| + u |q| + u |p + q| with u = 2^-8, and terms of u^2 below a hundredth of that.  (A
    # bound by the sum alone does not hold: where the shares nearly cancel, their roundings remain.)
    V = W.shape[1]
    q = kd.embedding_backward(got[4], s["tokens"], V, s["mask"], 4.0, tied=True, grad_dtype=torch.float32).double()
    p = got[7].double() - q
    off = (got[7].double() - W.grad.double()).abs()
    assert bool((off <= 1.01 * 2.0 ** -8 * (p.abs() + q.abs() + (p + q).abs()) + 1e-12).all())


def test_checkpointed_step():
    """checkpoint_8bit around norm and loss: the gradients are those at the values that 8 bits hold."""
    s = model(seed=3)
    X = kd.embedding_forward(s["tokens"], s["W"], s["mask"], 4.0, tied=True)
    W, w, b = (s[k].clone().requires_grad_(True) for k in ("W", "w", "b"))

    def block(x, w, b, W):
        return kd.token_logp(kd.layer_norm(x, w, b, s["mask"]), W, s["labels"], s["mask"])

    x = X.clone().requires_grad_(True)
    out = kd.checkpoint_8bit(block, x, w, b, W, kind="e4m3", group=32)
    got = torch.autograd.grad(out, (x, w, b, W), s["up"])
    assert torch.equal(out, block(X, w, b, W))
    q, sc = kd.quantize_rows(X, "e4m3", 32)
    xd = kd.dequantize_rows(q, sc, 32, bf).requires_grad_(True)
    want = torch.autograd.grad(block(xd, w, b, W), (xd, w, b, W), s["up"])
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_saved_tensors_moved_and_changed():
    """What autograd saved may lie elsewhere by then (hooks that keep it on the host), and is refused if it changed."""
    s = model(seed=4)
    X = torch.randn(300, 128, device="cuda").to(bf)

    def run(hooks, kept):
        x, w, W = (t.clone().requires_grad_(True) for t in (X, s["w"], s["W"]))
        with torch.autograd.graph.save_on_cpu() if hooks else torch.enable_grad():
            y = kd.layer_norm(x, w, s["b"], s["mask"], checkpoint=kept) + kd.embedding(s["tokens"], W, s["mask"], tied=True)
        return torch.autograd.grad(y, (x, w, W), X)

    for kept in (None, "int8", "e4m3"):
        assert all(torch.equal(a, b) for a, b in zip(run(False, kept), run(True, kept)))
    x = X.clone().requires_grad_(True)
    z = x * 1
    y = kd.layer_norm(z, s["w"])
    z.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_gradients_that_come_expanded_or_not_at_all():
    s = model(seed=6)
    x, w, b = (t.clone().requires_grad_(True) for t in (torch.randn(300, 128, device="cuda"), s["w"].float(), s["b"].float()))
    y = kd.layer_norm(x, w, b, s["mask"])
    got = torch.autograd.grad(y.sum(), (x, w, b), retain_graph=True)  # an expanded upstream gradient
    want = torch.autograd.grad(y, (x, w, b), torch.ones_like(y))
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    (only,) = torch.autograd.grad(kd.layer_norm(x.detach(), w, None, s["mask"]).sum(), w)  # a leaf alone
    assert torch.equal(only, want[1])
    W = s["W"].clone().requires_grad_(True)
    (g,) = torch.autograd.grad(kd.embedding(s["tokens"], W, s["mask"], tied=True).sum(), W)
    assert torch.equal(g, kd.embedding_backward(torch.ones(300, 128, device="cuda", dtype=bf), s["tokens"], 520, s["mask"],
                                                tied=True))


def test_teacher_through_8_bits_to_the_loss():
    s = model(T=64, seed=5, masked=0.0)
    s["wq"], s["ws"] = kd.quantize_rows(s["W"].t().contiguous(), "int8", 0)
    H, _, _, Z = score(s)
    top, idx = Z.topk(8, 1)
    kl, lse, _ = kd.topk_kl_forward(H, s["W"], idx.int(), top)
    p = torch.softmax(top.double(), 1)
    z = (H.double() @ s["W"].double())
    want = (p * (p.log() - z.gather(1, idx))).sum(1) + torch.logsumexp(z, 1)
    assert bool(((kl.double() - want).abs() <= 1e-3).all())


@pytest.mark.parametrize("what", ["step", "score"])
def test_captured_and_replayed(what):
    """Two graphs captured over one pool, replayed in turn with new inputs and eager work between: every replay gives
    the eager call's bits."""
    say(f"layers captured: {what}")
    states = [model(seed=k, T=300 if k else 17000, d=64) for k in range(2)]
    fn = step if what == "step" else score
    for s in states:
        s["wq"], s["ws"] = kd.quantize_rows(s["W"].t().contiguous(), "int8", 0)
        fn(s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    pool = torch.cuda.graph_pool_handle()
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(fn(s))
        graphs.append(g)
    for rep in range(4):
        for s, g, o in zip(states, graphs, outs):
            V = s["W"].shape[1]
            s["tokens"].copy_(torch.randint(0, V, s["tokens"].shape, dtype=torch.int32))
            s["mask"].copy_((torch.rand(s["mask"].shape) < 0.7).to(torch.uint8))
            g.replay()
            got = [t.clone() for t in o]
            torch.cuda.synchronize()
            want = fn(s)
            for i, (a, b) in enumerate(zip(got, want)):
                assert torch.equal(a.float(), b.float()), f"replay {rep}, output {i}"


def test_two_streams_at_once():
    say("layers on two streams")
    states = [model(seed=k, T=500 + k) for k in range(2)]
    want = [[t.clone() for t in step(s)] for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for _ in range(3):
        for k, (s, st) in enumerate(zip(states, streams)):
            with torch.cuda.stream(st):
                got[k] = step(s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("T", [1, 777, 16385])
def test_workspaces_are_kept_to(T):
    say(f"layers' workspaces T={T}")
    V, d = 900, 72
    s = model(V, d, T)
    grad = torch.randn(T, d, device="cuda").to(bf)
    for tied in (False, True):
        w = Guarded(kd.kd_embedding_workspace_size(T, V, d, tied))
        out = torch.empty((d, V) if tied else (V, d), device="cuda")
        kd.kd_embedding_bwd(grad, s["tokens"], s["mask"], 1.0, V, tied, False, out, w.ws)
        assert w.intact()
    y, mean, rstd, _ = kd.layer_norm_forward(grad, s["w"], s["b"], s["mask"])
    w = Guarded(kd.kd_layer_norm_workspace_size(T, d))
    dx, dw, db = torch.empty_like(grad), torch.empty_like(s["w"]), torch.empty_like(s["w"])
    kd.kd_layer_norm_bwd(grad, grad, s["w"], s["mask"], mean, rstd, dx, dw, db, w.ws)
    assert w.intact()
    x, sx, wt, sw = (t.cuda() for t in R.make_int8(T, 208, 33000, 1))
    w = Guarded(kd.kd_int8_matmul_workspace_size(T, 208, 33000))
    kd.kd_int8_matmul(x, sx, wt, sw, torch.empty(T, 33000, device="cuda", dtype=bf), w.ws)
    assert w.intact()


def test_inputs_at_any_element(offset=1):
    """Arrays that begin in the middle of a 16-byte piece."""
    T, V, d = 37, 50, 136
    s = model(V, d, T, masked=0.0)

    def shifted(t):
        buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = buf[offset:offset + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    E = s["W"].t().contiguous()
    a = kd.embedding_forward(s["tokens"], E, None, 2.0)
    assert torch.equal(a, kd.embedding_forward(shifted(s["tokens"]), shifted(E), None, 2.0))
    g = kd.embedding_backward(a, s["tokens"], V)
    out = shifted(torch.zeros_like(E))
    assert torch.equal(g, kd.embedding_backward(shifted(a), s["tokens"], V, out=out))
    n = kd.layer_norm_forward(a, s["w"], s["b"])
    m = kd.layer_norm_forward(shifted(a), shifted(s["w"]), shifted(s["b"]))
    assert all(torch.equal(p, q) for p, q in zip(n[:3], m[:3]))
    p = kd.layer_norm_backward(a, a, s["w"], None, n[1], n[2])
    q = kd.layer_norm_backward(shifted(a), shifted(a), shifted(s["w"]), None, n[1], n[2])
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    for kind in ("int8", "e4m3"):
        for group in (0, 32):
            x, y = kd.quantize_rows(a, kind, group), kd.quantize_rows(shifted(a), kind, group)
            assert torch.equal(x[0].view(torch.uint8), y[0].view(torch.uint8)) and torch.equal(x[1], y[1])

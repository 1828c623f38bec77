"""The preference loss on the GPU against the 64-bit form."""
import math

import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import dev, say
from tests.policy_util import U32, near, preference_reference

pytestmark = pytest.mark.gpu


def make(T, P, seed, masked=0.3):
    g = torch.Generator().manual_seed(seed)
    logp = -5 * torch.rand(T, generator=g)
    ref = logp + 0.5 * torch.randn(T, generator=g)
    mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    cuts = torch.randint(0, T + 1, (2 * P - 1,), generator=g).sort().values
    cu = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(torch.int32)
    return logp, ref, mask, cu, torch.randn(P, generator=g)


def check(logp, cu, mask, grad, what, **kw):
    """All sums and the loss are in 64 bits: T terms of at most 20 each, off by T 2^-53 20 < 1e-10 in a sum, which
    beta, 1 / n or the squared loss (times 2 |D| + 1 / beta < 1e5) carries on; then one rounding to 32 bits."""
    say(what)
    loss, rewards, g = preference_reference(logp, cu, mask, grad=grad, **kw)
    dkw = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    a = (dev(logp), dev(cu), dev(mask))
    got = kd.preference_loss_forward_backward(*a, dev(grad), **dkw)
    near(got[0], loss, "loss", small=1e-5 if kw.get("kind") == "ipo" else 1e-10)
    near(got[1], rewards, "rewards", small=1e-10)
    near(got[2], g, "grad_logp", small=1e-9)
    l2, r2, sums = kd.preference_loss_forward(*a, **dkw)
    g2 = kd.preference_loss_backward(logp.numel(), a[1], a[2], sums, dev(grad), **dkw)
    assert torch.equal(l2, got[0]) and torch.equal(r2, got[1]) and torch.equal(g2, got[2])
    return got


@pytest.mark.parametrize("T,P", [(2, 1), (3, 4), (64, 1), (500, 3), (513, 40), (1024, 1), (3000, 2), (20000, 1),
                                 (40000, 7), (6000, 1500)])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
def test_shapes(T, P, kind, average):
    for masked in (0.0, 0.3):
        logp, ref, mask, cu, grad = make(T, P, T + P, masked)
        check(logp, cu, mask, grad, f"T={T} P={P} {kind} average={average} masked={masked}", ref_logp=ref, kind=kind,
              average=average)


def test_one_long_sequence_among_short_ones():
    T = 70000
    logp, ref, mask, _, grad = make(T, 4, 3)
    cu = torch.tensor([0, 3, 66000, 66000, 66512, 67024, 67025, 69000, T], dtype=torch.int32)
    check(logp, cu, mask, grad, "ragged", ref_logp=ref, average=True)
    edges = torch.tensor([0, 512, 1024, 1025, 2047, 2048, 2560, 40960, T], dtype=torch.int32)
    check(logp, edges, mask, grad, "sequences that end where a wave's tokens do", ref_logp=ref)


@pytest.mark.parametrize("kw", [dict(beta=2.5), dict(label_smoothing=0.3), dict(margin=1.5),
                                dict(kind="hinge", margin=-0.5), dict(kind="ipo", beta=0.01)])
def test_options(kw):
    logp, ref, mask, cu, grad = make(900, 9, 5)
    check(logp, cu, mask, grad, str(kw), ref_logp=ref, **kw)
    check(logp, cu, mask, grad, f"no reference {kw}", **kw)


def test_masked_values_and_tokens_outside():
    logp, ref, mask, _, grad = make(4000, 2, 7)
    cu = torch.tensor([50, 600, 600, 2300, 3500], dtype=torch.int32)
    clean = check(logp, cu, mask, grad, "clean", ref_logp=ref)
    off = mask == 0
    logp[off], ref[off] = float("nan"), -math.inf
    logp[:50], ref[3500:] = float("inf"), float("nan")
    dirty = check(logp, cu, mask, grad, "dirty", ref_logp=ref)
    assert all(torch.equal(x, y) for x, y in zip(clean, dirty))
    assert (dirty[2][:50] == 0).all() and (dirty[2][3500:] == 0).all()


@pytest.mark.parametrize("T", [0, 10])
def test_empty_pairs(T):
    """No valid token on either side: D = 0, log 2, no gradient."""
    cu = torch.tensor([0, 0, T, T, T], dtype=torch.int32, device="cuda")
    logp = torch.randn(T, device="cuda")
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    for average in (False, True):
        loss, rewards, g = kd.preference_loss_forward_backward(logp, cu, mask, torch.ones(2, device="cuda"),
                                                               average=average)
        near(loss, torch.full((2,), math.log(2.0)), "loss")
        assert (rewards == 0).all() and (g == 0).all()


def test_far_margins():
    """exp of hundreds: the loss is linear on one side and vanishes on the other."""
    logp = torch.tensor([-5000.0, 0.0, 0.0, -5000.0])
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32)
    check(logp, cu, None, torch.ones(2), "far", beta=1.0)


def test_infinite_margins():
    """A rejected sequence of no probability costs nothing, a chosen one everything; the gradients are the limits."""
    logp = torch.tensor([0.0, -math.inf, -math.inf, 0.0], device="cuda")
    cu = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    loss, rewards, g = kd.preference_loss_forward_backward(logp, cu, None, torch.ones(2, device="cuda"), beta=0.5)
    assert loss.tolist() == [0.0, math.inf] and rewards.tolist() == [0.0, -math.inf, -math.inf, 0.0]
    assert g.tolist() == [0.0, -0.5, 0.0, 0.5]


def test_autograd():
    logp, ref, mask, cu, grad = make(700, 5, 11)
    _, _, g = preference_reference(logp, cu, mask, ref_logp=ref, grad=grad, average=True)
    x = dev(logp).requires_grad_(True)
    loss, rewards = kd.preference_loss(x, dev(cu), dev(mask), ref_logp=dev(ref), average=True)
    assert not rewards.requires_grad
    (loss * dev(grad)).sum().backward()
    near(x.grad, g, "grad_logp", rel=8 * U32, small=1e-9)


def test_gradient_against_differences():
    """Central differences in 64 bits of the reference form, off by e^2 = 2^-20 of smooth terms."""
    logp, ref, mask, cu, _ = make(60, 2, 13)
    kw = dict(ref_logp=ref, label_smoothing=0.1, beta=0.5)
    g = kd.preference_loss_forward_backward(dev(logp), dev(cu), dev(mask), torch.ones(2, device="cuda"),
                                            **{k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()})[2]
    e = 2.0 ** -10
    for t in range(0, 60, 11):
        up, down = logp.double(), logp.double()
        up[t] += e
        down[t] -= e
        d = (preference_reference(up, cu, mask, **kw)[0].sum() - preference_reference(down, cu, mask, **kw)[0].sum()) / (2 * e)
        assert abs(float(g[t]) - float(d)) <= 1e-5


def test_stream_and_graph():
    logp, ref, mask, cu, grad = [dev(x) for x in make(50000, 30, 17)]
    call = lambda: kd.preference_loss_forward_backward(logp, cu, mask, grad, ref_logp=ref)  # noqa: E731
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for k in range(3):
        logp.mul_(0.9)
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out)), k

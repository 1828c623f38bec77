"""The clipped policy loss on the GPU against the 64-bit form."""
import math

import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import dev, say
from tests.policy_util import U32, near, policy_reference

pytestmark = pytest.mark.gpu


def make(T, S, seed, masked=0.3, per_sequence=False):
    g = torch.Generator().manual_seed(seed)
    logp = -5 * torch.rand(T, generator=g)
    old = logp + 0.3 * torch.randn(T, generator=g)
    ref = logp + 0.5 * torch.randn(T, generator=g)
    ent = 3 * torch.rand(T, generator=g)
    adv = torch.randn(S if per_sequence else T, generator=g)
    mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g).sort().values
    cu = torch.cat([torch.tensor([0]), cuts, torch.tensor([T])]).to(torch.int32)
    return logp, old, ref, ent, adv, mask, cu


def check(args, kw, what):
    """stats, both forms of the gradients.  stats are sums of 64-bit terms, off by what rounding the inputs' products
    costs in 64 bits, relative to the terms' sizes, and one rounding to 32 bits; the gradients one rounding each."""
    say(what)
    want, g, ge = policy_reference(*args, **kw)
    dargs = [dev(x) for x in args]
    dkw = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    stats, dlogp, dent = kd.policy_loss_forward_backward(*dargs, **dkw)
    scale = 1e-12 * (1 + want.abs().max())  # 64-bit sums of at most 1e5 terms of these sizes
    near(stats, want, "stats", small=scale)
    near(dlogp, g, "grad_logp", small=1e-14)
    again, weights = kd.policy_loss_forward(*dargs, **dkw)
    assert torch.equal(again, stats)
    up = torch.tensor(-1.75, device="cuda")
    g2, ge2 = kd.policy_loss_backward(*dargs, weights, up, **dkw)
    near(g2, -1.75 * g, "grad_logp, backward", small=1e-14)
    if kw.get("entropy") is not None:
        near(dent, ge, "grad_entropy", small=1e-14)
        near(ge2, -1.75 * ge, "grad_entropy, backward", small=1e-14)
    else:
        assert dent is None and ge2 is None
    return stats


@pytest.mark.parametrize("T,S", [(1, 1), (2, 3), (63, 5), (64, 1), (333, 20), (512, 4), (513, 1), (1025, 700),
                                 (5000, 3), (20000, 90)])
@pytest.mark.parametrize("reduction", ["sum", "token", "sequence"])
def test_shapes_and_reductions(T, S, reduction):
    for masked in (0.0, 0.4):
        logp, old, ref, ent, adv, mask, cu = make(T, S, T + S, masked)
        check((logp, old, adv, mask), dict(ref_logp=ref, entropy=ent, cu_seqlens=cu, kl_weight=0.1, entropy_weight=0.02,
                                           reduction=reduction, per_sequence=False),
              f"T={T} S={S} {reduction} masked={masked}")


@pytest.mark.parametrize("kl_kind", ["k1", "k2", "k3"])
@pytest.mark.parametrize("dual", [0.0, 1.5])
@pytest.mark.parametrize("per_sequence", [False, True])
def test_options(kl_kind, dual, per_sequence):
    logp, old, ref, ent, adv, mask, cu = make(1500, 17, 7, per_sequence=per_sequence)
    old = old - 0.4 * (torch.arange(1500) % 3 == 0)
    kw = dict(ref_logp=ref, cu_seqlens=cu, kl_weight=0.3, kl_kind=kl_kind, dual_clip=dual, clip_low=0.1, clip_high=0.28,
              per_sequence=per_sequence)
    check((logp, old, adv, mask), kw, f"{kl_kind} dual={dual} per_sequence={per_sequence}")
    check((logp, old, adv, mask), dict(kw, kl_weight=0.0, reduction="sequence"), "reported KL without weight")


def test_no_sequences():
    logp, old, ref, ent, adv, mask, _ = make(3000, 1, 9)
    check((logp, old, adv, mask), dict(), "bare")
    check((logp, old, adv, None), dict(entropy=ent, entropy_weight=-0.5, reduction="sum"), "no mask")


def test_tokens_outside_the_sequences():
    logp, old, ref, ent, adv, mask, _ = make(2000, 1, 11)
    cu = torch.tensor([100, 100, 700, 750, 1500], dtype=torch.int32)
    logp[:100], adv[1500:] = float("nan"), float("inf")
    for red in ("sum", "token", "sequence"):
        check((logp, old, adv, mask), dict(cu_seqlens=cu, reduction=red, per_sequence=False), red)


def test_masked_values_do_not_matter():
    logp, old, ref, ent, adv, mask, cu = make(700, 9, 13)
    kw = dict(ref_logp=ref, entropy=ent, cu_seqlens=cu, kl_weight=0.1, entropy_weight=0.1, reduction="sequence")
    a = check((logp, old, adv, mask), kw, "clean")
    off = mask == 0
    for x, v in ((logp, -math.inf), (old, math.nan), (ref, math.inf), (ent, math.nan), (adv, math.nan)):
        x[off] = v
    b = check((logp, old, adv, mask), kw, "dirty")
    assert torch.equal(a, b)


@pytest.mark.parametrize("reduction", ["sum", "token", "sequence"])
@pytest.mark.parametrize("T", [0, 5, 900])
def test_nothing_valid(T, reduction):
    x = torch.randn(T, device="cuda")
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 0, T], dtype=torch.int32, device="cuda")
    kw = dict(cu_seqlens=cu, reduction=reduction, per_sequence=False)
    stats, g, _ = kd.policy_loss_forward_backward(x, x, x, mask, **kw)
    assert (stats == 0).all() and (g == 0).all()
    logp = x.clone().requires_grad_(True)
    loss, stats = kd.policy_loss(logp, x, x, mask, **kw)
    loss.backward()
    assert float(loss.detach()) == 0 and (logp.grad == 0).all()


def test_borders():
    """Ratios that are exactly representable next to and on the borders (1 - 1/4, 1 + 1/2): logp - old is exact, and
    exp of it in 64 bits is compared with the border in 64 bits."""
    lo, hi = math.log(0.75), math.log(1.5)
    base = torch.tensor([lo, hi] * 6, dtype=torch.float64)
    step = torch.tensor([-2.0, -2, -1, -1, 0, 0, 1, 1, 2, 2, 0, 0], dtype=torch.float64)
    logp = (base * (1 + step * 2.0 ** -24)).float()
    old = torch.zeros_like(logp)
    for sign in (1.0, -1.0):
        adv = torch.full_like(logp, sign)
        check((logp, old, adv, None), dict(clip_low=0.25, clip_high=0.5, reduction="sum"), f"sign {sign}")
    one = torch.zeros(3)
    check((one, one, torch.tensor([1.0, -1.0, 0.0]), None), dict(clip_low=0.0, clip_high=0.0), "ratio 1, no room")


def test_extremes():
    """Ratios that overflow 32 bits, and zero advantages beside them."""
    logp = torch.tensor([0.0, 0.0, -300.0, 0.0, -1e30])
    old = torch.tensor([-200.0, -200.0, 0.0, -200.0, 0.0])
    adv = torch.tensor([1.0, -1.0, 1.0, 0.0, 1.0])
    stats, g, _ = kd.policy_loss_forward_backward(*[dev(x) for x in (logp, old, adv)], reduction="sum", dual_clip=3.0)
    assert g.tolist()[0] == 0 and g.tolist()[1] == 0 and g.tolist()[3] == 0 and g.tolist()[4] == 0
    near(stats[:1], torch.tensor([-1.2 + 3.0 - math.exp(-300.0)]), "total")


@pytest.mark.parametrize("kl_kind", ["k1", "k2", "k3"])
def test_unweighted_kl_leaves_the_gradient_alone(kl_kind):
    """A reference that is only counted may be infinitely far off."""
    logp, old, adv = torch.tensor([-1.0, -2.0]), torch.tensor([-1.25, -2.0]), torch.tensor([1.0, -1.0])
    ref = torch.tensor([-math.inf, math.inf])
    plain = kd.policy_loss_forward_backward(*[dev(x) for x in (logp, old, adv)])
    stats, g, _ = kd.policy_loss_forward_backward(*[dev(x) for x in (logp, old, adv)], ref_logp=dev(ref), kl_kind=kl_kind)
    assert torch.equal(g, plain[1]) and torch.equal(stats[:2], plain[0][:2])
    assert not torch.isfinite(stats[2])


def test_autograd_and_in_place_use():
    logp, old, ref, ent, adv, mask, cu = make(800, 6, 17)
    kw = dict(ref_logp=ref, cu_seqlens=cu, kl_weight=0.2, entropy_weight=0.05, reduction="sequence")
    _, g, ge = policy_reference(logp, old, adv, mask, entropy=ent, **kw)
    x, e = dev(logp).requires_grad_(True), dev(ent).requires_grad_(True)
    dkw = {k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
    loss, stats = kd.policy_loss(x, dev(old), dev(adv), dev(mask), entropy=e, **dkw)
    assert loss.shape == () and torch.equal(loss.detach(), stats[0]) and not stats.requires_grad
    loss += 1.0
    (3 * loss).backward()
    near(x.grad, 3 * g, "grad_logp", rel=8 * U32, small=1e-14)
    near(e.grad, 3 * ge, "grad_entropy", rel=8 * U32, small=1e-14)


def test_gradient_against_differences():
    """Away from the borders the total is smooth: central differences in 64 bits of the reference form agree with the
    kernel's gradient to e^2 = 2^-20 of the terms."""
    logp, old, ref, ent, adv, mask, cu = make(40, 4, 19)
    kw = dict(ref_logp=ref, cu_seqlens=cu, kl_weight=0.2, reduction="sequence", clip_low=0.9, clip_high=9.0)
    _, g, _ = kd.policy_loss_forward_backward(*[dev(x) for x in (logp, old, adv, mask)],
                                              **{k: dev(v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
    e = 2.0 ** -10
    for t in range(0, 40, 7):
        up, down = logp.double(), logp.double()
        up[t] += e
        down[t] -= e
        d = (policy_reference(up, old, adv, mask, **kw)[0][0] - policy_reference(down, old, adv, mask, **kw)[0][0]) / (2 * e)
        assert abs(float(g[t]) - float(d)) <= 1e-5 * (1 + abs(float(d)))


def test_stream_and_graph():
    logp, old, ref, ent, adv, mask, cu = [dev(x) for x in make(30000, 50, 23)]
    kw = dict(ref_logp=ref, cu_seqlens=cu, kl_weight=0.2, reduction="sequence")
    call = lambda: kd.policy_loss_forward_backward(logp, old, adv, mask, **kw)[:2]  # noqa: E731
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
        old.add_(0.01)
        mask.copy_((torch.rand(30000, device="cuda") > 0.2 * k).to(torch.uint8))
        want = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, out)), k

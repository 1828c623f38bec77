"""The operators together, as a training step uses them: log-probabilities through the head, a loss on them, the
gradients of the hidden states and the head, and their clipping."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import dev, say
from tests.policy_util import (U32, half_step, logp_reference, make_head, near, policy_reference, preference_reference,
                               within)

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32

# the register-fed tiles, the forward on the ring tiles, and everything on the ring tiles
SIZES = [(300, 128, 520, bf), (300, 128, 520, f32), (1000, 160, 7016, bf), (1000, 1056, 7016, bf)]


def cuts(T, S, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.cat([torch.tensor([0]), torch.randint(0, T + 1, (S - 1,), generator=g).sort().values,
                      torch.tensor([T])]).to(torch.int32)


def check_clipped(grads, kept, max_norm, norm):
    """The norm in 64 bits, rounded once; each gradient times the factor (rounded once), rounded once to its type."""
    want = torch.stack([k.double().square().sum() for k in kept]).sum().sqrt()
    near(norm, want.cpu(), "norm")
    factor = min(1.0, max_norm / (float(want) + 1e-6))
    for g, k in zip(grads, kept):
        w = k.double() * factor
        assert ((g.double() - w).abs() <= (half_step(k.dtype) + 4 * U32) * w.abs() + 1e-37).all()


@pytest.mark.parametrize("keep_logits", [False, True])
@pytest.mark.parametrize("T,d,V,dtype", SIZES)
def test_policy_step(T, d, V, dtype, keep_logits):
    say(f"policy step T={T} V={V} {dtype} keep_logits={keep_logits}")
    H, W, tokens, mask = make_head(T, d, V, dtype, 71, masked=0.3)
    gen = torch.Generator().manual_seed(72)
    cu, adv = cuts(T, 5, 73), torch.randn(5, generator=gen)
    h, w = dev(H).requires_grad_(True), dev(W).requires_grad_(True)
    logp, ent = kd.token_logp(h, w, dev(tokens), dev(mask), 0.7, want_entropy=True, keep_logits=keep_logits)
    old = (logp.detach() + 0.2 * dev(torch.randn(T, generator=gen))).contiguous()
    ref = (logp.detach() + 0.2 * dev(torch.randn(T, generator=gen))).contiguous()
    kw = dict(kl_weight=0.1, entropy_weight=0.03, reduction="sequence", per_sequence=True)
    loss, stats = kd.policy_loss(logp, old, dev(adv), dev(mask), ref, ent, dev(cu), **kw)
    loss.backward()
    # each stage against 64 bits, from what the stage before it gave
    x, e = logp.detach().cpu(), ent.detach().cpu()
    wstats, g, ge = policy_reference(x, old.cpu(), adv, mask, ref.cpu(), e, cu, **kw)
    near(stats, wstats, "stats", small=1e-12 * (1 + wstats.abs().max()))
    near(loss, wstats[0], "loss", small=1e-12 * (1 + wstats.abs().max()))
    want, bound = logp_reference(H, W, tokens, mask, 0.7, g, ge)
    for name, got in (("logp", logp), ("entropy", ent)):
        within(got, want[name], bound[name], name)
    for name, got in (("dH", h.grad), ("dW", w.grad)):  # g and ge themselves are rounded to 32 bits, 2^-24 of dZ
        within(got, want[name], 1.01 * bound[name], name)
    kept = [h.grad.clone(), w.grad.clone()]
    norm = kd.clip_grad_norm_([h.grad, w.grad], 0.01)
    check_clipped([h.grad, w.grad], kept, 0.01, norm)


@pytest.mark.parametrize("T,d,V,dtype", SIZES)
def test_preference_step(T, d, V, dtype):
    """The reference's log-probabilities come from another, frozen head."""
    say(f"preference step T={T} V={V} {dtype}")
    H, W, tokens, mask = make_head(T, d, V, dtype, 81, masked=0.2)
    W0 = make_head(T, d, V, dtype, 82)[1]
    cu = cuts(T, 6, 83)
    h, w = dev(H).requires_grad_(True), dev(W).requires_grad_(True)
    with torch.no_grad():
        ref = kd.token_logp(dev(H), dev(W0), dev(tokens), dev(mask))
    logp = kd.token_logp(h, w, dev(tokens), dev(mask))
    loss, rewards = kd.preference_loss(logp, dev(cu), dev(mask), ref, beta=0.3, average=True)
    loss.mean().backward()
    third = torch.full((3,), 1 / 3)
    wloss, wrewards, g = preference_reference(logp.detach().cpu(), cu, mask, ref.cpu(), 0.3, average=True, grad=third)
    near(loss, wloss, "loss", small=1e-12)
    near(rewards, wrewards, "rewards", small=1e-12)
    want, bound = logp_reference(H, W, tokens, mask, 1.0, g)
    within(h.grad, want["dH"], 1.01 * bound["dH"], "dH")
    within(w.grad, want["dW"], 1.01 * bound["dW"], "dW")
    kept = [h.grad.clone(), w.grad.clone()]
    norm = kd.clip_grad_norm_((p.grad for p in (h, w)), 0.05)
    check_clipped([h.grad, w.grad], kept, 0.05, norm)


class Step:
    """A policy step without autograd, over inputs of its own."""

    def __init__(self, T, d, V, dtype, seed):
        H, W, tokens, mask = make_head(T, d, V, dtype, seed, masked=0.3)
        gen = torch.Generator().manual_seed(seed + 1)
        self.h, self.w, self.tokens, self.mask = (dev(x) for x in (H, W, tokens, mask))
        self.old, self.adv = dev(-3 * torch.rand(T, generator=gen)), dev(torch.randn(T, generator=gen))
        self.cu = dev(cuts(T, 5, seed + 2))

    def run(self):
        a = (self.h, self.w, self.tokens, self.mask, 1.0)
        logp, lse, ent, z = kd.token_logp_forward(*a, want_entropy=True, keep_logits=True)
        stats, g, ge = kd.policy_loss_forward_backward(logp, self.old, self.adv, self.mask, cu_seqlens=self.cu,
                                                       entropy=ent, entropy_weight=0.02, reduction="sequence")
        dH, dW = kd.token_logp_backward(*a, lse, g, ent, ge, z, dw_dtype=self.w.dtype)
        norm = kd.clip_grad_norm([dH, dW], 0.01)
        return [logp, ent, stats, dH, dW, norm]


@pytest.mark.parametrize("T,d,V,dtype", SIZES)
def test_captured_step(T, d, V, dtype):
    say(f"captured step T={T} V={V} {dtype}")
    a, b = Step(T, d, V, dtype, 91), Step(T, d, V, dtype, 95)
    a.run()
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):  # two graphs, replayed in turn
        graphs.append((torch.cuda.CUDAGraph(), s))
        with torch.cuda.graph(graphs[-1][0]):
            s.out = s.run()
    for k in range(3):
        for graph, s in graphs:
            s.h.mul_(0.9)
            s.mask.copy_((torch.rand(T, device="cuda") >= 0.4 * k).to(torch.uint8))
            want = s.run()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(s.out, want)), f"replay {k}"


def test_two_streams_at_once():
    steps = [Step(*SIZES[3], 101), Step(*SIZES[0], 105)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(steps):
            with torch.cuda.stream(streams[i]):
                got[i].append(s.run())
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(out, want[i]))


def test_captured_autograd():
    """Leaves used on the capturing stream alone, and no other graph of them alive."""
    s = Step(*SIZES[0], 111)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    h, w = s.h.detach().clone().requires_grad_(True), s.w.detach().clone().requires_grad_(True)

    def run():
        logp, ent = kd.token_logp(h, w, s.tokens, s.mask, want_entropy=True, keep_logits=True)
        loss, _ = kd.policy_loss(logp, s.old, s.adv, s.mask, entropy=ent, cu_seqlens=s.cu, entropy_weight=0.02,
                                 reduction="sequence")
        return list(torch.autograd.grad(loss, (h, w)))

    with torch.cuda.stream(stream):
        run()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = run()
    for k in range(3):
        with torch.no_grad():
            s.h.mul_(0.8)
            h.copy_(s.h)
        logp, lse, ent, z = kd.token_logp_forward(s.h, s.w, s.tokens, s.mask, 1.0, True, True)
        _, g, ge = kd.policy_loss_forward_backward(logp, s.old, s.adv, s.mask, cu_seqlens=s.cu, entropy=ent,
                                                   entropy_weight=0.02, reduction="sequence")
        want = kd.token_logp_backward(s.h, s.w, s.tokens, s.mask, 1.0, lse, g, ent, ge, z, dw_dtype=bf)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), f"replay {k}"

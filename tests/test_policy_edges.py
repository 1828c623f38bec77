"""Calls of the policy operators at the edges of what their documentation allows, on the GPU."""
import math

import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import dev, say
from tests.policy_util import U32, half_step, make_head

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def test_the_largest_chunk_of_an_odd_vocabulary():
    """45056 rows of 47368 columns: dZ and the zeros behind it would pass 4 GB.  dH of a few rows."""
    T, d, V = 45056, 64, 47368
    say(f"largest chunk T={T} d={d} V={V}")
    H, W, tokens, _ = make_head(T, d, V, bf, 5)
    h, w, t = dev(H), dev(W), dev(tokens)
    g = torch.randn(T, generator=torch.Generator().manual_seed(6))
    _, lse, _, _ = kd.token_logp_forward(h, w, t)
    dH, _ = kd.token_logp_backward(h, w, t, None, 1.0, lse, dev(g), chunk_rows=T, want=(True, False))
    at = torch.cat([torch.arange(0, T, 1408), torch.tensor([T - 1])]).cuda()
    Hd, Wd, gd = h[at].double(), w.double(), dev(g)[at].double()[:, None]
    z = Hd @ Wd
    l64 = torch.logsumexp(z, 1, keepdim=True)
    q = (z - l64).exp()
    y = t[at].long()[:, None]
    dz, size = (-gd * q).scatter_add_(1, y, gd), (gd.abs() * q).scatter_add_(1, y, gd.abs())
    Wt = Wd.t().contiguous()
    want, u = dz @ Wt, half_step(bf)
    # as in logp_reference: 32-bit sums of d products, dZ's rounding, sums of V products, dH's rounding
    off = (d + 16) * U32 * (Hd.abs() @ Wd.abs()).amax(1, keepdim=True)
    sized = size @ Wt.abs()
    moved = (u + 4 * (2 * off + 2.0 ** -20 * (1 + l64.abs())) + 2.0 ** -18) * sized
    bound = moved + V * U32 * sized + u * (want.abs() + moved)
    assert ((dH[at].double() - want).abs() <= bound).all()


def test_parameters_are_not_clipped():
    """Their gradients are what is clipped; the weights stay as they were."""
    p = torch.nn.Parameter(torch.full((1000,), 3.0, device="cuda"))
    for call in (lambda: kd.clip_grad_norm_([p], 1.0), lambda: kd.clip_grad_norm([torch.ones_like(p)], 1.0, out=[p])):
        with pytest.raises(ValueError, match=r"\.grad"):
            call()
    p.grad = torch.full((1000,), 2.0, device="cuda")
    norm = kd.clip_grad_norm_([p.grad], 1.0)
    assert (p == 3.0).all() and abs(float(norm) - 2 * 1000 ** 0.5) < 1e-3 and abs(float(p.grad.norm()) - 1) < 1e-5
    kd.clip_grad_norm_([p.detach()], 1.0)
    assert abs(float(p.detach().norm()) - 1) < 1e-5
    assert abs(float(kd.clip_grad_norm([p], 0.5, out=[torch.empty(1000, device="cuda")])) - 1) < 1e-5


@pytest.mark.parametrize("numel", [2048, 32768])
def test_many_small_tensors_do_not_wait_for_each_other(numel):
    """The same elements in 132 tensors and in 8, in replayed graphs: a launch that walked the tensors one by one took
    10 times as long."""
    def replay(n):
        ts = [torch.full((numel // n,), 0.5, device="cuda") for _ in range(n)]
        outs = [torch.empty_like(t) for t in ts]
        norm = kd.clip_grad_norm(ts, 1.0, outs)
        assert abs(float(norm) - 0.5 * (n * (numel // n)) ** 0.5) < 1e-4
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                kd.clip_grad_norm(ts, 1.0, outs)
        best = math.inf
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    few, many = replay(8), replay(132)
    say(f"clip {numel} elements, 20 calls: 8 tensors {few * 1e3:.0f} us, 132 tensors {many * 1e3:.0f} us")
    assert many < 4 * few


@pytest.mark.parametrize("count", [7, 8, 9])
@pytest.mark.parametrize("empty", [0, 3])
def test_one_launch_and_three_agree(count, empty):
    """On both sides of the rule, empty tensors not counted."""
    ts = [dev((torch.arange(101 + i) % 7 - 3.0).to((f32, bf, torch.float16)[i % 3])) for i in range(count)]
    ts[1:1] = [torch.empty(0, device="cuda") for _ in range(empty)]
    want = math.sqrt(sum(float(t.double().square().sum()) for t in ts))
    outs = [torch.empty_like(t, dtype=f32) for t in ts]
    norm = kd.clip_grad_norm(ts, 0.5 * want, outs)
    assert abs(float(norm) - want) <= 2 * U32 * want
    for t, o in zip(ts, outs):
        w = t.double() * (0.5 * want / (want + 1e-6))
        assert ((o.double() - w).abs() <= 5 * U32 * w.abs()).all()

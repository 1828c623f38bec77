"""Calls of the policy operators at the edges of what their documentation allows, on the GPU."""
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

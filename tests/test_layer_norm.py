"""Layer norm and its gradients against plain forms in 64 bits."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests import layers_util as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
SHAPES = [  # T, d
    (1, 1), (2, 2), (1, 4096), (7, 9), (5, 511), (9, 512), (6, 513), (33, 1024), (10, 1337), (4, 2048), (3, 2049),
    (700, 64), (5, 4097), (3, 8192), (2, 8200), (3, 16384), (2, 16385), (3, 40003), (2100, 96),
]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
         (torch.float16, torch.float16)]


def make(T, d, dtype, wtype, masked, seed=0, offset=0.3):
    x, mask = R.make_rows(T, d, dtype, T + d + seed, offset, masked)
    g = R.gen(d)
    w, b = (1 + 0.3 * torch.randn(d, generator=g)).to(wtype), (0.2 * torch.randn(d, generator=g)).to(wtype)
    grad = torch.randn(T, d, generator=g).to(dtype)
    if mask is not None:
        grad[mask == 0] = float("inf")  # never read
    return x, mask, w, b, grad


@pytest.mark.parametrize("dtype,wtype", TYPES)
@pytest.mark.parametrize("T,d", SHAPES)
def test_both_passes(T, d, dtype, wtype):
    say(f"layer norm {dtype} weights {wtype} T={T} d={d}")
    for masked, with_w, with_b in ((0.0, True, True), (0.4, True, False), (0.0, False, True), (0.3, False, False)):
        x, mask, w, b, grad = make(T, d, dtype, wtype, masked)
        w, b = w if with_w else None, b if with_b else None
        y, mean, rstd, kept = kd.layer_norm_forward(x.cuda(), cuda(w), cuda(b), cuda(mask), 1e-5)
        assert kept is None
        want, bound = R.norm_reference(x, w, b, mask, 1e-5, grad)
        what = f"masked={masked} weight={with_w} bias={with_b} "
        for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
            R.check(got, want[name], bound[name], what + name)
        wt = wtype if with_w or with_b else dtype
        args = (grad.cuda(), x.cuda(), cuda(w), cuda(mask), mean, rstd)
        got = kd.layer_norm_backward(*args, grad_dtype=wt)
        for name, t in zip(("dx", "dw", "db"), got):
            R.check(t, want[name], bound[name], what + name)
        again = kd.layer_norm_backward(*args, grad_dtype=wt)
        assert all(torch.equal(p, q) for p, q in zip(got, again)), "not the same bits"
        for i in range(3):  # one alone
            alone = kd.layer_norm_backward(*args, grad_dtype=wt, want=[j == i for j in range(3)])
            assert torch.equal(alone[i], got[i]) and sum(t is None for t in alone) == 2


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [0, 32, 128, 512])
@pytest.mark.parametrize("T,d", [(1, 1), (7, 40), (33, 512), (5, 1337), (3, 4096), (700, 96), (2, 16384), (3, 16391)])
def test_backward_from_8_bits(T, d, group, kind):
    say(f"layer norm from 8 bits {kind} group={group} T={T} d={d}")
    for dtype, wtype in TYPES[:3]:
        for masked in (0.0, 0.3):
            x, mask, w, b, grad = make(T, d, dtype, wtype, masked)
            plain = kd.layer_norm_forward(x.cuda(), w.cuda(), b.cuda(), cuda(mask))
            y, mean, rstd, kept = kd.layer_norm_forward(x.cuda(), w.cuda(), b.cuda(), cuda(mask), checkpoint=kind,
                                                        group=group)
            assert all(torch.equal(p, q) for p, q in zip((y, mean, rstd), plain))
            clean = torch.where(R.valid_rows(mask, T)[:, None], x, torch.zeros((), dtype=dtype))
            q, s = kd.quantize_rows(clean.cuda(), kind, group)
            assert torch.equal(kept[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(kept[1], s)
            values = R.rows_values(q.cpu().to(torch.float32), s.cpu(), group)
            want, bound = R.norm_reference(x, w, b, mask, 1e-5, grad, values)
            got = kd.layer_norm_backward(grad.cuda(), None, w.cuda(), cuda(mask), mean, rstd, kept, group)
            for name, t in zip(("dx", "dw", "db"), got):
                R.check(t, want[name], bound[name], f"{dtype} masked={masked} {name}")


@pytest.mark.parametrize("T,d", [(17, 130), (9, 200), (8, 256), (11, 257), (5, 520), (4099, 600), (7, 1024), (3, 4608),
                                 (5, 6144), (3, 6145), (3, 9216)])
def test_rows_that_share_a_workgroup_and_wide_ones(T, d):
    """The last workgroup's rows end before the last of them, or its loop does; rows of three pieces a thread."""
    for dtype, wtype in TYPES[:3]:
        test_both_passes(T, d, dtype, wtype)
    for group, kind in ((0, "int8"), (32, "e4m3"), (128, "int8")):
        test_backward_from_8_bits(T, d, group, kind)



def test_large_means_and_constant_rows():
    """The variance is taken around the mean: rows far from 0 keep their digits, constant rows give the bias."""
    for d in (100, 4096, 20000):
        x, _, w, b, grad = make(6, d, torch.float32, torch.float32, 0.0, offset=1000.0)
        x[3] = 7.25
        y, mean, rstd, _ = kd.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
        want, bound = R.norm_reference(x, w, b, None, 1e-5)
        rows = [0, 1, 2, 4, 5]
        R.check(y[rows], want["y"][rows], bound["y"][rows], f"d={d}")
        # a constant row's own bound is its mean's rounding times 1 / sqrt(eps): the mean of equal values is off by at
        # most chain u |x|
        assert bool(((y[3].cpu().double() - b.double()).abs() <= bound["y"][3]).all())


def test_nothing_valid_and_no_rows():
    x, mask, w, b, grad = make(6, 70, torch.bfloat16, torch.bfloat16, 0.5)
    mask = torch.zeros(6, dtype=torch.uint8)
    y, mean, rstd, _ = kd.layer_norm_forward(x.cuda(), w.cuda(), b.cuda(), mask.cuda())
    assert not y.any() and not mean.any() and not rstd.any()
    assert not any(t.any() for t in kd.layer_norm_backward(grad.cuda(), x.cuda(), w.cuda(), mask.cuda(), mean, rstd))
    e = torch.empty(0, 70, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd, _ = kd.layer_norm_forward(e, w.cuda(), b.cuda())
    dx, dw, db = kd.layer_norm_backward(e, e, w.cuda(), None, mean, rstd)
    assert y.shape == dx.shape == (0, 70) and not dw.any() and not db.any()


def test_rows_with_nan_or_infinity_stay_among_themselves():
    x, _, w, b, grad = make(8, 200, torch.float32, torch.float32, 0.0)
    x[2, 5], x[4, 7] = float("nan"), float("inf")
    y, mean, rstd, _ = kd.layer_norm_forward(x.cuda(), w.cuda(), b.cuda())
    assert torch.equal(y.isnan().any(1).cpu(), torch.tensor([0, 0, 1, 0, 1, 0, 0, 0], dtype=torch.bool))


@pytest.mark.parametrize("kind", [None, "int8", "e4m3"])
def test_autograd_and_differences(kind):
    """dx against differences of the loss sum(up y) along a direction: central differences of step s leave s^2 times a
    third derivative and 2 u |loss terms| / s."""
    T, d = 12, 200
    x, mask, w, b, grad = make(T, d, torch.float32, torch.float32, 0.3)
    x = torch.where(mask[:, None] != 0, x, torch.zeros(()))
    grad = torch.where(mask[:, None] != 0, grad, torch.zeros(()))
    leaves = [t.cuda().requires_grad_(True) for t in (x, w, b)]
    y = kd.layer_norm(*leaves, mask.cuda(), checkpoint=kind, group=32)
    got = torch.autograd.grad(y, leaves, grad.cuda())
    values = None
    if kind:
        q, s = R.rows_reference(x, kind, 32)
        values = R.rows_values(q, s, 32).float().double()
    want, bound = R.norm_reference(x, w, b, mask, 1e-5, grad, values)
    for name, t in zip(("dx", "dw", "db"), got):
        R.check(t, want[name], bound[name], name)
    if kind:
        return
    step = 2.0 ** -6
    dirs = [torch.randn(t.shape, generator=R.gen(k)) for k, t in enumerate((x, w, b))]
    loss = [0.0, 0.0]
    for k, sign in enumerate((-1, 1)):
        moved = [(t + sign * step * v).cuda() for t, v in zip((x, w, b), dirs)]
        out = kd.layer_norm_forward(*moved, mask.cuda())[0].cpu().double()
        loss[k] = (out * grad.double()).sum()
    diff = (loss[1] - loss[0]) / (2 * step)
    slope = sum((g.cpu().double() * v.double()).sum() for g, v in zip(got, dirs))
    size = (y.detach().cpu().double().abs() * grad.double().abs()).sum()
    # rows of 200 values of size 1: the third derivative along a direction of that size is at most about 30 of the terms
    assert abs(diff - slope) <= 30 * step ** 2 * size + 64 * R.U32 * size / step


def test_offsets_beyond_32_bits():
    T, d = 600000, 4096
    say(f"layer norm T={T} d={d}")
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd, _ = kd.layer_norm_forward(x, w)
    dx, _, db = kd.layer_norm_backward(x, x, w, None, mean, rstd)
    for a in (0, T // 2, T - 64):
        p = x[a:a + 64].contiguous()
        ys, ms, rs, _ = kd.layer_norm_forward(p, w)
        assert torch.equal(ys, y[a:a + 64]) and torch.equal(ms, mean[a:a + 64])
        assert torch.equal(kd.layer_norm_backward(p, p, w, None, ms, rs)[0], dx[a:a + 64])


@pytest.mark.parametrize("kept", [None, "int8"])
@pytest.mark.parametrize("d", [72, 1000, 2048, 9216, 16385])
def test_masked_rows_get_no_gradient_whatever_the_weight_holds(d, kept):
    T = 9
    for dtype in R.TYPES:
        say(f"layer norm {dtype} d={d} kept={kept}")
        x, mask = R.make_rows(T, d, dtype, d, masked=0.4)
        x, mask = x.cuda(), mask.cuda()
        w = torch.ones(d, dtype=dtype, device="cuda")
        w[d // 2], w[d - 1] = float("inf"), float("nan")
        y, mean, rstd, k = kd.layer_norm_forward(x, w, None, mask, checkpoint=kept)
        args = (torch.randn(T, d, device="cuda").to(dtype), None if k else x, w, mask, mean, rstd, k)
        dx, dw, db = kd.layer_norm_backward(*args)
        off = mask == 0
        alone = kd.layer_norm_backward(*args, want=(True, False, False))[0]
        assert torch.equal(alone[off], dx[off])
        assert bool((y[off] == 0).all()) and bool((dx[off] == 0).all())
        assert bool(dx[~off].isnan().all()) and bool(dw.isfinite().all()) and bool(db.isfinite().all())

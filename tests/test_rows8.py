"""Rows in 8 bits against their exact definition, bit for bit."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests import layers_util as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 31), (2, 32), (70, 33), (5, 129), (33, 1000), (64, 1337), (9, 4096), (4, 8200), (3, 16384),
          (2, 16385), (2, 40007)]
KINDS = ["int8", "e4m3"]


def compare(x, kind, group):
    q, scale = kd.quantize_rows(x.cuda(), kind, group)
    wq, ws = R.rows_reference(x, kind, group)
    assert torch.equal(scale.cpu().nan_to_num(-1.0), ws.nan_to_num(-1.0)), "scale"
    assert torch.equal(scale.cpu().isnan(), ws.isnan())
    got = q.cpu().double()
    wrong = (got != wq).nonzero()
    assert len(wrong) == 0, f"{len(wrong)} values, first {wrong[0].tolist()}: {got[tuple(wrong[0])]} for {wq[tuple(wrong[0])]}"
    for dtype in R.TYPES:
        back = kd.dequantize_rows(q, scale, group, dtype).cpu()
        want = R.rows_values(wq, ws, group).float().to(dtype)  # one product in 32 bits, then the type's rounding
        assert torch.equal(back.isnan(), want.isnan()) and torch.equal(back.nan_to_num(), want.nan_to_num()), dtype


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", R.TYPES)
def test_shapes(dtype, kind, group):
    for T, d in SHAPES:
        say(f"rows {dtype} {kind} group={group} T={T} d={d}")
        x = (torch.randn(T, d, generator=R.gen(T * d + group)) * torch.rand(T, 1, generator=R.gen(7)) * 3).to(dtype)
        compare(x, kind, group)


@pytest.mark.parametrize("kind", KINDS)
def test_whole_rows_that_share_a_workgroup_and_wide_ones(kind):
    for T, d in ((17, 130), (9, 256), (5, 520), (16387, 600), (7, 1024), (3, 4608), (3, 6145), (3, 9216)):
        say(f"rows {kind} T={T} d={d}")
        for dtype in R.TYPES:
            compare(torch.randn(T, d, generator=R.gen(T)).to(dtype), kind, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_next_to_the_middle_of_two_steps(kind):
    """Values whose quotient is a tie, and their neighbours on both sides: rounding must see the exact quotient."""
    top = 127.0 if kind == "int8" else 448.0
    if kind == "int8":
        mids = torch.arange(-126.5, 127, 1.0, dtype=torch.float64)
    else:
        grid = R.e4m3_grid()
        mids = (grid[1:] + grid[:-1]) / 2
        mids = torch.cat([-mids, mids])
    rows = []
    for k in range(200):
        s = torch.rand((), generator=R.gen(k), dtype=torch.float64) * 2.0 ** ((k % 40) - 20)
        scale = ((s * top).float().double() / top).float().double()
        at = (mids * scale).float()
        near = torch.stack([at, torch.nextafter(at, at * 2), torch.nextafter(at, at * 0)]).flatten()
        rows.append(torch.cat([(s * top).float()[None], near.clamp(-float((s * top).float()), float((s * top).float()))]))
    x = torch.stack(rows)
    say(f"rows {kind}: {x.numel()} values at ties")
    compare(x, kind, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_ties_go_to_even(kind):
    top = 127.0 if kind == "int8" else 448.0
    for e in (-20, 0, 9):
        v = torch.arange(-126.5, 127, 1.0) if kind == "int8" else ((R.e4m3_grid()[1:] + R.e4m3_grid()[:-1]) / 2).float()
        x = torch.cat([torch.tensor([top]), v])[None] * 2.0 ** e
        compare(x, kind, 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [0, 32])
def test_small_large_and_not_finite(kind, group):
    g = R.gen(3)
    base = torch.randn(12, 96, generator=g)
    x = base.clone()
    x[0] = 0
    x[1] = -0.0
    x[2] *= 1e-38
    x[3] *= 1e-40  # subnormal
    x[4] = 0
    x[4, 5] = 2.0 ** -149  # a scale that rounds to 0
    x[5] *= 1e38 / 5
    x[6, 40] = float("inf")
    x[7, 3] = float("-inf")
    x[8, 95] = float("nan")
    x[9] = 0
    x[9, 70] = torch.finfo(torch.float32).max
    x[10] = torch.linspace(-1e-30, 1e-30, 96)
    x[11, :64] *= 2.0 ** -95
    compare(x, kind, group)
    compare(x.to(torch.float16), kind, group)
    compare(x.to(torch.bfloat16), kind, group)


@pytest.mark.parametrize("group", [0, 32])
def test_scales_below_the_normal_range(group):
    """448 j + 224 smallest steps of float32: a scale in the middle of two, whose even one it has to be."""
    j = torch.cat([torch.arange(0, 40), torch.randint(0, 1 << 16, (200,), generator=R.gen(1)), torch.arange((1 << 23) - 9, (1 << 23) + 9)])
    k = (448 * j + 224).double()
    k = torch.cat([k, k + 1, k - 1, k + 224])
    k = k[k == k.float().double()]
    say(f"rows e4m3 group={group}: {len(k)} scales")
    x = (k[:, None] * torch.linspace(1, -1, 32, dtype=torch.float64) * 2.0 ** -149).float()
    assert bool((x[:, 0].double() == k * 2.0 ** -149).all())
    for kind in ("e4m3", "int8"):
        compare(x, kind, group)


def test_every_value_of_a_16_bit_type():
    """All finite bfloat16 and float16 values with a scale each."""
    for dtype in (torch.bfloat16, torch.float16):
        v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
        v = v[torch.isfinite(v)]
        x = v[: v.numel() // 64 * 64].reshape(-1, 64)
        for kind in KINDS:
            compare(x, kind, 32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_ratio_of_a_16_bit_types_values(dtype, kind):
    """Every significand as the largest of its group and every one below it in 12 binades: all quotients that such
    values can have, ties and the nearest to ties among them."""
    n = 128 if dtype == torch.bfloat16 else 1024
    sig = torch.arange(n, 2 * n, dtype=torch.float64)
    below = torch.cat([sig / n * 2.0 ** -e for e in range(12)])
    below[1::2] *= -1
    for part in range(0, n, 256):
        top = sig[part:part + 256, None] / n
        x = torch.cat([top, torch.where(below.abs() < top, below, 0)], 1) * (1 if dtype == torch.float16 else 2.0 ** -40)
        say(f"rows {dtype} {kind}: {x.numel()} values from significand {part}")
        assert torch.equal(x, x.to(dtype).double())
        compare(x.to(dtype), kind, 0)


def test_nothing_and_offsets_beyond_32_bits():
    q, s = kd.quantize_rows(torch.empty(0, 64, device="cuda"), "int8", 32)
    assert q.shape == (0, 64) and s.shape == (0, 2) and kd.dequantize_rows(q, s, 32).shape == (0, 64)
    T, d = 1100000, 4096
    say(f"rows T={T} d={d}")
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    q, s = kd.quantize_rows(x, "int8", 128)
    back = kd.dequantize_rows(q, s, 128)
    for a in (0, T // 2, T - 64):
        part = kd.quantize_rows(x[a:a + 64].contiguous(), "int8", 128)
        assert torch.equal(q[a:a + 64], part[0]) and torch.equal(s[a:a + 64], part[1])
        assert torch.equal(back[a:a + 64], kd.dequantize_rows(*part, 128))


# ------------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("kind", KINDS)
def test_checkpoint_gives_the_gradients_at_what_8_bits_hold(kind):
    g = R.gen(1)
    x = torch.randn(2, 33, 70, generator=g).cuda().requires_grad_(True)
    w = torch.randn(70, 20, generator=g).cuda().requires_grad_(True)
    b = torch.randn(20, generator=g).cuda().requires_grad_(True)  # from elsewhere

    def block(x, w, k):
        return torch.tanh(x @ w) * k + b

    up = torch.randn(2, 33, 20, generator=g).cuda()
    y = kd.checkpoint_8bit(block, x, w, 0.5, kind=kind, group=32)
    assert torch.equal(y, block(x, w, 0.5))  # the forward pass sees x itself
    y.backward(up)
    q, s = kd.quantize_rows(x.detach().reshape(-1, 70), kind, 32)
    xd = kd.dequantize_rows(q, s, 32, torch.float32).reshape(x.shape).requires_grad_(True)
    wd = w.detach().clone().requires_grad_(True)
    dx, dw, db = torch.autograd.grad(block(xd, wd, 0.5), (xd, wd, b), up)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw) and torch.equal(b.grad, db)


def test_checkpoint_of_several_outputs_and_of_nothing_to_keep():
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    w = torch.randn(64, 64, device="cuda", requires_grad=True)
    a, b = kd.checkpoint_8bit(lambda x: (x * 2, x @ w), x)
    (dx,) = torch.autograd.grad(b.sum(), x)
    torch.testing.assert_close(dx, torch.ones(8, 64, device="cuda") @ w.t(), rtol=1e-5, atol=1e-5)
    y = kd.checkpoint_8bit(lambda x: x @ w, x.detach())  # only w, from elsewhere, needs a gradient
    assert torch.autograd.grad(y.sum(), w)[0].shape == w.shape
    with torch.no_grad():
        assert not kd.checkpoint_8bit(lambda x: x @ w, x).requires_grad
    a, b = kd.checkpoint_8bit(lambda x: [x * 2, x * 3], x[:0])  # no rows, a list of outputs
    assert torch.autograd.grad(a.sum() + b.sum(), x)[0].shape == x.shape


def test_checkpoint_refuses_what_changed_since():
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    w = torch.randn(64, 64, device="cuda")
    y = kd.checkpoint_8bit(lambda x, w: x @ w, x, w)
    w.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with pytest.raises(TypeError, match="last axis"):
        kd.checkpoint_8bit(abs, torch.ones(3, 0))


def test_checkpoint_draws_the_same_random_numbers_again():
    x = torch.randn(64, 256, device="cuda", requires_grad=True)
    fn = lambda x: torch.nn.functional.dropout(x, 0.5) * 3  # noqa: E731
    torch.manual_seed(5)
    y = kd.checkpoint_8bit(fn, x)
    torch.rand(7, device="cuda")
    state = torch.cuda.get_rng_state()
    (dx,) = torch.autograd.grad(y.sum(), x)
    assert torch.equal(torch.cuda.get_rng_state(), state)
    assert torch.equal(dx != 0, y != 0) and 0.4 < (y != 0).float().mean() < 0.6


def test_checkpoint_in_a_captured_graph():
    """Forward and backward captured together; a function that draws random numbers is refused there."""
    say("checkpoint_8bit captured")
    x, up = torch.randn(64, 256, device="cuda"), torch.randn(64, 256, device="cuda")
    fn = lambda x: torch.tanh(x) * x  # noqa: E731

    def step():
        leaf = x.detach().requires_grad_(True)
        y = kd.checkpoint_8bit(fn, leaf, kind="e4m3", group=32)
        return torch.autograd.grad(y, leaf, up)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="random numbers"):
            kd.checkpoint_8bit(lambda x: torch.nn.functional.dropout(x, 0.5), x.detach().requires_grad_(True))
        dx = step()
    for _ in range(3):
        x.normal_()
        graph.replay()
        got = dx.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, step())


def test_checkpoint_runs_again_under_the_same_autocast():
    x, w = (torch.randn(64, 64, device="cuda", requires_grad=True) for _ in range(2))
    types = []

    def fn(x):
        types.append((x @ w).dtype)
        return x @ w

    with torch.autocast("cuda", torch.bfloat16):
        y = kd.checkpoint_8bit(fn, x, kind="e4m3", group=32)
    y.float().sum().backward()
    assert types == [torch.bfloat16] * 2 and x.grad.dtype == w.grad.dtype == torch.float32

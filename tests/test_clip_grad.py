"""The global gradient norm and clipping on the GPU against the 64-bit form."""
import math

import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import say
from tests.policy_util import U32, half_step

pytestmark = pytest.mark.gpu
f32, bf, f16 = torch.float32, torch.bfloat16, torch.float16


def norm64(tensors):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in tensors))


def check(tensors, max_norm, out=None):
    """The norm is a 64-bit sum rounded once; each output is one 32-bit product (of a factor that is itself rounded
    once) rounded once to its type, below the type's smallest normal number by at most one step there."""
    want = norm64(tensors)
    before = [t.clone() for t in tensors]
    norm = kd.clip_grad_norm(tensors, max_norm, out)
    assert norm.shape == () and abs(float(norm) - want) <= 2 * U32 * want
    c = min(1.0, max_norm / (want + 1e-6))
    for b, o in zip(before, tensors if out is None else out):
        w = b.double() * c
        tiny = torch.finfo(o.dtype).smallest_normal * torch.finfo(o.dtype).eps
        err = (o.double() - w).abs() - (half_step(o.dtype) * (1 + 4 * U32) + 4 * U32) * w.abs() - tiny
        assert (err <= 0).all(), float(err.max())
    if out is not None:
        assert all(torch.equal(t, b) for t, b in zip(tensors, before))


def rand(n, dtype, seed=0, scale=1e-2):
    g = torch.Generator(device="cuda").manual_seed(seed + n)
    return (scale * torch.randn(n, generator=g, device="cuda")).to(dtype)


@pytest.mark.parametrize("dtype", [f32, bf, f16])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 255, 4096, 16383, 16384, 16385, 100003, 5000000])
def test_one_tensor(n, dtype):
    say(f"clip one tensor n={n} {dtype}")
    for ratio in (0.25, 3.0):
        x = rand(n, dtype)
        check([x], ratio * norm64([x]))


@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 8])
@pytest.mark.parametrize("dtype", [f32, bf, f16])
def test_unaligned_views(offset, dtype):
    """Views of a bucket that start anywhere, beside elements that must stay."""
    flat = rand(40000, dtype)
    keep = flat.clone()
    a, b = flat[offset:offset + 17001], flat[20000 + offset:39000]
    check([a, b], 0.5 * norm64([a, b]))
    for lo, hi in ((0, offset), (offset + 17001, 20000 + offset), (39000, 40000)):
        assert torch.equal(flat[lo:hi], keep[lo:hi])


@pytest.mark.parametrize("count", [2, 20, 95, 96, 97, 131, 132, 133, 188, 189, 300, 400])
def test_many_tensors_of_all_types(count):
    """More tensors than one launch takes, empty ones among them."""
    types = [f32, bf, f16]
    ts = [rand((37 * i * i) % 5000 if i % 11 else 0, types[i % 3], i) for i in range(count)]
    check(ts, 0.3 * norm64(ts))
    outs = [torch.empty_like(t, dtype=types[(i + i // 3) % 3]) for i, t in enumerate(ts)]
    check(ts, 0.7 * norm64(ts), outs)


def test_strides_and_shapes():
    a = rand(6000, f32).view(60, 100).t()
    b = rand(2400, bf).view(2, 30, 40).permute(2, 0, 1)
    c = rand(1, f32).view(())
    check([a, b, c], 0.1)
    outs = [torch.empty_like(a), torch.empty_like(b, dtype=f32), torch.empty_like(c)]
    assert outs[0].stride() == a.stride() and outs[1].stride() == b.stride()
    check([a, b, c], 0.05, outs)


def test_nothing_is_written_below_the_limit():
    x = rand(100000, bf)
    keep = x.clone()
    norm = kd.clip_grad_norm_([x], 1e9)
    assert torch.equal(x, keep) and float(norm) > 0
    kd.clip_grad_norm_([x], math.inf)
    assert torch.equal(x, keep)
    kd.clip_grad_norm_([x], 0.0)
    assert (x == 0).all()


def test_large_and_small_values():
    """Squares beyond the 32-bit range at both ends."""
    big, small = torch.full((1000,), 1e30, device="cuda"), torch.full((1000,), 1e-30, device="cuda")
    assert abs(float(kd.clip_grad_norm([big], math.inf)) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    assert abs(float(kd.clip_grad_norm([small], math.inf)) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6
    check([big, small], 1.0)
    h = torch.full((70000,), 65504.0, device="cuda", dtype=f16)
    check([h], 10.0)


def test_not_finite():
    for bad, rest in ((math.nan, math.nan), (math.inf, 0.0)):
        x, y = rand(50000, f32), rand(100, bf)
        x[12345] = bad
        norm = kd.clip_grad_norm_([x, y], 1.0)
        assert not math.isfinite(float(norm)) and math.isnan(float(x[12345]))
        assert bool(torch.isnan(y).all()) if math.isnan(rest) else bool((y == 0).all())
        z = rand(10, f32)
        z[3] = bad
        keep = z.clone()
        kd.clip_grad_norm_([z], math.inf)
        assert torch.equal(z[:3], keep[:3])


def test_parts_of_a_norm():
    """Two ranks' parts, added up before the clip, give what one call over all gives."""
    ts = [rand(30000, f32, 1), rand(40000, bf, 2), rand(999, f16, 3)]
    whole = [t.clone() for t in ts]
    norm = kd.clip_grad_norm_(whole, 0.4)
    total = kd.grad_sumsq(ts[:1]) + kd.grad_sumsq(ts[1:])
    for part in (ts[:1], ts[1:]):
        n = kd.clip_grad_norm_(part, 0.4, sumsq=total)
        assert abs(float(n) - float(norm)) <= 2 * U32 * float(norm)
    for a, b in zip(whole, ts):
        assert torch.equal(a, b)


def test_repeatable_and_graph():
    ts = [rand(300000, f32, 1), rand(100, bf, 2)]
    outs = [torch.empty_like(t) for t in ts]
    graph = torch.cuda.CUDAGraph()
    kd.clip_grad_norm(ts, 0.5, outs)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        n = kd.clip_grad_norm(ts, 0.5, outs)
    for k in range(3):
        ts[0].mul_(1.3)
        other = [torch.empty_like(t) for t in ts]
        want = kd.clip_grad_norm(ts, 0.5, other)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, want) and all(torch.equal(x, y) for x, y in zip(outs, other)), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = kd.clip_grad_norm(ts, 0.5, outs)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    x, y = torch.ones(100, device="cuda"), torch.ones(100, device="cuda")
    for bad, err in (([x, x], kd.KDError), ([x, x[50:]], kd.KDError), ([x[::2]], ValueError), ([x, y.cpu()], ValueError),
                     ([x, torch.ones(3, dtype=torch.int32, device="cuda")], TypeError)):
        with pytest.raises(err):
            kd.clip_grad_norm_(bad, 1.0)
    for out in ([y[:50]], [y, y], [x[1:]], [torch.ones(100, 2, device="cuda")]):
        with pytest.raises((ValueError, kd.KDError)):
            kd.clip_grad_norm([x], 1.0, out)
    with pytest.raises(ValueError):
        kd.clip_grad_norm([x, None], 1.0, [y, y])
    a = torch.ones(4, 5, device="cuda")
    with pytest.raises(ValueError, match="strides"):
        kd.clip_grad_norm([a], 1.0, [torch.ones(5, 4, device="cuda").t()])
    with pytest.raises(kd.KDError):
        kd.clip_grad_norm([x], -1.0)
    assert (x == 1).all() and (y == 1).all()


def test_no_gradients_and_generators():
    x = torch.full((9,), 2.0, device="cuda")
    assert float(kd.clip_grad_norm_((t for t in (None, x)), 1.0)) == 6.0
    assert abs(float(x.norm()) - 1.0) < 1e-5
    assert float(kd.clip_grad_norm_([torch.empty(0, device="cuda")], 1.0)) == 0.0


def test_autograd_sees_the_change():
    """A tensor clipped in place between a forward and its backward is refused there."""
    w = torch.ones(50, device="cuda", requires_grad=True)
    x = torch.full((50,), 3.0, device="cuda")
    y = (w * x).sum()
    kd.clip_grad_norm_([x], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()

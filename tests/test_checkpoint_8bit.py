"""checkpoint_8bit's part that is torch alone, on the CPU: with the rounding to 8 bits left out, every gradient has to be
that of the function itself."""
import collections
import dataclasses

import pytest
import torch
import torch.nn.functional as F

kd = pytest.importorskip("chunked_kl_loss_logit_amd")
L = kd.layers


@pytest.fixture(autouse=True)
def exact_rows(monkeypatch):
    """x itself in the place of its 8 bits."""
    monkeypatch.setattr(L, "quantize_rows", lambda x, kind, group: (x.clone(), torch.ones(1)))
    monkeypatch.setattr(L, "dequantize_rows", lambda q, scale, group, dtype: q.clone())


def leaves(*shapes):
    g = torch.Generator().manual_seed(len(shapes))
    return [torch.randn(*s, generator=g).requires_grad_(True) for s in shapes]


# ------------------------------------------------------------------ random numbers
@pytest.mark.parametrize("fn", [
    lambda x: F.dropout(x, 0.5) * x,
    lambda x: x * torch.rand(x.shape),
    lambda x: [x * torch.bernoulli(torch.full(x.shape, 0.5)), x * 2][0],
], ids=["dropout", "rand", "bernoulli"])
def test_random_numbers_are_drawn_alike_again(fn):
    (x,) = leaves((64, 32))
    torch.manual_seed(3)
    y = kd.checkpoint_8bit(fn, x)
    after = torch.get_rng_state()
    torch.rand(5)  # what is drawn between the two passes
    between = torch.get_rng_state()
    (dx,) = torch.autograd.grad(y.sum(), x)
    assert torch.equal(torch.get_rng_state(), between), "the backward pass moved the random state"
    torch.manual_seed(3)
    want = fn(x)
    assert torch.equal(y, want) and torch.equal(torch.get_rng_state(), after)
    assert torch.equal(dx, torch.autograd.grad(want.sum(), x)[0])


def test_random_numbers_drawn_aside_and_from_a_generator_of_its_own():
    (x,) = leaves((64, 32))

    def aside(x):  # the state is the same before and after
        with torch.random.fork_rng(devices=[]):
            return F.dropout(x, 0.5) * x

    def own(x, g):
        return x * x * torch.rand(x.shape, generator=g)

    for fn, others in ((aside, ()), (own, (torch.Generator().manual_seed(7),))):
        torch.manual_seed(3)
        y = kd.checkpoint_8bit(fn, x, *others)
        torch.rand(5)
        for g in others:
            torch.rand(5, generator=g)
        (dx,) = torch.autograd.grad(y.sum(), x)
        torch.manual_seed(3)
        want = fn(x, *(g.manual_seed(7) for g in others))
        assert torch.equal(y, want) and torch.equal(dx, torch.autograd.grad(want.sum(), x)[0])


def test_random_state_comes_back_after_an_error():
    (x,) = leaves((4, 8))
    runs = []

    def fn(x):
        runs.append(torch.rand(()).item())
        if len(runs) > 1:
            raise KeyError("again")
        return x * 2

    y = kd.checkpoint_8bit(fn, x)
    torch.rand(3)
    state = torch.get_rng_state()
    with pytest.raises(KeyError):
        y.sum().backward()
    assert runs[0] == runs[1] and torch.equal(torch.get_rng_state(), state)


def test_random_numbers_in_a_captured_graph_are_refused(monkeypatch):
    """The states of a graph under capture can be neither read nor set."""
    x, q = leaves((4, 8), (1, 2, 4, 8))
    monkeypatch.setattr(L, "_capturing", lambda: True)
    for fn in (lambda x: F.dropout(x, 0.5), lambda x: x * torch.rand(x.shape), lambda x: x * torch.randn_like(x)):
        with pytest.raises(RuntimeError, match="random numbers"):
            kd.checkpoint_8bit(fn, x)
    for fn, t in ((lambda x: torch.tanh(x) + F.dropout(x, 0.5, training=False), x),
                  (lambda q: F.scaled_dot_product_attention(q, q, q, dropout_p=0.0), q)):
        y = kd.checkpoint_8bit(fn, t)
        assert torch.equal(torch.autograd.grad(y.sum(), t)[0], torch.autograd.grad(fn(t).sum(), t)[0])


# ------------------------------------------------------------------ autocast
def seen(into):
    def fn(x, w):
        y = x @ w
        into.append((y.dtype, torch.is_autocast_enabled("cpu"), torch.is_autocast_cache_enabled()))
        return y
    return fn


@pytest.mark.parametrize("inside", [True, False], ids=["backward inside", "backward outside"])
@pytest.mark.parametrize("cache", [True, False])
def test_autocast_is_the_same_both_times(inside, cache):
    x, w = leaves((4, 8), (8, 8))
    types = []
    with torch.autocast("cpu", torch.bfloat16, cache_enabled=cache):
        y = kd.checkpoint_8bit(seen(types), x, w)
        if inside:
            got = torch.autograd.grad(y.float().sum(), (x, w))
        want = torch.autograd.grad((x @ w).float().sum(), (x, w))
    if not inside:
        got = torch.autograd.grad(y.float().sum(), (x, w))
    assert types == [(torch.bfloat16, True, cache)] * 2
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autocast_of_the_backward_pass_is_not_the_functions():
    x, w = leaves((4, 8), (8, 8))
    types = []
    y = kd.checkpoint_8bit(seen(types), x, w)
    with torch.autocast("cpu", torch.bfloat16):
        y.sum().backward()
    assert [t[:2] for t in types] == [(torch.float32, False)] * 2


@pytest.mark.parametrize("around", [True, False])
def test_a_weight_used_before_and_behind_under_autocast_keeps_its_gradient(around):
    """Autocast remembers the casts of leaves: one made while nothing is recorded has no gradient."""
    g = torch.Generator().manual_seed(1)  # small whole numbers: nothing is rounded
    x, w = (torch.randint(-3, 4, s, generator=g).float().requires_grad_(True) for s in ((4, 8), (8, 8)))

    def fn(x):
        with torch.autocast("cpu", torch.bfloat16):
            return x @ w

    with torch.autocast("cpu", torch.bfloat16, enabled=around):
        y = kd.checkpoint_8bit(fn, x)
        with torch.autocast("cpu", torch.bfloat16):
            z = x @ w
        (y.float().sum() + 2 * z.float().sum()).backward()
        dx, dw = torch.autograd.grad(3 * fn(x).float().sum(), (x, w))
    assert torch.equal(w.grad, dw) and torch.equal(x.grad, dx)


# ------------------------------------------------------------------ tensors from elsewhere
def test_gradients_asked_for_by_name_leave_the_others_alone():
    x, w, v = leaves((4, 8), (8, 8), (8, 8))
    fn = lambda x, v: torch.tanh(x @ w) @ v  # noqa: E731
    y = kd.checkpoint_8bit(fn, x, v)
    want = torch.autograd.grad(fn(x, v).sum(), (x, v, w))
    got = torch.autograd.grad(y.sum(), (x, v), retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(torch.autograd.grad(y.sum(), x, retain_graph=True)[0], want[0])
    assert x.grad is None and v.grad is None and w.grad is None
    y.sum().backward()
    assert all(torch.equal(t.grad, g) for t, g in zip((x, v, w), want))


def test_a_checkpoint_in_a_checkpoint():
    x, w, v = leaves((4, 8), (8, 8), (8, 8))
    inner = lambda x: torch.tanh(x @ w)  # noqa: E731
    y = kd.checkpoint_8bit(lambda x, v: kd.checkpoint_8bit(inner, x @ v) @ v, x, v)
    want = torch.autograd.grad((inner(x @ v) @ v).sum(), (x, v, w))
    got = torch.autograd.grad(y.sum(), (x, v), retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and w.grad is None
    y.sum().backward()
    assert all(torch.equal(t.grad, g) for t, g in zip((x, v, w), want))


def test_tensors_from_elsewhere_that_are_asked_for_are_refused():
    x, w = leaves((4, 8), (8, 8))
    y = kd.checkpoint_8bit(lambda x: x @ w, x)
    for inputs in ([x, w], [x]):  # which of the two it is, the backward pass does not see
        with pytest.raises(RuntimeError, match="among the others"):
            y.sum().backward(inputs=inputs, retain_graph=True)
    with pytest.raises(RuntimeError, match="among the others"):  # w also has a use that torch knows of
        torch.autograd.grad(y.sum() + w.sum(), (x, w), retain_graph=True)
    h = w * 2
    z = kd.checkpoint_8bit(lambda x: x @ h, x)
    with pytest.raises(RuntimeError, match="among the others"):
        torch.autograd.grad(z.sum() + h.sum(), (x, h), retain_graph=True)
    assert w.grad is None and x.grad is None
    f = w.detach()
    kd.checkpoint_8bit(lambda x: x @ f, x).sum().backward(inputs=[x])  # nothing else there
    assert torch.equal(x.grad, torch.autograd.grad((x @ f).sum(), x)[0])


def test_a_computed_tensor_among_the_others():
    x, w = leaves((4, 8), (8, 8))
    h = torch.tanh(w)
    y = kd.checkpoint_8bit(lambda x, h: x @ h, x, h) + kd.checkpoint_8bit(lambda x, h: x * h[:4], x, h)
    want = torch.autograd.grad((x @ h + x * h[:4]).sum() + (h * h).sum(), (x, w), retain_graph=True)
    (y.sum() + (h * h).sum()).backward()
    assert torch.equal(x.grad, want[0])
    torch.testing.assert_close(w.grad, want[1], rtol=0, atol=16 * 2.0 ** -24 * 40)  # a sum of 3 shares below 40, in another order


# ------------------------------------------------------------------ what fn returns
Pair = collections.namedtuple("Pair", "y z")


@dataclasses.dataclass
class Held:
    y: torch.Tensor


def test_outputs_that_hold_tensors_are_refused():
    (x,) = leaves((4, 8))
    for fn, name in ((lambda x: Held(x * 2), "Held"), (lambda x: (x, Held(x * 2)), "Held"), (lambda x: {"y": x}, "dict"),
                     (lambda x: [x, (x * 2,)], "tuple"), (lambda x: Pair(x, {1: x}), "dict"), (lambda x: (x, object()), "object")):
        with pytest.raises(TypeError, match=f"got a {name}"):
            kd.checkpoint_8bit(fn, x)


def test_outputs_come_back_as_what_they_are():
    (x,) = leaves((4, 8))
    y = kd.checkpoint_8bit(lambda x: Pair(x * 2, x.sum(0)), x)
    assert type(y) is Pair and torch.equal(torch.autograd.grad(y.z.sum() + y.y.sum(), x)[0], torch.full((4, 8), 3.0))
    y = kd.checkpoint_8bit(lambda x: torch.max(x, 1), x)
    assert torch.equal(y.indices, x.argmax(1)) and y.values.requires_grad
    assert torch.equal(torch.autograd.grad(y.values.sum(), x)[0].argmax(1), y.indices)
    a, none, n, s, flag = kd.checkpoint_8bit(lambda x: (x * 2, None, 3, "s", True), x)
    assert none is None and (n, s, flag) == (3, "s", True) and a.requires_grad
    assert type(kd.checkpoint_8bit(lambda x: (x * 2, x), x)) is tuple
    assert kd.checkpoint_8bit(lambda x: None, x) is None and kd.checkpoint_8bit(lambda x: 3.0, x) == 3.0


def test_tensors_from_elsewhere_that_are_returned_stay_what_they_are():
    x, w = leaves((4, 8), (8, 8))
    buffer, h = torch.ones(3), w * 2
    y, a, b, c = kd.checkpoint_8bit(lambda x: (x @ w, w, buffer, h), x)
    assert w.is_leaf and w.grad_fn is None and not buffer.requires_grad and h.grad_fn.name() == "MulBackward0"
    assert torch.equal(a, w) and torch.equal(b, buffer) and torch.equal(c, h)
    want = torch.autograd.grad((x @ w).sum() + (w * w).sum(), (x, w))
    (y.sum() + (a * w.detach()).sum() * 2).backward()
    assert torch.equal(x.grad, want[0])
    torch.testing.assert_close(w.grad, want[1], rtol=2.0 ** -22, atol=2.0 ** -20)  # two shares below 16, added up once
    x.grad = None
    y, same = kd.checkpoint_8bit(lambda x: (x * 2, x), x)
    (y.sum() + 3 * same.sum()).backward()
    assert x.is_leaf and torch.equal(x.grad, torch.full((4, 8), 5.0))

"""Token embeddings and their gradient against plain forms in 64 bits: rows of a table and columns of a tied head."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests import layers_util as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
cuda = lambda t: None if t is None else t.cuda()  # noqa: E731

SHAPES = [  # T, V, d
    (1, 1, 1), (1, 50, 7), (5, 32000, 64), (64, 300, 96), (65, 64, 513), (130, 1000, 1037), (777, 129, 520),
    (1025, 511, 40), (4097, 5000, 24), (2000, 70000, 16),
]


def layout(E, tied):
    return E.t().contiguous() if tied else E


@pytest.mark.parametrize("dtype", R.TYPES)
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("T,V,d", SHAPES)
def test_forward(T, V, d, tied, dtype):
    say(f"embedding forward {dtype} tied={tied} T={T} V={V} d={d}")
    E = torch.randn(V, d, generator=R.gen(T + d)).to(dtype)
    for masked in (0.0, 0.4):
        tokens, mask = R.make_tokens(T, V, T, masked)
        if T > 20:
            tokens[T // 3], tokens[T // 2] = V, -1  # no tokens of this vocabulary, masked or not
        out = kd.embedding_forward(tokens.cuda(), layout(E, tied).cuda(), cuda(mask), 1.7, tied=tied)
        want, bound = R.embedding_reference(tokens, E, mask, float(torch.tensor(1.7)))
        R.check(out, want, bound, f"masked={masked}")


@pytest.mark.parametrize("dtype,grad_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                              (torch.float32, torch.float32), (torch.float16, torch.float16),
                                              (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("T,V,d", SHAPES)
def test_backward(T, V, d, tied, dtype, grad_dtype):
    say(f"embedding backward {dtype} to {grad_dtype} tied={tied} T={T} V={V} d={d}")
    grad = torch.randn(T, d, generator=R.gen(T + d)).to(dtype)
    s = float(torch.tensor(0.37))
    for masked in (0.0, 0.4):
        tokens, mask = R.make_tokens(T, V, T + 1, masked)
        if mask is not None:
            grad[mask == 0] = float("nan")  # never read
        if T > 20:
            tokens[T // 3], tokens[T // 2] = V, -1
        args = (grad.cuda(), tokens.cuda(), V, cuda(mask), 0.37)
        got = kd.embedding_backward(*args, tied=tied, grad_dtype=grad_dtype)
        assert got.dtype == grad_dtype and got.shape == ((d, V) if tied else (V, d))
        want, bound = R.embedding_grad_reference(grad, tokens, mask, s, V, grad_dtype)
        R.check(got.t() if tied else got, want, bound, f"masked={masked}")
        assert torch.equal(got, kd.embedding_backward(*args, tied=tied, grad_dtype=grad_dtype)), "not the same bits"
        was = torch.randn(V, d, generator=R.gen(3)).to(grad_dtype)
        out = layout(was, tied).cuda()
        assert kd.embedding_backward(*args, tied=tied, out=out) is out
        want, bound = R.embedding_grad_reference(grad, tokens, mask, s, V, grad_dtype, was)
        R.check(out.t() if tied else out, want, bound, f"accumulate masked={masked}")
        seen = torch.zeros(V, dtype=torch.bool)
        ok = R.valid_rows(mask, T) & (tokens >= 0) & (tokens < V)
        seen[tokens[ok].long()] = True
        left = (out.t() if tied else out).cpu()[~seen]
        assert torch.equal(left, was[~seen]), "rows of tokens that do not occur"


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("T", [1023, 1024, 2049, 16384, 16385, 32767, 32768, 32769, 50001])
@pytest.mark.parametrize("V", [3, 300, 5000, 300001])
def test_backward_of_many_tokens(T, V, tied):
    """Chunks of a workgroup's sort, the passes over many, keys of one to three digits, runs over many pieces."""
    say(f"embedding backward T={T} V={V} tied={tied}")
    d = 8
    grad = torch.randn(T, d, generator=R.gen(T))
    tokens, mask = R.make_tokens(T, V, T + V, 0.1)
    got = kd.embedding_backward(grad.cuda(), tokens.cuda(), V, mask.cuda(), tied=tied)
    want, bound = R.embedding_grad_reference(grad, tokens, mask, 1.0, V, torch.float32)
    R.check(got.t() if tied else got, want, bound, "dE")


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("T", [1, 15, 16, 17, 33, 20000])
def test_one_token_only(T, tied):
    """Every row meets in one token: its run goes through all pieces."""
    say(f"embedding backward, one token T={T} tied={tied}")
    grad = torch.randn(T, 40, generator=R.gen(T))
    tokens = torch.full((T,), 2, dtype=torch.int32)
    got = kd.embedding_backward(grad.cuda(), tokens.cuda(), 5, tied=tied)
    want, bound = R.embedding_grad_reference(grad, tokens, None, 1.0, 5, torch.float32)
    R.check(got.t() if tied else got, want, bound, "dE")


@pytest.mark.parametrize("tied", [False, True])
def test_nothing_valid(tied):
    """No row at all, and rows that the mask or their tokens leave out."""
    E = torch.randn(9, 12).cuda()
    grad = torch.full((6, 12), float("nan")).cuda()
    for tokens, mask in ((torch.tensor([1, 2, 3, 4, 5, 6]), torch.zeros(6, dtype=torch.uint8)),
                         (torch.tensor([-1, 9, 10, -5, 1 << 30, -(1 << 31)]), None)):
        tokens, mask = tokens.int().cuda(), cuda(mask)
        y = kd.embedding_forward(tokens, E, mask, tied=False)
        assert bool((y == 0).all()) if mask is not None else bool(y.isnan().all())
        got = kd.embedding_backward(grad, tokens, 9, mask, tied=tied)
        assert got.shape == ((12, 9) if tied else (9, 12)) and bool((got == 0).all())
        out = torch.ones_like(got)
        assert bool((kd.embedding_backward(grad, tokens, 9, mask, tied=tied, out=out) == 1).all())
    none = torch.empty(0, dtype=torch.int32).cuda()
    assert kd.embedding_forward(none, E).shape == (0, 12)
    assert bool((kd.embedding_backward(grad[:0], none, 9, tied=tied) == 0).all())
    out = torch.ones(12, 9).cuda() if tied else torch.ones(9, 12).cuda()
    assert bool((kd.embedding_backward(grad[:0], none, 9, tied=tied, out=out) == 1).all())


@pytest.mark.parametrize("tied", [False, True])
def test_autograd(tied):
    """Gradients against the formula's and against differences (the loss is linear in the table: they are exact up to
    the roundings of a sum of T d products)."""
    T, V, d = 50, 30, 24
    tokens, mask = R.make_tokens(T, V, 5, 0.2)
    E = torch.randn(V, d, generator=R.gen(1))
    table = layout(E, tied).cuda().requires_grad_(True)
    up = torch.randn(T, d, generator=R.gen(2))
    y = kd.embedding(tokens.cuda(), table, mask.cuda(), 2.0, tied=tied)
    (g,) = torch.autograd.grad(y, table, up.cuda())
    want, bound = R.embedding_grad_reference(up, tokens, mask, 2.0, V, torch.float32)
    R.check(g.t() if tied else g, want, bound, "dE")
    step = torch.randn(V, d, generator=R.gen(3))
    with torch.no_grad():
        ys = [kd.embedding_forward(tokens.cuda(), layout(E + k * step, tied).cuda(), mask.cuda(), 2.0, tied=tied)
              for k in (-1, 1)]
    diff = ((ys[1] - ys[0]).cpu().double() * up.double()).sum() / 2
    assert abs(diff - (want * step.double()).sum()) <= 16 * R.U32 * (y.detach().cpu().double().abs() * up.double().abs()).sum() \
        + 16 * R.U32 * (want.abs() * step.double().abs()).sum() + 64 * R.U32 * up.double().abs().sum()


def test_slabs_of_a_tied_heads_columns():
    """A row of sums for each token, which pass 1 GiB: the columns are taken in slabs."""
    T, V, d = 300000, 600, 1100
    say(f"embedding backward tied T={T} V={V} d={d}")
    assert kd.kd_embedding_workspace_size(T, V, d, True) < 4 * T * d
    grad = torch.randn(T, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    tokens = torch.randint(0, V, (T,), dtype=torch.int32, generator=R.gen(4)).cuda()
    rows = kd.embedding_backward(grad, tokens, V)  # the same sums, tested above
    assert torch.equal(kd.embedding_backward(grad, tokens, V, tied=True), rows.t())
    out = torch.zeros(d, V, device="cuda")
    assert torch.equal(kd.embedding_backward(grad, tokens, V, tied=True, out=out), rows.t())


def test_offsets_beyond_32_bits():
    """Rows that lie beyond 4 GiB of the table, of the output and of the upstream gradient."""
    T, V, d = 600000, 270000, 8192 // 2
    say(f"embedding T={T} V={V} d={d}")
    E = torch.empty(V, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    tokens = torch.randint(0, V, (T,), dtype=torch.int32, generator=R.gen(4)).cuda()
    y = kd.embedding_forward(tokens, E, scale=1.0)
    for a in (0, T // 2, T - 1000):
        assert torch.equal(y[a:a + 1000], E[tokens[a:a + 1000].long()])
    g = kd.embedding_backward(y, tokens, V)
    n = torch.bincount(tokens.long(), minlength=V)
    for a in (0, V // 2, V - 1000):
        # n times one bf16 row: n - 1 float32 roundings and one to bf16
        want = E[a:a + 1000].double() * n[a:a + 1000, None]
        off = (g[a:a + 1000].double() - want).abs()
        assert bool((off <= want.abs() * (2.0 ** -8 + 64 * R.U32)).all())


def test_more_rows_than_a_launch_has_waves():
    T, V = (1 << 26) + 77, 7
    say(f"embedding T={T} V={V} d=1")
    tokens = torch.randint(-1, V, (T,), dtype=torch.int32, device="cuda",
                           generator=torch.Generator("cuda").manual_seed(1))
    mask = torch.arange(T, device="cuda") % 5 != 0
    E = torch.randn(V, 1, generator=R.gen(2)).to(torch.bfloat16).cuda()
    y = kd.embedding_forward(tokens, E, mask)
    want = torch.cat([E.new_full((1, 1), float("nan")), E])[tokens.long() + 1]
    want[~mask] = 0
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.nan_to_num(), want.nan_to_num())


def test_zeros_in_a_table_of_very_many_rows():
    V = (1 << 28) + 77
    say(f"embedding backward T=3 V={V} d=1")
    out = kd.embedding_backward(torch.ones(3, 1, device="cuda", dtype=torch.bfloat16),
                                torch.tensor([V - 1, 5, V - 1], dtype=torch.int32, device="cuda"), V)
    assert out[V - 1] == 2 and out[5] == 1 and int(torch.count_nonzero(out)) == 2

"""The product of 8-bit integers with scales for tokens and channels against sums in 64 bits."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests import layers_util as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

SHAPES = [  # T, d, V: few rows, rows of one and several blocks, tiles; lengths that are no multiple of anything
    (1, 16, 1), (1, 4096, 300), (3, 144, 65), (31, 128, 64), (32, 1024, 127), (33, 1040, 129), (64, 48, 1000),
    (65, 272, 31), (128, 528, 333), (129, 256, 70), (300, 2064, 515), (1000, 16, 40), (129, 64, 33000),
    (257, 1040, 16500), (1030, 256, 8200), (2049, 304, 4100), (1500, 2000, 5537),
    (2049, 48, 40000), (1030, 272, 20001),  # several tiles a workgroup, of one turn of the ring and of more
]


@pytest.mark.parametrize("dtype", R.TYPES)
@pytest.mark.parametrize("T,d,V", SHAPES)
def test_product(T, d, V, dtype):
    say(f"int8 {dtype} T={T} d={d} V={V}")
    x, sx, w, sw = R.make_int8(T, d, V, T + d + V)
    out = kd.int8_matmul(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), dtype)
    R.check(out, *R.int8_reference(x, sx, w, sw, dtype), "out")
    assert torch.equal(out, kd.int8_matmul(x.cuda(), sx[:, None].cuda(), w.cuda(), sw[:, None].cuda(), dtype))


@pytest.mark.parametrize("T,V", [(5, 70), (300, 16500)])
def test_largest_sums(T, V):
    """The longest contraction of the largest values: 2^17 - 16 products of 2^14 stay below 2^31."""
    d = (1 << 17) - 16
    x = torch.full((T, d), -128, dtype=torch.int8)
    w = torch.full((V, d), -128, dtype=torch.int8)
    one = torch.ones(1)
    out = kd.int8_matmul(x.cuda(), one.expand(T).contiguous().cuda(), w.cuda(), one.expand(V).contiguous().cuda(),
                         torch.float32)
    assert bool((out == float(d * 128 * 128)).all())


def test_no_rows_and_rows_behind_the_last_one():
    x, sx, w, sw = R.make_int8(0, 64, 100, 1)
    assert kd.int8_matmul(x.cuda(), sx.cuda(), w.cuda(), sw.cuda()).shape == (0, 100)
    for T, d, V in ((40, 208, 333), (400, 208, 33001)):  # what lies behind the output stays as it was
        x, sx, w, sw = (t.cuda() for t in R.make_int8(T, d, V, 2))
        buf = torch.full((T * V + 4096,), 7.0, device="cuda")
        ws = torch.empty(max(1, kd.kd_int8_matmul_workspace_size(T, d, V)), dtype=torch.uint8, device="cuda")
        kd.kd_int8_matmul(x, sx, w, sw, buf[:T * V].view(T, V), ws)
        assert bool((buf[T * V:] == 7.0).all())
        assert torch.equal(buf[:T * V].view(T, V), kd.int8_matmul(x, sx, w, sw, torch.float32))


def test_operands_beyond_4_gib():
    T, d, V = 300, 16384, 270000
    say(f"int8 T={T} d={d} V={V}")
    g = torch.Generator("cuda").manual_seed(3)
    w = torch.randint(-127, 128, (V, d), dtype=torch.int8, device="cuda", generator=g)
    x = torch.randint(-127, 128, (T, d), dtype=torch.int8, device="cuda", generator=g)
    sx, sw = torch.rand(T, device="cuda"), torch.rand(V, device="cuda")
    out = kd.int8_matmul(x, sx, w, sw, torch.float32)
    few = kd.int8_matmul(x[:7].contiguous(), sx[:7].contiguous(), w, sw, torch.float32)
    assert torch.equal(out[:7], few)  # both kernels' sums are exact
    for a in (0, V // 2, V - 500):
        part = kd.int8_matmul(x, sx, w[a:a + 500].contiguous(), sw[a:a + 500].contiguous(), torch.float32)
        assert torch.equal(out[:, a:a + 500], part)


def test_head_in_8_bits():
    """From a head and hidden states: off from the exact logits by the two roundings to 8 bits, half a step of each
    row's scale per value."""
    T, d, V = 50, 512, 700
    H, W = torch.randn(T, d, generator=R.gen(1)).bfloat16(), torch.randn(d, V, generator=R.gen(2)).bfloat16()
    q, s = kd.quantize_rows(H.cuda(), "int8", 0)
    wq, ws = kd.quantize_rows(W.t().contiguous().cuda(), "int8", 0)
    z = kd.int8_matmul(q, s, wq, ws, torch.float32).cpu().double()
    s, ws = s.cpu().double(), ws.cpu().double()[:, 0]
    exact = H.double() @ W.double()
    bound = 0.5 * s * W.double().abs().sum(0) + 0.5 * ws * H.double().abs().sum(1, keepdim=True) + 0.25 * d * s * ws
    assert bool(((z - exact).abs() <= bound * (1 + 1e-5)).all())

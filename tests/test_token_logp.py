"""Token log-probabilities through the head on the GPU against the 64-bit form: every kernel path, partial tiles and
chunks, masks, temperatures, stored logits, vocabulary shards, autograd, streams and captured graphs."""
import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import dev, say
from tests.policy_util import logp_reference, make_head, within

pytestmark = pytest.mark.gpu
bf, f32 = torch.bfloat16, torch.float32


def upstream(T, seed):
    g = torch.Generator().manual_seed(seed + 1000)
    return torch.randn(T, generator=g), torch.randn(T, generator=g)


SHAPES = [
    # T, d, V, dtype, masked, tau, chunk_rows
    (1, 128, 256, bf, 0.0, 1.0, 0),
    (1, 2048, 4096, bf, 0.0, 1.0, 0),
    (7, 256, 1032, bf, 0.0, 0.7, 0),
    (31, 384, 2056, bf, 0.4, 1.0, 0),
    (33, 512, 520, bf, 0.0, 1.0, 0),
    (65, 128, 264, bf, 0.3, 2.5, 0),
    (130, 640, 3000, bf, 0.0, 1.0, 0),
    (257, 128, 512, bf, 0.0, 1.0, 0),
    (300, 256, 1288, bf, 0.2, 1.3, 0),
    (700, 128, 1000, bf, 0.2, 1.0, 256),
    (513, 256, 776, bf, 0.0, 1.0, 512),
    (40, 96, 1600, bf, 0.2, 1.0, 0),    # contraction not a multiple of 128
    (20, 160, 488, bf, 0.0, 1.0, 0),
    (9, 72, 328, bf, 0.0, 1.0, 0),
    (300, 200, 8, bf, 0.1, 1.0, 0),     # less than a tile of vocabulary
    (5, 8, 16, bf, 0.0, 1.0, 0),
    # from 7 million logits a round on, the forward runs on the 256 x 256 ring tiles
    (600, 256, 12032, bf, 0.0, 1.0, 0),     # whole ring turns everywhere
    (601, 160, 12008, bf, 0.2, 0.8, 0),     # d, V inside a turn, V inside a 32-column stage
    (1100, 96, 6624, bf, 0.3, 1.0, 512),    # several chunks of a bf16 dW, V inside a turn
    (1300, 384, 5592, bf, 0.0, 1.0, 0),
    # and the backward from 7e9 terms of a product on
    (400, 2080, 8456, bf, 0.3, 0.9, 0),     # d inside a turn, V inside a 32-column stage
    (1500, 1056, 4456, bf, 0.2, 1.0, 512),  # several chunks of a bf16 dW
    (90, 8192, 9504, bf, 0.0, 1.0, 0),      # a row block mostly empty, V inside a turn
    (330, 4096, 5248, bf, 0.1, 1.0, 0),     # whole turns
    (1, 4, 4, f32, 0.0, 1.0, 0),
    (33, 12, 20, f32, 0.3, 1.0, 0),
    (65, 100, 260, f32, 0.0, 0.5, 0),
    (300, 64, 1004, f32, 0.2, 1.0, 256),
    (129, 256, 512, f32, 0.0, 1.0, 0),
]


@pytest.mark.parametrize("T,d,V,dtype,masked,tau,chunk", SHAPES)
@pytest.mark.parametrize("entropy,keep", [(False, False), (True, False), (True, True), (False, True)])
def test_forward_and_backward(T, d, V, dtype, masked, tau, chunk, entropy, keep):
    H, W, tokens, mask = make_head(T, d, V, dtype, T + d + V, masked=masked)
    tokens[0], tokens[-1] = V - 1, 0
    if mask is not None:
        mask[0] = 1
    g, ge = upstream(T, T)
    say(f"token_logp T={T} d={d} V={V} {dtype} masked={masked} entropy={entropy} keep={keep} chunk={chunk}")
    want, bound = logp_reference(H, W, tokens, mask, tau, g, ge if entropy else None)
    dH_, dW_, dt, dm = dev(H), dev(W), dev(tokens), dev(mask)
    logp, lse, ent, z = kd.token_logp_forward(dH_, dW_, dt, dm, tau, want_entropy=entropy, keep_logits=keep)
    got = dict(logp=logp, lse=lse)
    if entropy:
        got["entropy"] = ent
    for dw in ((f32, bf) if dtype == bf else (f32,)):
        got["dH"], got["dW"] = kd.token_logp_backward(dH_, dW_, dt, dm, tau, lse, dev(g), ent,
                                                      dev(ge) if entropy else None, z, chunk, dw)
        torch.cuda.synchronize()
        assert got["dH"].dtype == dtype and got["dW"].dtype == dw
        for k, v in got.items():
            within(v, want[k], bound[k], f"{k} ({dw})")
    if mask is not None:
        off = mask == 0
        for k in ("logp", "lse", "dH"):
            assert (got[k].cpu()[off] == 0).all(), k


def test_entropy_gradient_alone():
    H, W, tokens, mask = make_head(70, 256, 600, bf, 3, masked=0.2)
    _, ge = upstream(70, 3)
    want, bound = logp_reference(H, W, tokens, mask, 1.0, None, ge)
    a = [dev(x) for x in (H, W, tokens, mask)]
    _, lse, ent, _ = kd.token_logp_forward(*a, 1.0, want_entropy=True)
    dH, dW = kd.token_logp_backward(*a, 1.0, lse, None, ent, dev(ge))
    within(dH, want["dH"], bound["dH"], "dH")
    within(dW, want["dW"], bound["dW"], "dW")


def test_gradient_against_differences():
    """Central differences of the GPU forward itself, float32: along a direction, (f(x + e) - f(x - e)) / 2e is the
    gradient up to e^2 and up to the forward's own error over e.  With e = 2^-6 the first is below 1e-3 of these sums
    (third derivatives of log-softmax are below 1, the directions have unit-sized entries over 0.02) and the second,
    24 rows of 1e-6 over 2^-6, below 2e-3."""
    T, d, V = 24, 32, 200
    H, W, tokens, _ = make_head(T, d, V, f32, 5)
    g, ge = upstream(T, 5)
    gen = torch.Generator().manual_seed(9)
    vH, vW = torch.randn(T, d, generator=gen) * 0.05, torch.randn(d, V, generator=gen) * 0.05
    dg, dge, dt = dev(g), dev(ge), dev(tokens)

    def f(h, w):
        logp, _, ent, _ = kd.token_logp_forward(dev(h), dev(w), dt, None, 1.0, want_entropy=True)
        return float((logp.double() * dg).sum() + (ent.double() * dge).sum())

    _, lse, ent, _ = kd.token_logp_forward(dev(H), dev(W), dt, None, 1.0, want_entropy=True)
    dH, dW = kd.token_logp_backward(dev(H), dev(W), dt, None, 1.0, lse, dg, ent, dge)
    along = float((dH.double().cpu() * vH).sum() + (dW.double().cpu() * vW).sum())
    e = 2.0 ** -6
    diff = (f(H + e * vH, W + e * vW) - f(H - e * vH, W - e * vW)) / (2 * e)
    assert abs(diff - along) <= 3e-3 * (1 + abs(along)), (diff, along)


@pytest.mark.parametrize("V,rows,d", [(1000, 0, 128), (7016, 1024, 128), (7016, 1024, 1024)])
def test_tokens_at_every_tile_edge(V, rows, d):
    """One row per column where a tile, a wave's half or a lane's group begins or ends."""
    edges = sorted({max(0, min(V - 1, b + o)) for b in range(0, V + 32, 32) for o in (-1, 0, 3, 4)} | {744, 743, 767, 768})
    edges = (edges + list(range(rows)))[:max(rows, len(edges))]
    T = len(edges)
    H, W, _, _ = make_head(T, d, V, bf, 11)
    tokens = torch.tensor(edges, dtype=torch.int32)
    g, _ = upstream(T, 11)
    want, bound = logp_reference(H, W, tokens, None, 1.0, g)
    a = (dev(H), dev(W), dev(tokens), None)
    logp, lse, _, z = kd.token_logp_forward(*a, 1.0, keep_logits=True)
    within(logp, want["logp"], bound["logp"], "logp")
    for zz in (None, z):
        dH, dW = kd.token_logp_backward(*a, 1.0, lse, dev(g), logits=zz)
        within(dH, want["dH"], bound["dH"], "dH")
        within(dW, want["dW"], bound["dW"], "dW")


@pytest.mark.parametrize("T,V,d", [(20, 776, 128), (300, 776, 128), (1000, 7016, 128), (1000, 7016, 1024)])
def test_large_logits(T, V, d):
    """Logits of hundreds: every 2^x must be taken relative to the row's maximum, and rows past the last valid one
    (whose accumulators hold a copy of a real row) must not reach dW."""
    H, W, tokens, mask = make_head(T, d, V, bf, 13, scale=30.0, masked=0.1)
    g, ge = upstream(T, 13)
    want, bound = logp_reference(H, W, tokens, mask, 1.0, g, ge)
    a = [dev(x) for x in (H, W, tokens, mask)]
    logp, lse, ent, z = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True)
    for k, v in (("logp", logp), ("lse", lse), ("entropy", ent)):
        within(v, want[k], bound[k], k)
    for zz in (None, z):
        dH, dW = kd.token_logp_backward(*a, 1.0, lse, dev(g), ent, dev(ge), zz)
        within(dH, want["dH"], bound["dH"], "dH")
        within(dW, want["dW"], bound["dW"], "dW")


@pytest.mark.parametrize("T,V,d,dtype", [(12, 520, 128, bf), (300, 520, 128, bf), (1000, 7016, 128, bf),
                                         (1000, 7016, 1024, bf), (12, 520, 128, f32)])
def test_masked_rows_are_not_read(T, V, d, dtype):
    H, W, tokens, _ = make_head(T, d, V, dtype, 17)
    mask = torch.ones(T, dtype=torch.uint8)
    mask[::3] = 0
    g, ge = upstream(T, 17)
    want, bound = logp_reference(H, W, tokens, mask, 1.0, g, ge)
    H[::3] = float("nan")
    tokens[::3] = -100
    g[::3], ge[::3] = float("inf"), float("nan")
    a = [dev(x) for x in (H, W, tokens, mask)]
    logp, lse, ent, z = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True)
    for k, v in (("logp", logp), ("lse", lse), ("entropy", ent)):
        within(v, want[k], bound[k], k)
    for zz in (None, z):
        dH, dW = kd.token_logp_backward(*a, 1.0, lse, dev(g), ent, dev(ge), zz)
        within(dH, want["dH"], bound["dH"], "dH")
        within(dW, want["dW"], bound["dW"], "dW")
    some = kd.token_logp_forward(a[0], a[1], a[2], dev(mask.bool()), 1.0)
    assert torch.equal(some[0], logp)


@pytest.mark.parametrize("T,V,d", [(5, 264, 128), (1000, 7016, 128), (1000, 7016, 1024)])
def test_every_row_masked_and_no_rows(T, V, d):
    H, W, tokens, _ = make_head(T, d, V, bf, 19)
    a = [dev(x) for x in (H, W, tokens, torch.zeros(T, dtype=torch.uint8))]
    logp, lse, ent, z = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True)
    g = torch.ones(T, device="cuda")
    for zz in (None, z):
        for dt in (f32, bf):
            dH, dW = kd.token_logp_backward(*a, 1.0, lse, g, ent, g, zz, dw_dtype=dt)
            for x in (logp, lse, ent, dH, dW):
                assert (x == 0).all()
    e = [a[0][:0], a[1], a[2][:0], None]
    logp, lse, ent, z = kd.token_logp_forward(*e, 1.0, want_entropy=True, keep_logits=True)
    dH, dW = kd.token_logp_backward(*e, 1.0, lse, g[:0], dw_dtype=bf)
    assert logp.numel() == 0 and dH.shape == (0, d) and (dW == 0).all()


@pytest.mark.parametrize("T,V", [(6, 264), (300, 264), (1000, 7016)])
def test_a_token_outside_the_vocabulary_is_nan(T, V):
    H, W, tokens, _ = make_head(T, 128, V, bf, 23)
    want, bound = logp_reference(H, W, tokens, None, 1.0)
    tokens[1], tokens[4] = -100, V
    logp, lse, _, _ = kd.token_logp_forward(dev(H), dev(W), dev(tokens), None, 1.0)
    got = logp.cpu()
    assert torch.isnan(got[[1, 4]]).all()
    keep = [i for i in range(T) if i not in (1, 4)]
    within(got[keep], want["logp"][keep], bound["logp"][keep], "logp")
    within(lse, want["lse"], bound["lse"], "lse")


@pytest.mark.parametrize("T,cuts,dtype,d", [(90, (0, 264, 600, 1288), bf, 128), (90, (0, 8, 1288), bf, 128),
                                            (90, (0, 500, 1004), f32, 128), (1000, (0, 7016, 14048), bf, 128),
                                            (1000, (0, 7016, 14048), bf, 1024)])
def test_vocabulary_shards(T, cuts, dtype, d):
    V = cuts[-1]
    H, W, tokens, mask = make_head(T, d, V, dtype, 29, masked=0.2)
    g, ge = upstream(T, 29)
    want, bound = logp_reference(H, W, tokens, mask, 1.3, g, ge)
    h, dt, dm = dev(H), dev(tokens), dev(mask)
    parts = [dev(W[:, a:b].contiguous()) for a, b in zip(cuts, cuts[1:])]
    fw = [kd.token_logp_shard_forward(h, w, a, dt, dm, 1.3, keep_logits=True) for w, a in zip(parts, cuts)]
    logp, lse, ent = kd.token_logp_shard_combine([r for r, _ in fw], dm, 1.3, want_entropy=True)
    for k, v in (("logp", logp), ("lse", lse), ("entropy", ent)):
        within(v, want[k], bound[k], k)
    for keep in (False, True):
        bw = [kd.token_logp_shard_backward(h, w, a, dt, dm, 1.3, lse, dev(g), ent, dev(ge), z if keep else None)
              for w, a, (_, z) in zip(parts, cuts, fw)]
        within(sum(x for x, _ in bw), want["dH"], bound["dH"], "dH")
        within(torch.cat([x for _, x in bw], 1), want["dW"], bound["dW"], "dW")


@pytest.mark.parametrize("keep", [False, True])
def test_autograd(keep):
    H, W, tokens, mask = make_head(60, 256, 520, bf, 31, masked=0.2)
    g, ge = upstream(60, 31)
    want, bound = logp_reference(H, W, tokens, mask, 1.0, g, ge)
    h, w = dev(H).requires_grad_(True), dev(W).requires_grad_(True)
    logp, ent = kd.token_logp(h, w, dev(tokens), dev(mask), want_entropy=True, keep_logits=keep)
    ((logp * dev(g)).sum() + (ent * dev(ge)).sum()).backward()
    assert h.grad.dtype == bf and w.grad.dtype == bf
    within(h.grad, want["dH"], bound["dH"], "dH")
    within(w.grad, want["dW"], bound["dW"], "dW")
    only, bo = logp_reference(H, W, tokens, mask, 1.0, g)
    dH, = torch.autograd.grad(kd.token_logp(h, w, dev(tokens), dev(mask), keep_logits=keep), h, dev(g))
    within(dH, only["dH"], bo["dH"], "dH alone")


@pytest.mark.parametrize("T,d,V", [(70, 128, 520), (1000, 160, 7016), (1000, 1056, 7016)])
def test_nothing_around_the_buffers_changes(T, d, V):
    """Outputs and workspace of exactly the asked size inside larger buffers."""
    Vp = -(-V // 256) * 256
    H, W, tokens, mask = make_head(T, d, V, bf, 37, masked=0.3)
    B = kd._policy_binding
    say("guards around every output and the workspace")

    def guarded(n, dtype):
        n_b = n * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((n_b + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        return raw, raw[256:256 + n_b].view(dtype)

    nb = B.kd_token_logp_workspace_size(T, d, V, bf, bf)
    raws = {}
    out = {}
    for k, (n, dt) in dict(ws=(nb, torch.uint8), logp=(T, f32), lse=(T, f32), ent=(T, f32), z=(T * Vp, f32),
                           dH=(T * d, bf), dW=(d * V, bf)).items():
        raws[k], out[k] = guarded(n, dt)
    z = out["z"].view(T, Vp)
    a = [dev(x) for x in (H, W, tokens, mask)]
    B.kd_token_logp_fwd(*a, 1.0, out["logp"], out["lse"], out["ent"], z, out["ws"])
    g = torch.randn(T, device="cuda")
    for zz in (None, z):
        B.kd_token_logp_bwd(*a, 1.0, out["lse"], out["ent"], zz, g, g, out["dH"].view(T, d), out["dW"].view(d, V), 0,
                            out["ws"])
    torch.cuda.synchronize()
    for k, raw in raws.items():
        assert (raw[:256] == 0x5A).all() and (raw[-256:] == 0x5A).all(), k


@pytest.mark.parametrize("T,V,d", [(300, 1288, 256), (1000, 7016, 256), (1000, 7016, 1024)])
def test_another_stream_and_the_same_bits(T, V, d):
    H, W, tokens, mask = make_head(T, d, V, bf, 41, masked=0.2)
    a = [dev(x) for x in (H, W, tokens, mask)]
    g = torch.randn(T, device="cuda")

    def calls():
        logp, lse, ent, z = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True)
        return [logp, lse, ent, *kd.token_logp_backward(*a, 1.0, lse, g, ent, g, z),
                *kd.token_logp_backward(*a, 1.0, lse, g, ent, g)]

    first = calls()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = calls()
    s.synchronize()
    for x, y in zip(first, second):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,V,d", [(9, 776, 256), (300, 776, 256), (1000, 7016, 256), (1000, 7016, 1024)])
def test_captured_and_replayed(T, V, d):
    H, W, tokens, mask = make_head(T, d, V, bf, 43, masked=0.2)
    a = [dev(x) for x in (H, W, tokens, mask)]
    g = torch.randn(T, device="cuda")

    def calls():
        logp, lse, ent, z = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True)
        return [logp, ent, *kd.token_logp_backward(*a, 1.0, lse, g, ent, g, z, dw_dtype=bf)]

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for k in range(4):
        h2, _, t2, m2 = make_head(T, d, V, bf, 50 + k, masked=0.1 * k)
        a[0].copy_(h2)
        a[2].copy_(t2)
        a[3].copy_(torch.ones(T, dtype=torch.uint8) if m2 is None else m2)
        want = calls()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y), f"replay {k}"


@pytest.mark.parametrize("T,V,d,dtype", [(40, 520, 128, bf), (1000, 7016, 128, bf), (1000, 7016, 1024, bf),
                                         (40, 520, 128, f32)])
def test_one_gradient_alone(T, V, d, dtype):
    """A frozen head wants dH only, a probe on frozen states dW only; each is the same bits as together."""
    H, W, tokens, mask = make_head(T, d, V, dtype, 61, masked=0.2)
    a = [dev(x) for x in (H, W, tokens, mask)]
    g = torch.randn(T, device="cuda")
    _, lse, _, z = kd.token_logp_forward(*a, 1.0, keep_logits=True)
    for zz in (None, z):
        dH, dW = kd.token_logp_backward(*a, 1.0, lse, g, logits=zz, dw_dtype=dtype)
        x, none = kd.token_logp_backward(*a, 1.0, lse, g, logits=zz, dw_dtype=dtype, want=(True, False))
        assert none is None and torch.equal(x, dH)
        none, y = kd.token_logp_backward(*a, 1.0, lse, g, logits=zz, dw_dtype=dtype, want=(False, True))
        assert none is None and torch.equal(y, dW)
    h = a[0].clone().requires_grad_(True)
    kd.token_logp(h, a[1], a[2], a[3]).backward(g)
    assert a[1].grad is None and torch.equal(h.grad, kd.token_logp_backward(*a, 1.0, lse, g, dw_dtype=dtype)[0])


@pytest.mark.parametrize("T", [65536, 65537, 70001])
def test_many_short_rows(T):
    """Many chunks of rows, where the mask is counted in another way than for few."""
    H, W, tokens, mask = make_head(T, 16, 64, f32, 67, masked=0.3)
    mask[:5000] = 0
    g = torch.randn(T, generator=torch.Generator().manual_seed(68))
    want, bound = logp_reference(H, W, tokens, mask, 1.0, g)
    a = [dev(x) for x in (H, W, tokens, mask)]
    logp, lse, _, _ = kd.token_logp_forward(*a)
    dH, dW = kd.token_logp_backward(*a, 1.0, lse, dev(g))
    for name, got in (("logp", logp), ("lse", lse), ("dH", dH), ("dW", dW)):
        within(got, want[name], bound[name], name)
    assert (dH[a[3] == 0] == 0).all() and (logp[a[3] == 0] == 0).all()


@pytest.mark.parametrize("T", [1, 2, 31, 32])
@pytest.mark.parametrize("kept", [False, True])
def test_few_rows_keep_the_rest_of_dz(T, kept):
    """Up to 32 bf16 rows, dH and dW are off by their own rounding (and 2^-16 of dZ's)."""
    H, W, tokens, mask = make_head(T, 256, 1288, bf, 69, masked=0.3 if T > 2 else 0.0)
    gen = torch.Generator().manual_seed(70)
    g, ge = torch.randn(T, generator=gen), torch.randn(T, generator=gen)
    want, bound = logp_reference(H, W, tokens, mask, 1.0, g, ge)
    a = [dev(x) for x in (H, W, tokens, mask)]
    _, lse, ent, z = kd.token_logp_forward(*a, want_entropy=True, keep_logits=kept)
    dH, dW = kd.token_logp_backward(*a, 1.0, lse, dev(g), ent, dev(ge), z, dw_dtype=bf)
    for name, got in (("dH", dH), ("dW", dW)):
        within(got, want[name], bound[name], name)
        off = (got.double().cpu() - want[name]).norm() / want[name].norm()
        assert off <= 0.0025, (name, float(off))  # a rounding to bf16 is off by 2^-9 to 2^-8 at most, 0.0017 on average

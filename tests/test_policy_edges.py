"""Calls of the policy operators at the edges of what their documentation allows, on the GPU."""
import math

import pytest
import torch

import chunked_kl_loss_logit_amd as kd
from tests.gpu_util import dev, say
from tests.policy_util import U32, half_step, logp_reference, make_head, within

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


def masked_head(T, d, V, dtype, blocked, value, seed, masked=0.0):
    """A head with columns masked through its last row, which every hidden state meets with 1: logits of `value` there,
    and the same head without those columns."""
    H, W, tokens, mask = make_head(T, d, V, dtype, seed, masked=masked)
    keep = torch.ones(V, dtype=torch.bool)
    for a, b in blocked:
        keep[a:b] = False
    H[:, -1] = 1
    W[-1] = 0
    W[:, ~keep] = 0
    W[-1, ~keep] = value
    to = torch.cumsum(keep, 0) - 1  # place among the columns that stay
    allowed = torch.nonzero(keep)[:, 0]
    tokens = allowed[tokens.long() % allowed.numel()].to(torch.int32)
    return H, W, tokens, mask, keep, W[:, keep].contiguous(), to[tokens.long()].to(torch.int32)


# the register-fed tiles, then the forward and everything on the ring tiles
MASKED_HEADS = [(5, 128, 1024, bf), (90, 128, 1032, bf), (40, 72, 520, f32), (1000, 160, 7016, bf), (1000, 1056, 7016, bf)]


@pytest.mark.parametrize("T,d,V,dtype", MASKED_HEADS)
@pytest.mark.parametrize("value", [-1e4, -3.7e9, -1e38, None])
@pytest.mark.parametrize("blocks", ["one", "tiles", "first", "last"])
def test_masked_columns(T, d, V, dtype, value, blocks):
    """A vocabulary partly masked by large negative logits, down to the type's lowest value: such columns have
    probability 0 and add nothing, also where a whole tile of them comes first."""
    value = torch.finfo(dtype).min if value is None else value
    blocked = dict(one=[(7, 8)], tiles=[(128, 512)], first=[(0, 264)], last=[(V - 200, V)])[blocks]
    say(f"masked columns T={T} d={d} V={V} {dtype} {value} {blocked}")
    H, W, tokens, mask, keep, Wk, tk = masked_head(T, d, V, dtype, blocked, value, 53, masked=0.2 if T > 5 else 0.0)
    gen = torch.Generator().manual_seed(54)
    g, ge = torch.randn(T, generator=gen), torch.randn(T, generator=gen)
    want, bound = logp_reference(H, Wk, tk, mask, 1.0, g, ge)
    a = [dev(x) for x in (H, W, tokens, mask)]
    logp, lse, ent, z = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True)
    for name, got in (("logp", logp), ("lse", lse), ("entropy", ent)):
        within(got, want[name], bound[name], name)
    for zz in (None, z):
        dH, dW = kd.token_logp_backward(*a, 1.0, lse, dev(g), ent, dev(ge), zz)
        within(dH, want["dH"], bound["dH"], "dH")
        within(dW.cpu()[:, keep], want["dW"], bound["dW"], "dW")
        assert (dW.cpu()[:, ~keep] == 0).all()


@pytest.mark.parametrize("T,d,V,dtype", MASKED_HEADS[1:4])
def test_masked_columns_of_any_size(T, d, V, dtype):
    """Whichever way the largest logit of a masked tile rounds in base 2."""
    H, W, tokens, _, keep, Wk, tk = masked_head(T, d, V, dtype, [(0, 264)], 0.0, 59)
    want, bound = logp_reference(H, Wk, tk, None, 1.0)
    h, w, t = dev(H), dev(W), dev(tokens)
    gen = torch.Generator().manual_seed(60)
    for value in (-10 ** (3 + 35.5 * torch.rand(24, generator=gen))).tolist():
        w[-1, :264] = value * (1 + 0.1 * torch.rand(264, generator=gen)).cuda()
        for tau in (1.0, 0.4):
            logp, lse, ent, _ = kd.token_logp_forward(h, w, t, None, tau, want_entropy=True)
            if tau == 1.0:
                for name, got in (("logp", logp), ("lse", lse), ("entropy", ent)):
                    within(got, want[name], bound[name], f"{name} at {value}")
            assert torch.isfinite(logp).all() and torch.isfinite(ent).all(), value


def test_a_masked_shard_and_a_masked_token():
    T, d, V = 30, 128, 1024
    H, W, tokens, _, keep, Wk, tk = masked_head(T, d, V, bf, [(0, 512)], torch.finfo(bf).min, 55)
    want, bound = logp_reference(H, Wk, tk, None, 1.0)
    h, t = dev(H), dev(tokens)
    recs = [kd.token_logp_shard_forward(h, dev(W[:, a:a + 512].contiguous()), a, t)[0] for a in (0, 512)]
    logp, lse, ent = kd.token_logp_shard_combine(recs, want_entropy=True)
    for name, got in (("logp", logp), ("lse", lse), ("entropy", ent)):
        within(got, want[name], bound[name], name)
    tokens[3] = 9  # masked: log-probability -3.39e38, which 32 bits hold
    logp = kd.token_logp_forward(h, dev(W), dev(tokens))[0].cpu()
    assert abs(float(logp[3]) / float(torch.finfo(bf).min) - 1) < 1e-6
    W[-1] = torch.finfo(bf).min  # every column: below what 32 bits hold in base 2, NaN rather than a wrong number
    H[:, :-1] = 0
    logp, lse, ent, _ = kd.token_logp_forward(dev(H), dev(W), t, want_entropy=True)
    assert torch.isnan(logp).all() and torch.isnan(lse).all() and torch.isnan(ent).all()


@pytest.mark.parametrize("T,d,V,dtype", MASKED_HEADS)
def test_nan_and_infinite_logits_stay_visible(T, d, V, dtype):
    """A row whose hidden state is NaN, or overflows, is NaN in all it gives; the others are as they were."""
    H, W, tokens, _ = make_head(T, d, V, dtype, 57)
    a = (dev(W), dev(tokens), None)
    clean = kd.token_logp_forward(dev(H), *a, 1.0, want_entropy=True)[:3]
    H[1, 0], H[3, :] = float("nan"), 3e38
    h = dev(H)
    got = kd.token_logp_forward(h, *a, 1.0, want_entropy=True, keep_logits=True)
    z = got[3]
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[1] = bad[3] = True
    for x, y in zip(got, clean):
        assert torch.isnan(x[bad]).all() and torch.equal(x[~bad], y[~bad])
    g = torch.ones(T, device="cuda")
    for zz in (None, z):
        dH, _ = kd.token_logp_backward(h, *a, 1.0, got[1], g, got[2], g, zz)
        assert torch.isnan(dH[bad]).all() and torch.isfinite(dH[~bad]).all()


def big_inputs(which, T):
    gen = torch.Generator(device="cuda").manual_seed(61)
    r = lambda: torch.randn(T, generator=gen, device="cuda")  # noqa: E731
    cu = torch.tensor([0, 5, T // 2, T // 2, T], dtype=torch.int32, device="cuda")
    mask = (r() > -1).to(torch.uint8)
    if which == "policy":
        return r().requires_grad_(True), (r(), r(), mask), dict(ref_logp=r(), entropy=r(), cu_seqlens=cu, kl_weight=0.1,
                                                                entropy_weight=0.1, reduction="sequence", per_sequence=False)
    return r().requires_grad_(True), (cu, mask), dict(ref_logp=r(), average=True)


def loss_of(which, x, args, kw):
    return kd.policy_loss(x, *args, **kw)[0] if which == "policy" else kd.preference_loss(x, *args, **kw)[0].sum()


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_inputs_go_where_saved_tensors_go(which):
    """Offloaded while the loss waits for its backward, and let go after it; the gradients are the same bits."""
    T = 1 << 20
    x, args, kw = big_inputs(which, T)
    loss = loss_of(which, x, args, kw)
    want, = torch.autograd.grad(loss, x, retain_graph=True)
    again, = torch.autograd.grad(loss, x)
    assert torch.equal(again, want)
    ref = kw["ref_logp"]
    size = ref.numel() * 4
    del loss
    with torch.autograd.graph.save_on_cpu():
        loss = loss_of(which, x, args, kw)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    del ref, args, kw
    assert before - torch.cuda.memory_allocated() >= size
    got, = torch.autograd.grad(loss, x)
    assert torch.equal(got, want)
    x, args, kw = big_inputs(which, T)
    loss = loss_of(which, x, args, kw)
    loss.backward()
    before = torch.cuda.memory_allocated()
    del args, kw
    assert before - torch.cuda.memory_allocated() >= size and float(loss.detach()) == float(loss.detach())


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_saved_tensors_that_come_back_changed_are_refused(which):
    x, args, kw = big_inputs(which, 1000)
    for unpack in (lambda t: t[:-1], lambda t: t.double(), lambda t: t.cpu(), lambda t: t.repeat_interleave(2, 0)[::2]):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
            loss = loss_of(which, x, args, kw)
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            loss.backward()
    loss = loss_of(which, x, args, kw)
    kw["ref_logp"].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("T,d,V,dtype", [(70, 128, 520, bf), (70, 128, 520, f32), (1000, 160, 7016, bf), (5000, 160, 2056, bf)])
def test_a_forward_in_its_own_workspace(T, d, V, dtype):
    """In exactly the bytes asked for, between guards, with the results of any other workspace; a scoring call takes no
    more than that and its outputs."""
    H, W, tokens, mask = make_head(T, d, V, dtype, 63, masked=0.3)
    a = [dev(x) for x in (H, W, tokens, mask)]
    B = kd._policy_binding
    nb = B.kd_token_logp_fwd_workspace_size(T, d, V, dtype)
    raw = torch.full((nb + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = raw[4096:4096 + nb]
    big = torch.empty(B.kd_token_logp_workspace_size(T, d, V, dtype), dtype=torch.uint8, device="cuda")
    want = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True, workspace=big)
    got = kd.token_logp_forward(*a, 1.0, want_entropy=True, keep_logits=True, workspace=ws)
    rec = kd.token_logp_shard_forward(a[0], a[1], 0, a[2], a[3], workspace=ws)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got[:3], want[:3])) and torch.isfinite(rec).all()
    assert (raw[:4096] == 0xA5).all() and (raw[-4096:] == 0xA5).all()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    kd.token_logp_forward(*a, 1.0)
    assert torch.cuda.max_memory_allocated() - before <= nb + 2 * 4 * T + 4 * 512


@pytest.mark.parametrize("T", [1, 7, 32])
@pytest.mark.parametrize("cuts", [(0, 256, 768), (0, 512, 520), (0, 1288, 4096)])
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_vocabulary_shards_of_few_rows(T, cuts, masked):
    """A float32 part of dH from the two planes of dZ: shards of one vocabulary range (512 columns and fewer) and of
    several."""
    d, V = 160, cuts[-1]
    H, W, tokens, mask = make_head(T, d, V, bf, 65, masked=masked if T > 1 else 0.0)
    gen = torch.Generator().manual_seed(66)
    g, ge = torch.randn(T, generator=gen), torch.randn(T, generator=gen)
    want, bound = logp_reference(H, W, tokens, mask, 0.8, g, ge)
    h, t, m = dev(H), dev(tokens), dev(mask)
    parts = [dev(W[:, a:b].contiguous()) for a, b in zip(cuts, cuts[1:])]
    fw = [kd.token_logp_shard_forward(h, w, a, t, m, 0.8, keep_logits=True) for w, a in zip(parts, cuts)]
    logp, lse, ent = kd.token_logp_shard_combine([r for r, _ in fw], m, 0.8, want_entropy=True)
    for name, got in (("logp", logp), ("lse", lse), ("entropy", ent)):
        within(got, want[name], bound[name], name)
    for keep in (False, True):
        for dw in (f32, bf):
            bw = [kd.token_logp_shard_backward(h, w, a, t, m, 0.8, lse, dev(g), ent, dev(ge), z if keep else None, dw_dtype=dw)
                  for w, a, (_, z) in zip(parts, cuts, fw)]
            assert all(x.dtype == f32 and y.dtype == dw for x, y in bw)
            dH = sum(x for x, _ in bw)
            within(dH, want["dH"], bound["dH"], "dH")
            within(torch.cat([y for _, y in bw], 1), want["dW"], bound["dW"], "dW")
            # float32 parts are off by dZ's 2^-16 and the logits' own error alone
            assert (dH.double().cpu() - want["dH"]).norm() <= 2.0 ** -12 * want["dH"].norm() + 1e-30
            if mask is not None:
                assert (dH[m == 0] == 0).all()

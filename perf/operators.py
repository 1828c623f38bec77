"""What the policy- and preference-training operators cost and how exact they are.

Each case is one call (or one training step) as a program makes it: token log-probabilities through the output
head, the clipped policy loss, the preference loss and gradient clipping.  `run` computes them in plain torch where
`own` is false, and with this package's operators where it is true.
"""
import math

import torch

own = False

NEG = -1  # label of rows that the mask leaves out: never a vocabulary index


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # scoring the few tokens of a short answer: one read of the head is all there is to do
        dict(name="logp few rows", op="logp", T=7, d=2048, V=32000, dtype="bf16", masked=0.0, entropy=False),
        # the log-probabilities of a batch of samples under a frozen reference, prompt rows masked
        dict(name="logp reference", op="logp", T=1500, d=4096, V=128256, dtype="bf16", masked=0.3, entropy=True),
        # the head's part of a training step: log-probabilities, entropy and both gradients
        dict(name="logp step", op="logp_step", T=4096, d=2048, V=128256, dtype="bf16", masked=0.0, entropy=True),
        # the same in float32 on a small head, an odd number of rows
        dict(name="logp step fp32", op="logp_step", T=777, d=1024, V=32000, dtype="f32", masked=0.1, entropy=True),
        # one micro-batch of a policy update: a few hundred tokens, through autograd
        dict(name="policy small", op="policy", T=333, S=5, masked=0.2, kl="k3", dual=0.0, reduction="token",
             entropy=False, per_seq=False, autograd=True),
        # a whole rollout batch: a million packed tokens, one advantage per sample, mean over samples
        dict(name="policy rollout", op="policy", T=1048576, S=1000, masked=0.25, kl="k3", dual=3.0,
             reduction="sequence", entropy=True, per_seq=True, autograd=False),
        # a few pairs of short answers, through autograd
        dict(name="preference small", op="preference", T=900, P=4, masked=0.3, kind="sigmoid", average=False,
             autograd=True),
        # a large batch of pairs of ragged lengths
        dict(name="preference batch", op="preference", T=700001, P=384, masked=0.2, kind="sigmoid", average=False,
             autograd=False),
        # a whole preference step through the head: log-probabilities, pair losses, gradients of H and W
        dict(name="preference step", op="pair_step", T=1600, d=2048, V=32000, P=6, dtype="bf16", masked=0.25),
        # the gradients of a small model's layers, views of two buckets, clipped into the optimizer's buckets
        dict(name="clip many", op="clip", n=290, numel=30000000, dtype="bf16", ratio=0.3),
        # the gradients of an output head and its input, accumulated in float32
        dict(name="clip head", op="clip", n=3, numel=400000000, dtype="f32", ratio=0.5),
        # a handful of small tensors: latency
        dict(name="clip few", op="clip", n=6, numel=40000, dtype="f32", ratio=2.0),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["logp", "logp", "logp_step", "logp_step", "policy", "preference", "pair_step", "clip"])
    masked = rng.choice([0.0, rng.uniform(0.05, 0.6)])
    if op in ("logp", "logp_step", "pair_step"):
        dtype = "bf16" if op == "pair_step" else rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = 64 * _log(rng, 4, 64)
        V = 8 * _log(rng, 100, 16032)
        most = 4096 * 2048 * 128256 // (1 if dtype == "bf16" else 24)  # what the largest listed one costs
        T = _log(rng, 12 if op == "pair_step" else 1, max(16, min(4096, most // (d * V))))
        c = dict(op=op, T=T, d=d, V=V, dtype=dtype, masked=masked if T >= 16 else 0.0)
        if op == "pair_step":
            return dict(c, P=rng.randint(1, max(1, min(32, T // 12))))
        return dict(c, entropy=rng.random() < 0.6)
    if op == "policy":
        T = _log(rng, 1, 1000000)
        return dict(op=op, T=T, S=rng.randint(1, min(2000, 1 + T // 8)), masked=masked if T >= 16 else 0.0,
                    kl=rng.choice(["none", "k1", "k2", "k3"]), dual=rng.choice([0.0, 2.5]),
                    reduction=rng.choice(["sum", "token", "sequence"]), entropy=rng.random() < 0.5,
                    per_seq=rng.random() < 0.5, autograd=rng.random() < 0.3)
    if op == "preference":
        T = _log(rng, 16, 700000)
        return dict(op=op, T=T, P=rng.randint(1, min(512, T // 8)), masked=masked,
                    kind=rng.choice(["sigmoid", "hinge", "ipo"]), average=rng.random() < 0.4,
                    autograd=rng.random() < 0.3)
    return dict(op=op, n=rng.randint(1, 300), numel=_log(rng, 3000, 100000000), dtype=rng.choice(["bf16", "f32", "f16"]),
                ratio=rng.uniform(0.1, 3.0))


# ------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def _cuts(gen, n, total):
    """n + 1 ascending ints from 0 to total: ragged lengths, some of them zero where total is short."""
    inner = torch.randint(0, total + 1, (n - 1,), generator=gen, device="cuda") if n > 1 else torch.empty(0, dtype=torch.int64, device="cuda")
    ends = torch.tensor([0, total], device="cuda")
    return torch.cat([ends[:1], inner.sort().values, ends[1:]]).to(torch.int32)


def _head(c, gen):
    """Hidden states, head and target tokens: logits of standard deviation 2, the target's raised by 0 to 12 as a
    trained model's are."""
    T, d, V, dt = c["T"], c["d"], c["V"], _TYPES[c["dtype"]]
    W = (torch.randn(d, V, generator=gen, device="cuda", dtype=dt) * (2.0 / math.sqrt(d))).to(dt)
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    lift = torch.rand(T, 1, generator=gen, device="cuda") * 3
    H = (torch.randn(T, d, generator=gen, device="cuda") + lift * W.index_select(1, tokens.long()).t().float()).to(dt)
    mask = (torch.rand(T, generator=gen, device="cuda") >= c["masked"]).to(torch.uint8) if c["masked"] else None
    if mask is not None:
        tokens = torch.where(mask != 0, tokens, torch.full_like(tokens, NEG))
    return dict(H=H, W=W, tokens=tokens, mask=mask)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = case
    rand = lambda *n: torch.rand(*n, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *n: torch.randn(*n, generator=gen, device="cuda")  # noqa: E731
    if c["op"] in ("logp", "logp_step", "pair_step"):
        s = _head(c, gen)
        s["tau"] = 1.0
        T = c["T"]
        if c["op"] == "logp_step":
            s["g"], s["ge"] = -rand(T) / T, (-0.01 / T) * torch.ones(T, device="cuda")
        if c["op"] == "pair_step":
            s["cu"] = _cuts(gen, 2 * c["P"], T)
            s["ref"] = -6.0 + 2.0 * randn(T)
            s["beta"], s["kind"], s["average"] = 0.1, "sigmoid", False
            s["grad"] = torch.full((c["P"],), 1.0 / c["P"], device="cuda")
        if c["op"] != "logp":
            s["H"].requires_grad_(True)
            s["W"].requires_grad_(True)
    elif c["op"] == "policy":
        T, S = c["T"], c["S"]
        s = dict(cu=_cuts(gen, S, T))
        s["logp"] = -rand(T) * 5
        s["old"] = s["logp"] + 0.2 * randn(T)
        s["ref"] = s["logp"] + 0.5 * randn(T) if c["kl"] != "none" else None
        s["adv"] = randn(S if c["per_seq"] else T) + 0.3
        s["mask"] = (rand(T) >= c["masked"]).to(torch.uint8) if c["masked"] else None
        s["entropy"] = 3 * rand(T) if c["entropy"] else None
        if s["mask"] is not None:  # what a masked row holds is nobody's: NaN and infinities may not matter
            for k in ("old", "logp"):
                s[k] = torch.where(s["mask"] != 0, s[k], torch.full_like(s[k], math.nan if k == "old" else -math.inf))
        if c["autograd"]:
            s["logp"].requires_grad_(True)
    elif c["op"] == "preference":
        T, P = c["T"], c["P"]
        s = dict(cu=_cuts(gen, 2 * P, T), logp=-rand(T) * 5, beta=0.1, kind=c["kind"], average=c["average"])
        s["ref"] = s["logp"] + 0.3 * randn(T)
        s["mask"] = (rand(T) >= c["masked"]).to(torch.uint8) if c["masked"] else None
        s["grad"] = torch.full((P,), 1.0 / P, device="cuda") * (0.5 + rand(P))
        if s["mask"] is not None:
            s["ref"] = torch.where(s["mask"] != 0, s["ref"], torch.full_like(s["ref"], -math.inf))
        if c["autograd"]:
            s["logp"].requires_grad_(True)
    else:
        n, dt = c["n"], _TYPES[c["dtype"]]
        cuts = torch.cat([rand(n), torch.ones(1, device="cuda") * 0.001]).cumsum(0)
        ends = [0] + [int(x) for x in (cuts / cuts[-1] * c["numel"]).tolist()[:-1]] + [c["numel"]]
        flat = (1e-3 * randn(c["numel"])).to(dt)
        out = torch.empty_like(flat)
        s = dict(flat=flat, out=out)
        s["tensors"] = [flat[a:b] for a, b in zip(ends, ends[1:])]
        s["outs"] = [out[a:b] for a, b in zip(ends, ends[1:])]
        s["max_norm"] = c["ratio"] * 1e-3 * math.sqrt(c["numel"])
    return dict(s, case=c)


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    if c["op"] == "logp":
        z, logp, lse, ent, valid = _plain_logp(s)
        return dict(logp=logp, entropy=ent) if c["entropy"] else dict(logp=logp)
    if c["op"] == "logp_step":
        z, logp, lse, ent, valid = _plain_logp(s)
        dH, dW = _plain_logp_grad(s, z, lse, ent, s["g"], s["ge"] if c["entropy"] else None, valid)
        return dict(logp=logp, entropy=ent, dH=dH, dW=dW) if c["entropy"] else dict(logp=logp, dH=dH, dW=dW)
    if c["op"] == "policy":
        return _plain_policy(s, c)
    if c["op"] == "preference":
        return _plain_preference(s, s["logp"].detach(), s["grad"])
    if c["op"] == "pair_step":
        z, logp, lse, ent, valid = _plain_logp(s)
        r = _plain_preference(s, logp, s["grad"])
        dH, dW = _plain_logp_grad(s, z, lse, ent, r["dlogp"], None, valid)
        return dict(loss=r["loss"], rewards=r["rewards"], dH=dH, dW=dW)
    return _plain_clip(s)


def _own(s, c):
    import chunked_kl_loss_logit_amd as kd

    if c["op"] == "logp":
        logp, _, ent, _ = kd.token_logp_forward(s["H"], s["W"], s["tokens"], s["mask"], s["tau"],
                                                want_entropy=c["entropy"])
        return dict(logp=logp, entropy=ent) if c["entropy"] else dict(logp=logp)
    if c["op"] == "logp_step":
        got = kd.token_logp(s["H"], s["W"], s["tokens"], s["mask"], s["tau"], want_entropy=c["entropy"],
                            keep_logits=True)
        if not c["entropy"]:
            dH, dW = torch.autograd.grad(got, (s["H"], s["W"]), s["g"])
            return dict(logp=got.detach(), dH=dH, dW=dW)
        dH, dW = torch.autograd.grad(got, (s["H"], s["W"]), (s["g"], s["ge"]))
        return dict(logp=got[0].detach(), entropy=got[1].detach(), dH=dH, dW=dW)
    if c["op"] == "policy":
        kw = dict(ref_logp=s["ref"], entropy=s["entropy"], cu_seqlens=s["cu"], clip_low=0.2, clip_high=0.25,
                  dual_clip=c["dual"], kl_weight=0.0 if c["kl"] == "none" else 0.05,
                  kl_kind="k3" if c["kl"] == "none" else c["kl"], entropy_weight=0.01 if c["entropy"] else 0.0,
                  reduction=c["reduction"], per_sequence=c["per_seq"])
        if c["autograd"]:
            loss, stats = kd.policy_loss(s["logp"], s["old"], s["adv"], s["mask"], **kw)
            return dict(stats=stats, dlogp=torch.autograd.grad(loss, s["logp"])[0])
        stats, dlogp, dent = kd.policy_loss_forward_backward(s["logp"], s["old"], s["adv"], s["mask"], **kw)
        return dict(stats=stats, dlogp=dlogp, dent=dent) if c["entropy"] else dict(stats=stats, dlogp=dlogp)
    if c["op"] == "preference":
        kw = dict(ref_logp=s["ref"], beta=s["beta"], kind=s["kind"], average=s["average"], label_smoothing=0.05 if s["kind"] == "sigmoid" else 0.0)
        if c["autograd"]:
            loss, rewards = kd.preference_loss(s["logp"], s["cu"], s["mask"], **kw)
            return dict(loss=loss.detach(), rewards=rewards, dlogp=torch.autograd.grad(loss, s["logp"], s["grad"])[0])
        loss, rewards, dlogp = kd.preference_loss_forward_backward(s["logp"], s["cu"], s["mask"], s["grad"], **kw)
        return dict(loss=loss, rewards=rewards, dlogp=dlogp)
    if c["op"] == "pair_step":
        logp = kd.token_logp(s["H"], s["W"], s["tokens"], s["mask"], s["tau"], keep_logits=True)
        loss, rewards = kd.preference_loss(logp, s["cu"], s["mask"], ref_logp=s["ref"], beta=s["beta"], kind=s["kind"],
                                           average=s["average"], label_smoothing=0.05)
        dH, dW = torch.autograd.grad(loss, (s["H"], s["W"]), s["grad"])
        return dict(loss=loss.detach(), rewards=rewards, dH=dH, dW=dW)
    norm = kd.clip_grad_norm(s["tensors"], s["max_norm"], out=s["outs"])
    return dict(norm=norm, out=s["out"])


# ------------------------------------------------------------------ plain forms, 32 bits
def _plain_logp(s):
    H, W, tokens, mask = s["H"].detach(), s["W"].detach(), s["tokens"], s["mask"]
    valid = torch.ones_like(tokens, dtype=torch.bool) if mask is None else mask != 0
    z = (H.float() @ W.float()) / s["tau"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    y = torch.where(valid, tokens, 0).long()
    logp = torch.where(valid, z.gather(1, y[:, None])[:, 0] - lse, 0.0)
    ent = None
    if s["case"].get("entropy"):
        ent = torch.where(valid, torch.log(total[:, 0]) - (e * (z - top)).sum(1) / total[:, 0], 0.0)
    return z, logp, lse, ent, valid


def _plain_logp_grad(s, z, lse, ent, g, ge, valid):
    H, W = s["H"].detach(), s["W"].detach()
    lq = z - lse[:, None]
    g = torch.where(valid, g, 0.0)
    a = g[:, None] if ge is None else g[:, None] + torch.where(valid, ge, 0.0)[:, None] * (ent[:, None] + lq)
    dz = -torch.exp(lq) * a
    y = torch.where(valid, s["tokens"], 0).long()[:, None]
    dz.scatter_add_(1, y, g[:, None])
    dz = dz / s["tau"]
    return (dz @ W.float().t()).to(H.dtype), (H.float().t() @ dz).to(W.dtype)


def _places(cu, T):
    """The sequence of each of T tokens."""
    at = torch.arange(T, device=cu.device)
    return torch.searchsorted(cu[1:].long().contiguous(), at, right=True)


def _plain_policy(s, c):
    T, S = c["T"], c["S"]
    logp, old, ref, ent = s["logp"].detach(), s["old"], s["ref"], s["entropy"]
    valid = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    seq = _places(s["cu"], T)
    adv = s["adv"][seq] if c["per_seq"] else s["adv"]
    # 64 bits up to the comparison with the clip's borders
    ratio = torch.where(valid, torch.exp(logp.double() - old.double()), 1.0)
    cut = ((adv > 0) & (ratio > 1 + 0.25)) | ((adv < 0) & (ratio < 1 - 0.2))
    r = ratio.float()
    pg = -torch.minimum(r * adv, r.clamp(1 - 0.2, 1 + 0.25) * adv)
    if c["dual"]:
        cut = cut | ((adv < 0) & (ratio > c["dual"]))
        pg = torch.where(adv < 0, torch.minimum(pg, -c["dual"] * adv), pg)
    grad = torch.where(cut, 0.0, -adv * r)
    kl = torch.zeros_like(pg)
    if c["kl"] != "none":
        d = torch.where(valid, ref - logp, 0.0).double()
        kl, dkl = {"k1": (-d, torch.ones_like(d)), "k2": (d * d / 2, -d), "k3": (torch.expm1(d) - d, -torch.expm1(d))}[c["kl"]]
        grad = grad + 0.05 * dkl.float()
    loss = pg.double() + (0.05 * kl.double() if c["kl"] != "none" else 0)
    if ent is not None:
        loss = loss - 0.01 * ent.double()
    n = valid.double().sum()
    if c["reduction"] == "sum":
        w = torch.ones(T, device="cuda", dtype=torch.float64)
    elif c["reduction"] == "token":
        w = torch.full((T,), 1.0, device="cuda", dtype=torch.float64) / n.clamp(min=1)
    else:
        per = torch.zeros(S, device="cuda", dtype=torch.float64).index_add_(0, seq, valid.double())
        w = (1 / (per.clamp(min=1) * (per > 0).double().sum().clamp(min=1)))[seq]
    w = torch.where(valid, w, 0.0)
    total = lambda x: (w * torch.where(valid, x.double(), 0.0)).sum()  # noqa: E731
    stats = torch.stack([total(loss), total(pg), total(kl), total(ent) if ent is not None else n * 0, total(cut), n])
    got = dict(stats=stats.float(), dlogp=torch.where(valid, w * grad, 0.0).float())
    if ent is not None and not c["autograd"]:
        got["dent"] = (-0.01 * w).float()
    return got


def _plain_preference(s, logp, grad):
    T, P, beta = logp.numel(), s["cu"].numel() // 2, s["beta"]
    valid = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    seq = _places(s["cu"], T)
    x = torch.where(valid, logp.double() - s["ref"].double(), 0.0)
    sums = torch.zeros(2 * P, device="cuda", dtype=torch.float64).index_add_(0, seq, x)
    n = torch.zeros(2 * P, device="cuda", dtype=torch.float64).index_add_(0, seq, valid.double()).clamp(min=1)
    if s["average"]:
        sums = sums / n
    D = sums[:P] - sums[P:]
    h = beta * D
    eps = 0.05
    if s["kind"] == "sigmoid":
        loss = (1 - eps) * torch.log1p(torch.exp(-h.abs())) + eps * torch.log1p(torch.exp(-h.abs())) \
            + (1 - eps) * (-h).clamp(min=0) + eps * h.clamp(min=0)
        dD = beta * (1 / (1 + torch.exp(-h)) - (1 - eps))
    elif s["kind"] == "hinge":
        loss, dD = (1 - h).clamp(min=0), torch.where(h < 1, -beta, 0.0)
    else:
        loss, dD = (D - 1 / (2 * beta)) ** 2, 2 * (D - 1 / (2 * beta))
    k = grad.double() * dD
    k = torch.cat([k, -k]) / (n if s["average"] else 1)
    return dict(loss=loss.float(), rewards=(beta * sums).float(), dlogp=torch.where(valid, k[seq], 0.0).float())


def _plain_clip(s):
    norm = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["tensors"]]).sum().sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    [o.copy_(t.float() * scale) for t, o in zip(s["tensors"], s["outs"])]
    return dict(norm=norm.float(), out=s["out"])


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_logp(s, g=None, ge=None, block=1024, pairs=None):
    """Block by block of rows; `pairs(logp)` gives the rows' upstream gradients where they depend on all rows."""
    T, W = s["H"].shape[0], s["W"].detach().double()
    out = {"logp": torch.zeros(T, device="cuda", dtype=torch.float64), "entropy": torch.zeros(T, device="cuda", dtype=torch.float64)}
    keep = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    for rows in keep.split(block):
        lq = torch.log_softmax((s["H"].detach()[rows].double() @ W) / s["tau"], 1)
        out["logp"][rows] = lq[torch.arange(len(rows), device="cuda"), s["tokens"][rows].long()]
        out["entropy"][rows] = -(lq.exp() * lq).sum(1)
    more = {}
    if pairs is not None:
        more = pairs(out["logp"])
        g = more["dlogp"]
    if g is not None:
        dH, dW = torch.zeros(T, W.shape[0], device="cuda", dtype=torch.float64), torch.zeros_like(W)
        for rows in keep.split(block):
            h = s["H"].detach()[rows].double()
            lq = torch.log_softmax((h @ W) / s["tau"], 1)
            q = lq.exp()
            dz = -q * g[rows].double()[:, None]
            dz[torch.arange(len(rows), device="cuda"), s["tokens"][rows].long()] += g[rows].double()
            if ge is not None:
                dz -= ge[rows].double()[:, None] * q * (lq + out["entropy"][rows][:, None])
            dz /= s["tau"]
            dH[rows] = dz @ W.t()
            dW += h.t() @ dz
        out.update(dH=dH, dW=dW)
    out.update(more)
    return out


def _exact_policy(s, c):
    T, S = c["T"], c["S"]
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(S, device="cuda"), cu[1:] - cu[:-1])
    ok = torch.arange(T, device="cuda") if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    q = seq[ok]
    lp, lo = s["logp"].detach()[ok].double(), s["old"][ok].double()
    A = (s["adv"][q] if c["per_seq"] else s["adv"][ok]).double()
    r = (lp - lo).exp()
    inside = (r <= 1.25) & (r >= 0.8)
    free = inside | ((A > 0) & (r < 0.8)) | ((A < 0) & (r > 1.25)) | (A == 0)
    pg = torch.where(free, -r * A, -torch.where(A > 0, 1.25, 0.8) * A)
    if c["dual"]:
        far = (A < 0) & (r > c["dual"])
        pg, free = torch.where(far, -c["dual"] * A, pg), free & ~far
    g = torch.where(free, -r * A, 0.0)
    kl = torch.zeros_like(pg)
    if c["kl"] != "none":
        t = lp - s["ref"][ok].double()
        if c["kl"] == "k1":
            kl, dk = t, torch.ones_like(t)
        elif c["kl"] == "k2":
            kl, dk = t.square() / 2, t
        else:
            kl, dk = torch.expm1(-t) + t, -torch.expm1(-t)
        g = g + 0.05 * dk
    H = s["entropy"][ok].double() if s["entropy"] is not None else torch.zeros_like(pg)
    wH = 0.01 if s["entropy"] is not None else 0.0
    if c["reduction"] == "sum":
        w = torch.ones_like(pg)
    elif c["reduction"] == "token":
        w = torch.ones_like(pg) / max(1, len(ok))
    else:
        n = torch.bincount(q, minlength=S)
        w = 1.0 / (n[q].double() * max(1, int((n > 0).sum())))
    full = lambda v: torch.zeros(T, device="cuda", dtype=torch.float64).index_copy_(0, ok, v)  # noqa: E731
    kw = 0.05 if c["kl"] != "none" else 0.0
    stats = torch.stack([(w * (pg + kw * kl - wH * H)).sum(), (w * pg).sum(), (w * kl).sum(), (w * H).sum(),
                         (w * (~free).double()).sum(), torch.tensor(float(len(ok)), device="cuda", dtype=torch.float64)])
    got = dict(stats=stats, dlogp=full(w * g))
    if s["entropy"] is not None and not c["autograd"]:
        got["dent"] = full(-0.01 * w)
    return got


def _exact_preference(s, logp, grad):
    P, b = s["cu"].numel() // 2, s["beta"]
    ok = torch.ones(logp.numel(), dtype=torch.float64, device="cuda") if s["mask"] is None else (s["mask"] != 0).double()
    x = torch.where(ok > 0, logp.double() - s["ref"].double(), torch.zeros_like(ok))
    zero = torch.zeros(1, dtype=torch.float64, device="cuda")
    at = s["cu"].long()
    cx, cn = torch.cat([zero, x.cumsum(0)])[at], torch.cat([zero, ok.cumsum(0)])[at]
    total, n = cx[1:] - cx[:-1], (cn[1:] - cn[:-1]).clamp(min=1)
    value = total / n if s["average"] else total
    D = (value[:P] - value[P:]).requires_grad_(True)
    if s["kind"] == "sigmoid":
        loss = -0.95 * torch.nn.functional.logsigmoid(b * D) - 0.05 * torch.nn.functional.logsigmoid(-b * D)
    elif s["kind"] == "hinge":
        loss = torch.relu(1 - b * D)
    else:
        loss = (D - 0.5 / b).square()
    dD, = torch.autograd.grad(loss, D, grad.double())
    per = torch.cat([dD, -dD]) / (n if s["average"] else torch.ones_like(n))
    dlogp = torch.repeat_interleave(per, at[1:] - at[:-1]) * ok
    return dict(loss=loss.detach(), rewards=b * value, dlogp=dlogp)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "logp":
        r = _exact_logp(s)
        return {k: r[k] for k in (("logp", "entropy") if c["entropy"] else ("logp",))}
    if c["op"] == "logp_step":
        r = _exact_logp(s, s["g"], s["ge"] if c["entropy"] else None)
        return {k: r[k] for k in (("logp", "entropy", "dH", "dW") if c["entropy"] else ("logp", "dH", "dW"))}
    if c["op"] == "policy":
        return _exact_policy(s, c)
    if c["op"] == "preference":
        return _exact_preference(s, s["logp"].detach(), s["grad"])
    if c["op"] == "pair_step":
        r = _exact_logp(s, pairs=lambda logp: _exact_preference(s, logp, s["grad"]))
        return {k: r[k] for k in ("loss", "rewards", "dH", "dW")}
    norm = torch.sqrt(sum((x.double() ** 2).sum() for x in s["flat"].split(1 << 26)))
    scale = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return dict(norm=norm, out=s["flat"].double() * scale)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] in ("logp", "logp_step", "pair_step"):
        T, d, V = c["T"], c["d"], c["V"]
        e = 2 if c["dtype"] == "bf16" else 4
        rows = T * (1 - c["masked"])
        head = d * V * e
        if c["op"] == "logp":
            return {"bytes": head + rows * d * e + 13 * T, "flops": 2 * rows * d * V}
        return {"bytes": 2 * head + 2 * T * d * e + 21 * T, "flops": 6 * rows * d * V}
    if c["op"] == "policy":
        arrays = 3 + (c["kl"] != "none") + 2 * bool(c["entropy"]) + (not c["per_seq"])
        return {"bytes": c["T"] * (4 * arrays + bool(c["masked"])), "flops": 30 * c["T"]}
    if c["op"] == "preference":
        return {"bytes": c["T"] * (12 + bool(c["masked"])), "flops": 4 * c["T"]}
    e = 4 if c["dtype"] == "f32" else 2
    return {"bytes": 2 * e * c["numel"], "flops": 3 * c["numel"]}

"""Plain 64-bit forms of the policy- and preference-training operators, on the CPU, and the error bounds their tests
use.  u(t) is half a step of a type, the largest relative error of one rounding."""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ token log-probabilities
def make_head(T, d, V, dtype, seed, scale=2.0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(d, V, generator=g) * scale / math.sqrt(d)).to(dtype)
    tokens = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    H = (torch.randn(T, d, generator=g) + torch.rand(T, 1, generator=g) * W[:, tokens.long()].float().t()).to(dtype)
    mask = None if not masked else (torch.rand(T, generator=g) >= masked).to(torch.uint8)
    return H, W, tokens, mask


def logp_reference(H, W, tokens, mask, tau, g=None, ge=None):
    """logp, lse, entropy, dH, dW in 64 bits, and the bounds of each for this path's roundings.

    z is a sum of d products in 32 bits: off by at most d u |h|.|w| (a(t) below, the row's largest, over tau).  logp and
    lse move by at most twice that, 2^x and log2 by a few u of the result.  d ent / d s = -q (log q + ent) sums to at
    most 2 ent + 2 <= 2 log V + 2 in absolute value.  dZ is rounded to the inputs' type (twice its bits up to 32 rows);
    its own 32-bit error is q's relative one, 2 a plus a few u.  dH and dW then sum V or T products in 32 bits and are
    rounded once."""
    T, d = H.shape
    V = W.shape[1]
    Hd, Wd = H.double(), W.double()
    ok = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    Hd = torch.where(ok[:, None], Hd, torch.zeros(()).double())
    y = torch.where(ok & (tokens >= 0) & (tokens < V), tokens, 0).long()[:, None]
    s = Hd @ Wd / tau
    lse = torch.logsumexp(s, 1)
    lq = s - lse[:, None]
    q = lq.exp()
    ent = -(q * lq).sum(1)
    zero = torch.zeros(T).double()
    off = (d + 16) * U32 * (Hd.abs() @ Wd.abs()).amax(1) / tau
    r = dict(logp=torch.where(ok, lq.gather(1, y)[:, 0], zero), lse=torch.where(ok, lse, zero),
             entropy=torch.where(ok, ent, zero))
    base = 2 * off + 2.0 ** -20 * (1 + lse.abs())
    bound = dict(logp=base + 2.0 ** -20 * lq.gather(1, y)[:, 0].abs(), lse=base,
                 entropy=2 * off * (2 + 2 * math.log(V)) + 2.0 ** -18 * (1 + ent))
    if g is None and ge is None:
        return r, bound
    g = zero if g is None else torch.where(ok, g.double(), zero)
    ge = zero if ge is None else torch.where(ok, ge.double(), zero)
    dz = -q * (g[:, None] + ge[:, None] * (ent[:, None] + lq))
    size = q * (g.abs()[:, None] + ge.abs()[:, None] * (ent[:, None] + lq.abs() + 1))
    dz.scatter_add_(1, y, g[:, None])
    size.scatter_add_(1, y, g.abs()[:, None])
    dz, size = dz / tau, size / tau
    r["dH"], r["dW"] = dz @ Wd.t(), Hd.t() @ dz
    uz = half_step(H.dtype)
    udz = min(uz, 2.0 ** -16) if T <= 32 else uz  # up to 32 rows keep what the rounding leaves, rounded again
    rel = (udz + 4 * base[:, None] + 2.0 ** -18)
    szW, Hsz = (rel * size) @ Wd.abs().t(), Hd.abs().t() @ (rel * size)
    bound["dH"] = szW + V * U32 * (size @ Wd.abs().t()) + uz * (r["dH"].abs() + szW) + 1e-30
    bound["dW"] = Hsz + T * U32 * (Hd.abs().t() @ size) + uz * (r["dW"].abs() + Hsz) + 1e-30
    return r, bound


def within(got, want, bound, what):
    got = got.detach().double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} beyond the bound, worst by {over.max():.3e}"


# ------------------------------------------------------------------ policy loss
def policy_reference(logp, old, adv, mask=None, ref_logp=None, entropy=None, cu_seqlens=None, clip_low=0.2,
                     clip_high=0.2, dual_clip=0.0, kl_weight=0.0, kl_kind="k3", entropy_weight=0.0, reduction="token",
                     per_sequence=False):
    """stats [6], grad_logp, grad_entropy in 64 bits, token by token."""
    T = logp.numel()
    cu = None if cu_seqlens is None else cu_seqlens.tolist()
    S = 1 if cu is None else len(cu) - 1
    seq = [0] * T if cu is None else [-1] * T
    if cu is not None:
        for s in range(S):
            for t in range(cu[s], cu[s + 1]):
                seq[t] = s
    ok = [seq[t] >= 0 and (mask is None or bool(mask[t])) for t in range(T)]
    n = [0] * S
    for t in range(T):
        if ok[t]:
            n[seq[t]] += 1
    N, some = sum(n), sum(k > 0 for k in n)
    w = {"sum": lambda s: 1.0, "token": lambda s: 1.0 / N, "sequence": lambda s: 1.0 / (n[s] * some)}[reduction]
    stats = [0.0] * 6
    stats[5] = float(N)
    g, ge = torch.zeros(T).double(), torch.zeros(T).double()
    for t in range(T):
        if not ok[t]:
            continue
        A = float(adv[seq[t] if per_sequence else t])
        r = math.exp(float(logp[t]) - float(old[t]))
        cut = (A > 0 and r > 1 + clip_high) or (A < 0 and r < 1 - clip_low)
        pg = -min(r * A, min(max(r, 1 - clip_low), 1 + clip_high) * A)
        if dual_clip and A < 0 and pg > -dual_clip * A:
            pg, cut = -dual_clip * A, True
        d = 0.0 if cut else -A * r
        kl = 0.0
        if ref_logp is not None:
            x = float(ref_logp[t]) - float(logp[t])
            kl, dk = {"k1": (-x, 1.0), "k2": (x * x / 2, -x), "k3": (math.expm1(x) - x, -math.expm1(x))}[kl_kind]
            d += kl_weight * dk
        h = 0.0 if entropy is None else float(entropy[t])
        ws = w(seq[t])
        for i, v in enumerate((pg + kl_weight * kl - entropy_weight * h, pg, kl, h, float(cut))):
            stats[i] += ws * v
        g[t], ge[t] = ws * d, -ws * entropy_weight
    return torch.tensor(stats, dtype=torch.float64), g, ge


# ------------------------------------------------------------------ preference loss
def preference_reference(logp, cu_seqlens, mask=None, ref_logp=None, beta=0.1, kind="sigmoid", label_smoothing=0.0,
                         margin=0.0, average=False, grad=None):
    """loss [P], rewards [2P], grad_logp in 64 bits, and the sums' absolute size per sequence."""
    T, cu = logp.numel(), cu_seqlens.tolist()
    P = (len(cu) - 1) // 2
    ok = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    x = logp.double() - (0.0 if ref_logp is None else ref_logp.double())
    R, n = [], []
    for s in range(2 * P):
        at = [t for t in range(cu[s], cu[s + 1]) if ok[t]]
        n.append(len(at))
        R.append(math.fsum(float(x[t]) for t in at) / (max(1, len(at)) if average else 1))
    loss, g = [], torch.zeros(T).double()
    for p in range(P):
        D = R[p] - R[P + p]
        h = beta * D - margin
        sig = lambda v: 1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v))  # noqa: E731
        soft = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))  # noqa: E731
        if kind == "sigmoid":
            loss.append((1 - label_smoothing) * soft(-h) + label_smoothing * soft(h))
            dD = beta * (label_smoothing - sig(-h))
        elif kind == "hinge":
            loss.append(max(0.0, 1 - h))
            dD = -beta if h < 1 else 0.0
        else:
            loss.append((D - 1 / (2 * beta)) ** 2)
            dD = 2 * (D - 1 / (2 * beta))
        if grad is not None:
            for s, sign in ((p, 1), (P + p, -1)):
                for t in range(cu[s], cu[s + 1]):
                    if ok[t]:
                        g[t] = sign * float(grad[p]) * dD / (n[s] if average else 1)
    return (torch.tensor(loss, dtype=torch.float64), torch.tensor([beta * r for r in R], dtype=torch.float64), g)


def near(got, want, what, rel=4 * U32, small=1e-30):
    """Every value within `rel` of its own size: results of 64-bit arithmetic, rounded once to 32."""
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, {tuple(want.shape)} wanted"
    over = (got - want).abs() - rel * want.abs() - small
    assert not torch.isnan(got).any() and (over <= 0).all(), f"{what}: worst beyond by {over.max():.3e}"

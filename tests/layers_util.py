"""Plain 64-bit forms of the operators of kdlayers.h, on the CPU, and the error bounds their tests use.

u(t) = half a step of a type, the largest relative error of one rounding; U32 that of float32.  TINY(t): half the
smallest step of a type, what a rounding in its subnormal range may be off by."""
import torch

U32 = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def rounded(y, before, dtype):
    """The bound of a value y that is off by `before` and then rounded to dtype."""
    return before + half_step(dtype) * (y.abs() + before) + tiny(dtype)


def check(got, want, bound, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    off = (got - want).abs()[~nan]
    worst = (off - bound.expand(want.shape)[~nan]).max() if off.numel() else -1
    assert worst <= 0, f"{what}: off by up to {off.max():.3e}, {worst:.3e} over its bound"


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ token embeddings
def make_tokens(T, V, seed, masked=0.0, hot=0.3):
    """Tokens, some of them very frequent; the mask's rows hold tokens of no vocabulary."""
    g = gen(seed)
    tokens = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    tokens = torch.where(torch.rand(T, generator=g) < hot, torch.tensor(V // 2, dtype=torch.int32), tokens)
    mask = None
    if masked:
        mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8)
        tokens = torch.where(mask != 0, tokens, torch.tensor(-7, dtype=torch.int32))
    return tokens, mask


def valid_rows(mask, T):
    return torch.ones(T, dtype=torch.bool) if mask is None else mask != 0


def embedding_reference(tokens, table, mask, scale):
    """One product in 32 bits, rounded."""
    T, (V, d) = tokens.numel(), table.shape
    ok = valid_rows(mask, T)
    inside = (tokens >= 0) & (tokens < V)
    y = table.double()[torch.where(inside, tokens, 0).long()] * scale
    y[~inside] = float("nan")
    y[~ok] = 0
    return y, rounded(y.nan_to_num(), y.nan_to_num().abs() * U32, table.dtype)


def embedding_grad_reference(grad, tokens, mask, scale, V, dtype, was=None):
    """A sum of n terms in any order of pairs is off by at most (n - 1) u sum |terms|; one product by the scale and,
    with accumulate, one sum follow, and the rounding."""
    T, d = grad.shape
    ok = valid_rows(mask, T) & (tokens >= 0) & (tokens < V)
    g = grad.double()[ok]
    at = tokens.long()[ok]
    y = torch.zeros(V, d, dtype=torch.float64).index_add_(0, at, g)
    size = torch.zeros(V, d, dtype=torch.float64).index_add_(0, at, g.abs())
    n = torch.bincount(at, minlength=V).double()[:, None]
    y, off = y * scale, (n + 2) * U32 * size * abs(scale)
    if was is not None:
        y = torch.where(n > 0, was.double() + y, was.double())
        off = torch.where(n > 0, off + U32 * (y.abs() + off), 0)
    return y, rounded(y, off, dtype)


# ------------------------------------------------------------------ rows in 8 bits
def e4m3_grid():
    """The format's values that are not negative, in ascending order."""
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def rows_reference(x, kind, group):
    """q (the values, in units of the scale) and scale, exactly: the quotient of two 24-bit numbers lies 2^-34 of
    itself or more from the middle of two steps, or on it, and its error in 64 bits is 2^-53."""
    T, d = x.shape
    size = group or d
    top = 127.0 if kind == "int8" else 448.0
    q, scales = torch.zeros(T, d, dtype=torch.float64), []
    for a in range(0, d, size):
        part = x[:, a:a + size].double()
        s = (part.abs().amax(1) / top).float()
        bad = ~torch.isfinite(part).all(1)
        r = torch.where((s > 0)[:, None], part / s.double()[:, None], torch.zeros(()).double()).clamp(-top, top)
        if kind == "int8":
            v = torch.round(r)  # ties to even
        else:
            grid = e4m3_grid()
            hi = torch.searchsorted(grid, r.abs().contiguous()).clamp(max=126)
            lo = (hi - 1).clamp(min=0)
            up, down = grid[hi] - r.abs(), r.abs() - grid[lo]
            v = grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)] * torch.sign(r)
        v[bad] = 0
        q[:, a:a + size] = v
        scales.append(torch.where(bad, float("nan"), s))
    return q, torch.stack(scales, 1)


def rows_values(q, scale, group):
    """What rows in 8 bits stand for, in 64 bits."""
    d = q.shape[1]
    return q.double() * scale.double().repeat_interleave(group or d, 1)[:, :d]


# ------------------------------------------------------------------ layer norm
def make_rows(T, d, dtype, seed, offset=0.3, masked=0.0):
    g = gen(seed)
    x = (torch.randn(T, d, generator=g) * (0.5 + torch.rand(T, 1, generator=g)) + offset).to(dtype)
    mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    if mask is not None:
        x[mask == 0] = float("nan")
    return x, mask


def chain(d):
    """The most additions on the way of a term into a sum over a row: at most 32 in a lane (or d / 1024 where a row is
    not held in registers), 6 over a wave, 16 over waves, and a few for the products before and after."""
    return max(32, d / 1024 + 8) + 6 + 16 + 6


def norm_reference(x, w, b, mask, eps, grad=None, kept=None):
    """y, mean, rstd (and dx, dw, db) in 64 bits, and the bounds for sums of `chain` roundings: the mean is off by
    chain u mean|x|, h = (x - mean) r by r times that and by r's own relative error (chain / 2 + 3) u, and whatever
    follows by what its inputs are off, plus u for each operation."""
    T, d = x.shape
    ok = valid_rows(mask, T)
    xd = torch.where(ok[:, None], x.double(), torch.zeros(()).double())
    wd = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    bd = torch.zeros(d, dtype=torch.float64) if b is None else b.double()
    L = chain(d)
    mean = xd.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((xd - mean) ** 2).mean(1, keepdim=True) + eps)
    h = (xd - mean) * r
    dmean = L * U32 * xd.abs().mean(1, keepdim=True)
    # the variance around a mean that is off by dmean is off by dmean^2, and by the sum's L u of itself
    rel_r = (L / 2 + 4) * U32 + (dmean * r) ** 2
    dh = r * dmean + h.abs() * (rel_r + 2 * U32)
    y = h * wd + bd
    off = wd.abs() * dh + 2 * U32 * (h * wd).abs() + U32 * y.abs()
    zero = ~ok[:, None]
    res = dict(y=y.masked_fill(zero, 0), mean=mean[:, 0].masked_fill(~ok, 0), rstd=r[:, 0].masked_fill(~ok, 0))
    bound = dict(y=rounded(y, off, x.dtype), mean=dmean[:, 0] + tiny(torch.float32), rstd=(rel_r * r)[:, 0])
    if grad is None:
        return res, bound
    gd = torch.where(ok[:, None], grad.double(), torch.zeros(()).double())
    if kept is not None:  # the row as 8 bits hold it: one more rounding
        xd = torch.where(ok[:, None], kept, torch.zeros(()).double())
        h = (xd - mean) * r
        dh = r * (dmean + U32 * xd.abs()) + h.abs() * (rel_r + 2 * U32)
    g = gd * wd
    c0, c1 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dc0 = (L + 2) * U32 * g.abs().mean(1, keepdim=True)
    dc1 = (L + 4) * U32 * (g * h).abs().mean(1, keepdim=True) + (g.abs() * dh).mean(1, keepdim=True)
    dx = r * (g - c0 - h * c1)
    off = r * (dc0 + h.abs() * dc1 + dh * c1.abs() + 4 * U32 * (g.abs() + c0.abs() + (h * c1).abs())) + rel_r * dx.abs()
    # T rows in any order of pairs
    dw, db = (gd * h).sum(0), gd.sum(0)
    offw = (T + 4) * U32 * (gd * h).abs().sum(0) + (gd.abs() * dh).sum(0)
    offb = (T + 4) * U32 * gd.abs().sum(0)
    wt = x.dtype if w is None and b is None else (b if w is None else w).dtype
    res.update(dx=dx.masked_fill(zero, 0), dw=dw, db=db)
    bound.update(dx=rounded(dx, off, x.dtype), dw=rounded(dw, offw, wt), db=rounded(db, offb, wt))
    return res, bound


# ------------------------------------------------------------------ product of 8-bit integers
def make_int8(T, d, V, seed):
    g = gen(seed)
    x = torch.randint(-128, 128, (T, d), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (V, d), generator=g, dtype=torch.int8)
    return x, torch.rand(T, generator=g) * 1e-2 + 1e-4, w, torch.rand(V, generator=g) * 1e-2 + 1e-4


def int8_reference(x, sx, w, sw, dtype):
    """Sums of up to 2^17 products below 2^14 are exact in 64 bits; the 32-bit integer's conversion and the two
    products round once each."""
    y = (x.double() @ w.double().t()) * sx.double()[:, None] * sw.double()
    return y, rounded(y, 3.01 * U32 * y.abs(), dtype)

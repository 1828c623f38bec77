"""What the operators on the model's side of the output head cost and how exact they are.

Each case is one call (or one training step) as a program makes it: token embeddings from a table or from the head
itself, layer norm, rows held in 8 bits, and the product of 8-bit integers with a scale for each token and channel.
`run` computes them in plain torch where `own` is false, and with this package's operators where it is true.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the tokens of one decoding step of a few sequences: latency
        dict(name="embed few", op="embed", T=5, V=32000, d=2048, dtype="bf16", tied=False, masked=0.0),
        # a batch through a model whose embedding is its output head (columns of W), padding masked
        dict(name="embed head", op="embed", T=4096, V=128256, d=2048, dtype="bf16", tied=True, masked=0.1),
        # a training step's lookup and gradient of a large table, tokens as frequent as in text
        dict(name="embed step", op="embed_step", T=16384, V=128256, d=2048, dtype="bf16", grad="bf16", tied=False,
             masked=0.0),
        # the gradient of a tied head's columns in float32, as the head's own gradient is held
        dict(name="embed head step", op="embed_step", T=3001, V=32000, d=2048, dtype="bf16", grad="f32", tied=True,
             masked=0.1),
        # the norm before the head in one decoding step: latency
        dict(name="norm few", op="norm", T=3, d=4096, dtype="bf16", weight="bf16", bias=True, masked=0.0),
        # a training step's norm, forward and backward, through autograd
        dict(name="norm step", op="norm_step", T=16384, d=4096, dtype="bf16", weight="bf16", bias=True, masked=0.0,
             kind="none", group=0),
        # a small float32 model of an odd width, a padded batch
        dict(name="norm step odd", op="norm_step", T=777, d=1337, dtype="f32", weight="f32", bias=True, masked=0.2,
             kind="none", group=0),
        # the same step where the backward pass reads its input from 8 bits
        dict(name="norm step in 8 bits", op="norm_step", T=8192, d=8192, dtype="bf16", weight="f32", bias=False,
             masked=0.0, kind="int8", group=128),
        # hidden states of a batch put away in 8 bits and taken back
        dict(name="rows int8", op="rows", T=16384, d=4096, dtype="bf16", kind="int8", group=128),
        # a few float32 rows of an odd width in 8-bit floating point, one scale a row
        dict(name="rows e4m3 odd", op="rows", T=100, d=1001, dtype="f32", kind="e4m3", group=0),
        # a frozen 8-bit head for the tokens of one decoding step: one read of the head
        dict(name="int8 few", op="int8", T=4, d=4096, V=32000, out="f32"),
        # the teacher's logits of a batch through a frozen 8-bit head
        dict(name="int8 batch", op="int8", T=4001, d=4096, V=128256, out="bf16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["embed", "embed_step", "embed_step", "norm", "norm_step", "norm_step", "rows", "rows", "int8",
                     "int8"])
    masked = rng.choice([0.0, rng.uniform(0.05, 0.6)])
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    if op in ("embed", "embed_step"):
        d = rng.choice([8 * _log(rng, 8, 512), _log(rng, 64, 2048)])
        tied = rng.random() < 0.4
        V = _log(rng, 500, min(128256, 128256 * 2048 // d) // (4 if tied else 1))
        T = _log(rng, 1, max(16, min(16384, 16384 * 2048 // d) // (4 if tied else 1)))
        c = dict(op=op, T=T, V=V, d=d, dtype=dtype, tied=tied, masked=masked if T >= 16 else 0.0)
        return c if op == "embed" else dict(c, grad=rng.choice([dtype, "f32"]))
    if op in ("norm", "norm_step"):
        d = rng.choice([64 * _log(rng, 1, 160), _log(rng, 33, 12000)])
        T = _log(rng, 1, max(16, min(65536, 16384 * 4096 // d)))
        c = dict(op=op, T=T, d=d, dtype=dtype, weight=rng.choice([dtype, "f32"]), bias=rng.random() < 0.7,
                 masked=masked if T >= 16 else 0.0)
        if op == "norm":
            return c
        return dict(c, kind=rng.choice(["none", "none", "int8", "e4m3"]), group=rng.choice([0, 32, 64, 128, 256]))
    if op == "rows":
        d = rng.choice([64 * _log(rng, 1, 160), _log(rng, 33, 12000)])
        T = _log(rng, 1, max(16, min(65536, 16384 * 4096 // d)))
        return dict(op=op, T=T, d=d, dtype=dtype, kind=rng.choice(["int8", "e4m3"]),
                    group=rng.choice([0, 32, 64, 128, 256, 512]))
    d = 16 * _log(rng, 4, 512)
    V = _log(rng, 300, 128256)
    T = _log(rng, 1, max(16, min(4096, 4001 * 4096 * 128256 // (d * V))))
    return dict(op=op, T=T, d=d, V=V, out=rng.choice(["bf16", "f32", "f16"]))


# ------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}


def _activations(T, d, gen):
    """Hidden states: rows of different sizes, a few channels much larger than the others, an offset."""
    x = torch.randn(T, d, generator=gen, device="cuda")
    x *= 0.5 + torch.rand(T, 1, generator=gen, device="cuda")
    loud = torch.rand(d, generator=gen, device="cuda") < 0.01
    return x * torch.where(loud, 8.0, 1.0) + 0.1


def _tokens(T, V, gen):
    """Tokens about as frequent as in text: the k-th with a probability near 1 / k."""
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
    return (V ** u - 1).clamp(0, V - 1).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = case
    rand = lambda *n: torch.rand(*n, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *n: torch.randn(*n, generator=gen, device="cuda")  # noqa: E731
    s = dict(case=c)
    dt = _TYPES[c.get("dtype", "f32")]
    if c.get("masked"):
        s["mask"] = (rand(c["T"]) >= c["masked"]).to(torch.uint8)
    else:
        s["mask"] = None
    if c["op"] in ("embed", "embed_step"):
        T, V, d = c["T"], c["V"], c["d"]
        s["tokens"] = _tokens(T, V, gen)
        s["scale"] = math.sqrt(d)
        shape = (d, V) if c["tied"] else (V, d)
        s["table"] = torch.randn(*shape, generator=gen, device="cuda", dtype=dt) * 0.02
        if c["op"] == "embed_step":
            s["dY"] = (1e-2 * randn(T, d)).to(dt)
    elif c["op"] in ("norm", "norm_step"):
        T, d, wt = c["T"], c["d"], _TYPES[c["weight"]]
        s["x"] = _activations(T, d, gen).to(dt)
        s["w"] = (1 + 0.2 * randn(d)).to(wt)
        s["b"] = (0.1 * randn(d)).to(wt) if c["bias"] else None
        s["eps"] = 1e-5
        if c["op"] == "norm_step":
            s["dY"] = (1e-2 * randn(T, d)).to(dt)
            s["leaves"] = [t for t in (s["x"], s["w"], s["b"]) if t is not None]
            s["leaves"] = [t.requires_grad_(True) for t in s["leaves"]]
    elif c["op"] == "rows":
        s["x"] = _activations(c["T"], c["d"], gen).to(dt)
    else:
        T, d, V = c["T"], c["d"], c["V"]
        # what rounding normal values to 127 steps of their row's largest leaves: a standard deviation of about 30
        s["x"] = (30 * randn(T, d)).round().clamp(-127, 127).to(torch.int8)
        s["w"] = (30 * torch.randn(V, d, generator=gen, device="cuda", dtype=torch.float16)).round().clamp(
            -127, 127).to(torch.int8)
        s["sx"], s["sw"] = 0.01 + 0.03 * rand(T), (0.5 + rand(V)) * (0.03 / math.sqrt(d))
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        return _own(s, c)
    with torch.no_grad():
        if c["op"] == "embed":
            return _plain_embed(s, c)
        if c["op"] == "embed_step":
            return dict(Y=_plain_embed(s, c), dE=_plain_embed_grad(s, c))
        if c["op"] == "norm":
            return _plain_norm(s)[0]
        if c["op"] == "norm_step":
            return _plain_norm_step(s, c)
        if c["op"] == "rows":
            q, scale = _plain_quantize(s["x"], c["kind"], c["group"])
            return dict(x=_plain_dequantize(q, scale, c["group"]).to(s["x"].dtype), scale=scale)
        return ((s["x"].float() @ s["w"].float().t()) * s["sx"][:, None] * s["sw"]).to(_TYPES[c["out"]])


def _own(s, c):
    import chunked_kl_loss_logit_amd as kd

    if c["op"] == "embed":
        return kd.embedding_forward(s["tokens"], s["table"], s["mask"], s["scale"], tied=c["tied"])
    if c["op"] == "embed_step":
        Y = kd.embedding_forward(s["tokens"], s["table"], s["mask"], s["scale"], tied=c["tied"])
        dE = kd.embedding_backward(s["dY"], s["tokens"], c["V"], s["mask"], s["scale"], tied=c["tied"],
                                   grad_dtype=_TYPES[c["grad"]])
        return dict(Y=Y, dE=dE)
    if c["op"] == "norm":
        return kd.layer_norm_forward(s["x"], s["w"], s["b"], s["mask"], s["eps"])[0]
    if c["op"] == "norm_step":
        y = kd.layer_norm(s["x"], s["w"], s["b"], s["mask"], s["eps"],
                          checkpoint=None if c["kind"] == "none" else c["kind"], group=c["group"])
        return dict(zip(("dx", "dw", "db"), torch.autograd.grad(y, s["leaves"], s["dY"])), y=y.detach())
    if c["op"] == "rows":
        q, scale = kd.quantize_rows(s["x"], c["kind"], c["group"])
        return dict(x=kd.dequantize_rows(q, scale, c["group"], s["x"].dtype), scale=scale)
    return kd.int8_matmul(s["x"], s["sx"], s["w"], s["sw"], _TYPES[c["out"]])


# ------------------------------------------------------------------ plain forms, 32 bits
def _plain_embed(s, c):
    at = s["tokens"].long()
    rows = s["table"].index_select(1, at).t() if c["tied"] else s["table"].index_select(0, at)
    Y = rows.float() * s["scale"]
    if s["mask"] is not None:
        Y = torch.where(s["mask"][:, None] != 0, Y, 0.0)
    return Y.to(s["table"].dtype)


def _plain_embed_grad(s, c):
    dY = s["dY"].float() * s["scale"]
    if s["mask"] is not None:
        dY = torch.where(s["mask"][:, None] != 0, dY, 0.0)
    at = s["tokens"].long()
    if c["tied"]:
        dE = torch.zeros(c["d"], c["V"], device="cuda").index_add_(1, at, dY.t())
    else:
        dE = torch.zeros(c["V"], c["d"], device="cuda").index_add_(0, at, dY)
    return dE.to(_TYPES[c["grad"]])


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = torch.rsqrt(((x - mean) ** 2).mean(1, keepdim=True) + s["eps"])
    y = (x - mean) * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["mask"] is not None:
        y = torch.where(s["mask"][:, None] != 0, y, 0.0)
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_step(s, c):
    y, mean, rstd = _plain_norm(s)
    x = s["x"].float()
    if c["kind"] != "none":
        x = _plain_dequantize(*_plain_quantize(s["x"], c["kind"], c["group"]), c["group"])
    dY = s["dY"].float()
    if s["mask"] is not None:
        dY = torch.where(s["mask"][:, None] != 0, dY, 0.0)
    xh = (x - mean) * rstd
    g = dY * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    got = dict(y=y, dx=dx.to(s["x"].dtype), dw=(dY * xh).sum(0).to(s["w"].dtype))
    if s["b"] is not None:
        got["db"] = dY.sum(0).to(s["w"].dtype)
    return got


def _groups(x, group):
    """x [T, d] as [T, n, group], zeros behind the row's end."""
    d = x.shape[1]
    group = group or d
    n = -(-d // group)
    return torch.nn.functional.pad(x, (0, n * group - d)).reshape(x.shape[0], n, group)


def _plain_quantize(x, kind, group):
    """The values (in units of their scale) that 8 bits hold of x, and the groups' scales."""
    d = x.shape[1]
    xg = _groups(x.float(), group)
    top = 127.0 if kind == "int8" else 448.0
    # 64 bits: torch divides by a number in 32 bits by its rounded reciprocal, and a quotient next to the middle of two
    # steps goes to the nearer one
    scale = (xg.abs().amax(2).double() / top).float()
    r = torch.where(scale[..., None] > 0, xg.double() / scale[..., None].double(), 0.0)
    if kind == "int8":
        q = torch.round(r)
    else:
        step = torch.exp2(torch.frexp(r)[1].clamp(min=-5).double() - 4)  # 4 significant bits, 2^-9 at least
        q = torch.round(r / step) * step
    return q.clamp(-top, top).float().reshape(x.shape[0], -1)[:, :d], scale


def _plain_dequantize(q, scale, group):
    d = q.shape[1]
    return (_groups(q, group) * scale[..., None]).reshape(q.shape[0], -1)[:, :d]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c.get("dtype") in ("bf16", "f16") else 4
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] in ("embed", "embed_step"):
        n = c["T"] * c["d"]
        b = 2 * n * e + 4 * c["T"]
        if c["op"] == "embed_step":
            b += n * e + c["V"] * c["d"] * size[c["grad"]]
        return dict(bytes=b, flops=n * (1 if c["op"] == "embed" else 3))
    if c["op"] in ("norm", "norm_step"):
        n, p = c["T"] * c["d"], c["d"] * size[c["weight"]] * (2 if c["bias"] else 1)
        if c["op"] == "norm":
            return dict(bytes=2 * n * e + p, flops=7 * n)
        kept = 0 if c["kind"] == "none" else n  # written in 8 bits, and read instead of the input
        return dict(bytes=(4 if kept else 5) * n * e + 2 * kept + 3 * p, flops=25 * n)
    if c["op"] == "rows":
        n = c["T"] * c["d"]
        groups = c["T"] * -(-c["d"] // (c["group"] or c["d"]))
        return dict(bytes=2 * n * e + 2 * n + 8 * groups, flops=6 * n)
    T, d, V = c["T"], c["d"], c["V"]
    return dict(bytes=T * d + V * d + T * V * size[c["out"]] + 4 * (T + V), flops=2 * T * d * V)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    def e4m3_values():
        """The 127 values >= 0 of the format in ascending order: the index's lowest bit is the significand's."""
        values = [m * 2.0 ** -9 for m in range(8)]
        values += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
        return torch.tensor(values[:127], device="cuda", dtype=torch.float64)

    def exact_rows(x, kind, group):
        """The values that 8 bits hold of x in 64 bits, and the scales, which are float32 by definition."""
        d, top = x.shape[1], 127 if kind == "int8" else 448
        out, scales = torch.empty(x.shape, device="cuda", dtype=torch.float64), []
        for a in range(0, d, group or d):
            part = x[:, a:a + (group or d)].double()
            scale = (part.abs().amax(1, keepdim=True) / top).float().double()
            r = part / scale
            if kind == "int8":
                tie = r - torch.floor(r) == 0.5
                even = 2 * torch.floor(torch.floor(r) / 2 + 0.5)
                q = torch.where(tie, even, torch.floor(r + 0.5))
            else:
                grid = e4m3_values()
                mag = r.abs().clamp(max=448.0).contiguous()
                hi = torch.searchsorted(grid, mag).clamp(max=grid.numel() - 1)
                lo = (hi - 1).clamp(min=0)
                up, down = grid[hi] - mag, mag - grid[lo]
                pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
                q = torch.where(r < 0, -grid[pick], grid[pick])
            out[:, a:a + (group or d)] = q.clamp(-top, top) * scale
            scales.append(scale[:, 0])
        return out, torch.stack(scales, 1)

    s, c = prepare(case, seed), case
    keep = None if s["mask"] is None else (s["mask"] == 0).nonzero()[:, 0]
    with torch.no_grad():
        if c["op"] in ("embed", "embed_step"):
            at = s["tokens"].long()
            Y = (s["table"][:, at].double().t() if c["tied"] else s["table"][at].double()) * s["scale"]
            if keep is not None:
                Y[keep] = 0
            if c["op"] == "embed":
                return Y
            live = torch.arange(c["T"], device="cuda") if keep is None else s["mask"].nonzero()[:, 0]
            dE = torch.zeros(c["V"], c["d"], device="cuda", dtype=torch.float64)
            dE.index_put_((at[live],), s["dY"][live].double() * s["scale"], accumulate=True)
            return dict(Y=Y, dE=dE.t() if c["tied"] else dE)
        if c["op"] == "rows":
            x, scale = exact_rows(s["x"], c["kind"], c["group"])
            return dict(x=x, scale=scale)
        if c["op"] == "int8":
            return (s["x"].double() * s["sx"].double()[:, None]) @ (s["w"].double() * s["sw"].double()[:, None]).t()
        x, w = s["x"].double(), s["w"].double()
        b = 0.0 if s["b"] is None else s["b"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        sd = (var + s["eps"]).sqrt()
        y = (x - mean) / sd * w + b
        if keep is not None:
            y[keep] = 0
        if c["op"] == "norm":
            return y
        if c["kind"] != "none":
            x = exact_rows(s["x"], c["kind"], c["group"])[0]
        dY = s["dY"].double()
        if keep is not None:
            dY[keep] = 0
        z, g = (x - mean) / sd, dY * w
        dx = (c["d"] * g - g.sum(1, keepdim=True) - z * (g * z).sum(1, keepdim=True)) / (c["d"] * sd)
        got = dict(y=y, dx=dx, dw=torch.einsum("td,td->d", dY, z))
        if s["b"] is not None:
            got["db"] = dY.sum(0)
        return got

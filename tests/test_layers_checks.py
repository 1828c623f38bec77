"""The Python layer of the operators of kdlayers.h refuses wrong shapes, types, devices and options before it takes a
pointer.  On the CPU a call whose arguments pass stops at the "must be on the GPU" test."""
import pytest
import torch

kd = pytest.importorskip("chunked_kl_loss_logit_amd")
B = kd._layers_binding
T, D, V = 6, 48, 40
bf, f16, f32, f64, i32, i8, u8 = (torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int32, torch.int8,
                                  torch.uint8)
f8 = torch.float8_e4m3fn


def z(*shape, dtype=f32):
    return torch.zeros(*shape, dtype=dtype)


def gpu_only(fn):
    with pytest.raises(ValueError, match="on the GPU"):
        fn()


def refused(fn, err, match):
    with pytest.raises(err, match=match):
        fn()


def table(fn, base, cases):
    for over, err, match in cases:
        refused(lambda: fn(**{**base, **over}), err, match)


def test_embedding_fwd():
    a = dict(tokens=z(T, dtype=i32), table=z(V, D, dtype=bf), mask=z(T, dtype=u8), scale=1.0, tied=False,
             out=z(T, D, dtype=bf))
    gpu_only(lambda: B.kd_embedding_fwd(**a))
    gpu_only(lambda: B.kd_embedding_fwd(**{**a, "table": z(D, V, dtype=bf), "tied": True, "mask": None}))
    table(B.kd_embedding_fwd, a, [
        (dict(tokens=z(T, dtype=torch.int64)), TypeError, r"tokens must be torch.int32.*\.int\(\)"),
        (dict(tokens=z(T, 1, dtype=i32)), ValueError, "tokens must be 1-D"),
        (dict(tokens=None), ValueError, "tokens is required"),
        (dict(table=z(V, D, dtype=f64)), TypeError, "table must be"),
        (dict(table=z(V * D, dtype=bf)), ValueError, "table must be 2-D"),
        (dict(mask=z(T)), TypeError, "mask must be"),
        (dict(mask=z(T + 1, dtype=u8)), ValueError, "mask must have shape"),
        (dict(out=z(T, D)), TypeError, "out must be torch.bfloat16"),
        (dict(out=z(T, V, dtype=bf)), ValueError, "out must have shape"),
        (dict(tied=True), ValueError, "out must have shape"),
    ])
    for fn in (kd.embedding_forward, kd.embedding):
        gpu_only(lambda: fn(z(T, dtype=i32), z(V, D)))
        refused(lambda: fn(z(T, dtype=i32), z(V)), ValueError, "table must be 2-D")


def test_embedding_bwd():
    a = dict(grad=z(T, D, dtype=bf), tokens=z(T, dtype=i32), mask=None, scale=1.0, V=V, tied=False, accumulate=False,
             grad_table=z(V, D), workspace=z(64, dtype=u8))
    gpu_only(lambda: B.kd_embedding_bwd(**a))
    table(B.kd_embedding_bwd, a, [
        (dict(grad=z(T + 1, D, dtype=bf)), ValueError, "grad must have 6 rows"),
        (dict(grad=z(T, D, dtype=i32)), TypeError, "grad must be"),
        (dict(grad_table=z(D, V)), ValueError, "grad_table must have shape"),
        (dict(grad_table=z(V, D, dtype=f64)), TypeError, "grad_table must be"),
        (dict(V=V + 1), ValueError, "grad_table must have shape"),
    ])
    refused(lambda: kd.embedding_backward(z(T, D), z(T, dtype=i32), V, out=z(V, D), grad_dtype=bf), TypeError, "out must be")
    p = torch.nn.Parameter(z(V, D))
    refused(lambda: kd.embedding_backward(z(T, D), z(T, dtype=i32), V, out=p), ValueError, "must not require a gradient")


def test_rows():
    a = dict(x=z(T, D), kind="int8", group=32, q=z(T, D, dtype=i8), scale=z(T, 2))
    gpu_only(lambda: B.kd_rows_quantize(**a))
    gpu_only(lambda: B.kd_rows_quantize(z(T, D), "e4m3", 0, z(T, D, dtype=f8), z(T, 1)))
    table(B.kd_rows_quantize, a, [
        (dict(kind="int4"), ValueError, "kind must be one of"),
        (dict(group=48), ValueError, "group must be one of"),
        (dict(q=z(T, D, dtype=f8)), TypeError, "q must be torch.int8"),
        (dict(q=z(T, D + 1, dtype=i8)), ValueError, "q must have 48 columns"),
        (dict(scale=z(T, 1)), ValueError, "scale must have shape"),
        (dict(scale=z(T, 2, dtype=bf)), TypeError, "scale must be"),
        (dict(x=z(T)), ValueError, "x must be 2-D"),
    ])
    gpu_only(lambda: kd.dequantize_rows(z(T, D, dtype=i8), z(T, 2), 32, f16))
    table(kd.dequantize_rows, dict(q=z(T, D, dtype=f8), scale=z(T, 1), group=0, dtype=f32), [
        (dict(q=z(T, D, dtype=u8)), TypeError, "q must be"),
        (dict(group=64, scale=z(T, 2)), ValueError, "scale must have shape"),
        (dict(dtype=f64), TypeError, "out must be"),
    ])
    refused(lambda: kd.checkpoint_8bit(abs, 3.0), TypeError, "x must be a tensor")
    refused(lambda: kd.checkpoint_8bit(abs, z(3, dtype=i32)), TypeError, "x must be one of")
    refused(lambda: kd.checkpoint_8bit(abs, z(3), group=31), ValueError, "group must be one of")


def test_checkpointed_functions():
    x, w = z(3, 8).requires_grad_(True), z(3, 8)
    refused(lambda: kd.checkpoint_8bit(lambda x: x.add_(1), x * 2), RuntimeError, "in place")
    refused(lambda: kd.checkpoint_8bit(lambda x, w: x * w.add_(1), x, w), RuntimeError, "in place")
    refused(lambda: kd.checkpoint_8bit(lambda x: {"y": x * 2}, x), TypeError, "got a dict")
    refused(lambda: kd.checkpoint_8bit(lambda x: (x * 2, [x * 3]), x), TypeError, "got a list")


def test_layer_norm():
    a = dict(x=z(T, D, dtype=bf), weight=z(D), bias=z(D), mask=z(T, dtype=torch.bool), eps=1e-5, y=z(T, D, dtype=bf),
             mean=z(T), rstd=z(T))
    gpu_only(lambda: B.kd_layer_norm_fwd(**a))
    gpu_only(lambda: B.kd_layer_norm_fwd(**{**a, "kind": "int8", "group": 32, "q": z(T, D, dtype=i8), "scale": z(T, 2)}))
    table(B.kd_layer_norm_fwd, a, [
        (dict(weight=z(D, dtype=f16)), TypeError, "weight must be"),
        (dict(weight=z(D, dtype=bf)), TypeError, "weight and bias must have one type"),
        (dict(bias=z(D + 1)), ValueError, "bias must have shape"),
        (dict(y=z(T, D)), TypeError, "y must be"),
        (dict(mean=z(T + 1)), ValueError, "mean must have shape"),
        (dict(kind="int8"), ValueError, "q is required"),
        (dict(q=z(T, D, dtype=i8)), ValueError, "q and scale need a kind"),
        (dict(kind="e4m3", group=32, q=z(T, D, dtype=i8), scale=z(T, 2)), TypeError, "q must be torch.float8_e4m3fn"),
    ])
    for fn in (kd.layer_norm, kd.layer_norm_forward):
        gpu_only(lambda: fn(z(T, D)))
        refused(lambda: fn(z(T, D), checkpoint="int4"), ValueError, "kind must be one of") if fn is not kd.layer_norm \
            else refused(lambda: fn(z(T, D).requires_grad_(True), checkpoint="int4"), ValueError, "kind must be one of")
    refused(lambda: kd.layer_norm(z(T, D), checkpoint="int4"), ValueError, "kind must be one of")  # also without gradients
    refused(lambda: kd.layer_norm(z(T, D), checkpoint="int8", group=31), ValueError, "group must be one of")


def test_layer_norm_bwd():
    a = dict(grad=z(T, D, dtype=bf), x=z(T, D, dtype=bf), weight=z(D), mask=None, mean=z(T), rstd=z(T),
             dx=z(T, D, dtype=bf), dweight=z(D), dbias=z(D), workspace=z(64, dtype=u8))
    gpu_only(lambda: B.kd_layer_norm_bwd(**a))
    kept = dict(x=None, group=32, q=z(T, D, dtype=f8), scale=z(T, 2))
    gpu_only(lambda: B.kd_layer_norm_bwd(**{**a, **kept}))
    table(B.kd_layer_norm_bwd, a, [
        (dict(x=z(T, D)), TypeError, "x must be"),
        (dict(x=None), ValueError, "x is required"),
        ({**kept, "x": a["x"]}, ValueError, "x must be None"),
        ({**kept, "scale": z(T, 1)}, ValueError, "scale must have shape"),
        (dict(scale=z(T, 1)), ValueError, "scale needs q"),
        (dict(dweight=z(D, dtype=bf)), TypeError, "dweight must be"),
        (dict(weight=None, dweight=z(D, dtype=bf)), TypeError, "dweight and dbias must have one type"),
        (dict(dx=None, dweight=None, dbias=None), ValueError, "all None"),
        (dict(rstd=z(T, dtype=bf)), TypeError, "rstd must be"),
    ])


def test_int8_matmul():
    a = dict(x=z(T, D, dtype=i8), x_scale=z(T), w=z(V, D, dtype=i8), w_scale=z(V, 1), out=z(T, V), workspace=None)
    gpu_only(lambda: B.kd_int8_matmul(**a))
    table(B.kd_int8_matmul, a, [
        (dict(x=z(T, D, dtype=u8)), TypeError, "x must be torch.int8"),
        (dict(w=z(V, D + 16, dtype=i8)), ValueError, "w must have 48 columns"),
        (dict(w=z(V, D)), TypeError, "w must be"),
        (dict(x_scale=z(T + 1)), ValueError, "x_scale must have shape"),
        (dict(w_scale=z(1, V)), ValueError, "w_scale must have shape"),
        (dict(out=z(V, T)), ValueError, "out must have shape"),
        (dict(out=z(T, V, dtype=f64)), TypeError, "out must be"),
    ])
    gpu_only(lambda: kd.int8_matmul(a["x"], a["x_scale"], a["w"], a["w_scale"]))
    refused(lambda: kd.int8_matmul(z(T, 40, dtype=i8), z(T), z(V, 40, dtype=i8), z(V)), kd.KDError, "multiple of 16")


def test_layer_norm_keeps_its_input_only_for_a_backward_pass(monkeypatch):
    """The copy in 8 bits is a third of the forward's traffic."""
    asked = []

    def forward(x, weight, bias, mask, eps, checkpoint, group):
        asked.append(checkpoint)
        return x * 1, z(T), z(T), None if checkpoint is None else (x.to(i8), z(T, 1))

    monkeypatch.setattr(kd.layers, "layer_norm_forward", forward)
    x, w = z(T, D), z(D)
    for grad, leaf, want in ((True, w, "int8"), (False, w, None), (True, x, "int8"), (False, x, None), (True, None, None)):
        for t in (x, w):
            t.requires_grad_(t is leaf)
        with torch.set_grad_enabled(grad):
            y = kd.layer_norm(x, w, checkpoint="int8")
        assert asked.pop() == want and y.requires_grad == (want is not None)
    with torch.inference_mode():
        kd.layer_norm(x, w.requires_grad_(True), checkpoint="int8")
    assert asked == [None]

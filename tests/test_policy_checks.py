"""The Python layer of the policy- and preference-training operators refuses wrong shapes, types, devices and options
before it takes a pointer.  On the CPU a call whose arguments pass stops at the "must be on the GPU" test."""
import pytest
import torch

kd = pytest.importorskip("chunked_kl_loss_logit_amd")
B = kd._policy_binding
T, D, V, S = 6, 16, 40, 3
bf, f32, f64, i32, u8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


def z(*shape, dtype=f32):
    return torch.zeros(*shape, dtype=dtype)


def gpu_only(fn):
    with pytest.raises(ValueError, match="on the GPU"):
        fn()


def refused(fn, err, match):
    with pytest.raises(err, match=match):
        fn()


def head(**over):
    a = dict(H=z(T, D, dtype=bf), W=z(D, V, dtype=bf), tokens=z(T, dtype=i32), mask=z(T, dtype=u8), tau=1.0, logp=z(T),
             lse=z(T), entropy=z(T), logits=z(T, 256), workspace=z(64, dtype=u8))
    a.update(over)
    return a


HEAD = [
    (dict(H=z(T, D, dtype=torch.float16)), TypeError, "H must be"),
    (dict(H=z(T * D, dtype=bf)), ValueError, "H must be 2-D"),
    (dict(W=z(D, V)), TypeError, "W must be torch.bfloat16"),
    (dict(W=z(D + 8, V, dtype=bf)), ValueError, "W must have 16 rows"),
    (dict(tokens=z(T, dtype=torch.int64)), TypeError, r"tokens must be torch.int32.*\.int\(\)"),
    (dict(tokens=z(T + 1, dtype=i32)), ValueError, "tokens must have shape"),
    (dict(tokens=None), ValueError, "tokens is required"),
    (dict(mask=z(T)), TypeError, "mask must be"),
    (dict(mask=z(T - 1, dtype=u8)), ValueError, "mask must have shape"),
    (dict(lse=z(T, dtype=f64)), TypeError, "lse must be"),
    (dict(entropy=z(T + 1)), ValueError, "entropy must have shape"),
    (dict(logits=z(T, V)), ValueError, "logits must have shape"),
]


def test_token_logp_fwd():
    gpu_only(lambda: B.kd_token_logp_fwd(**head()))
    gpu_only(lambda: B.kd_token_logp_fwd(**head(mask=None, entropy=None, logits=None)))
    gpu_only(lambda: B.kd_token_logp_fwd(**head(H=z(T, D), W=z(D, V), mask=z(T, dtype=torch.bool))))
    for over, err, match in HEAD + [(dict(logp=z(T + 1)), ValueError, "logp must have shape")]:
        refused(lambda: B.kd_token_logp_fwd(**head(**over)), err, match)


def test_token_logp_bwd():
    def args(**over):
        a = head(grad_logp=z(T), grad_entropy=z(T), dH=z(T, D, dtype=bf), dW=z(D, V), chunk_rows=0)
        del a["logp"]
        a.update(over)
        return a

    gpu_only(lambda: B.kd_token_logp_bwd(**args()))
    gpu_only(lambda: B.kd_token_logp_bwd(**args(dW=z(D, V, dtype=bf), grad_entropy=None)))
    for over, err, match in HEAD + [
        (dict(grad_logp=z(T, dtype=bf)), TypeError, "grad_logp must be"),
        (dict(grad_entropy=z(T, 1)), ValueError, "grad_entropy must have shape"),
        (dict(dH=z(T, D)), TypeError, "dH must be"),
        (dict(dW=z(V, D)), ValueError, "dW must have shape"),
        (dict(dW=z(D, V, dtype=torch.float16)), TypeError, "dW must be"),
        (dict(lse=None), ValueError, "lse is required"),
    ]:
        refused(lambda: B.kd_token_logp_bwd(**args(**over)), err, match)


def test_shards():
    refused(lambda: B.kd_token_logp_shard_combine(z(T, 4), None, 1.0, z(T), z(T), None), ValueError, "rec must be")
    refused(lambda: B.kd_token_logp_shard_combine(z(2, T, 8), None, 1.0, z(T), z(T), None), ValueError, "rec must be")
    refused(lambda: B.kd_token_logp_shard_combine(z(2, T, 4), None, 1.0, z(T - 1), z(T), None), ValueError, "logp must")
    gpu_only(lambda: B.kd_token_logp_shard_combine(z(2, T, 4), None, 1.0, z(T), z(T), z(T)))


def policy(logp=None, **kw):
    a = dict(old_logp=z(T), advantages=z(T), mask=z(T, dtype=u8))
    a.update(kw)
    return B.PolicyOptions(z(T) if logp is None else logp, **a)


def test_policy_loss():
    cu = z(S + 1, dtype=i32)
    gpu_only(lambda: policy())
    gpu_only(lambda: policy(cu_seqlens=cu, advantages=z(S), reduction="sequence", mask=None))
    gpu_only(lambda: policy(cu_seqlens=z(T + 1, dtype=i32), per_sequence=True))
    for kw, err, match in [
        (dict(logp=z(T, 1)), ValueError, "logp must be 1-D"),
        (dict(logp=z(T, dtype=bf)), TypeError, "logp must be"),
        (dict(old_logp=z(T + 1)), ValueError, "old_logp must have shape"),
        (dict(old_logp=None), ValueError, "old_logp is required"),
        (dict(advantages=z(S)), ValueError, "advantages must have shape"),
        (dict(advantages=z(S), per_sequence=True), ValueError, "per_sequence needs cu_seqlens"),
        (dict(advantages=z(S + 1), cu_seqlens=cu), ValueError, "advantages must have shape"),
        (dict(cu_seqlens=z(T + 1, dtype=i32)), ValueError, "per_sequence must be given"),
        (dict(cu_seqlens=z(S + 1)), TypeError, "cu_seqlens must be"),
        (dict(cu_seqlens=z(1, dtype=i32)), ValueError, "at least two"),
        (dict(ref_logp=z(S)), ValueError, "ref_logp must have shape"),
        (dict(entropy=z(T, dtype=f64)), TypeError, "entropy must be"),
        (dict(mask=z(T)), TypeError, "mask must be"),
    ]:
        refused(lambda: policy(**kw), err, match)
    refused(lambda: kd.policy_loss(z(T), z(T), z(T), reduction="mean"), ValueError, "on the GPU|reduction")
    refused(lambda: kd.policy_loss(z(T), z(T), z(T), nonsense=1), TypeError, "nonsense")


def test_preference_loss():
    cu = z(5, dtype=i32)
    gpu_only(lambda: kd.preference_loss(z(T), cu))
    for a, kw, err, match in [
        ((z(T, 1), cu), {}, ValueError, "logp must be 1-D"),
        ((z(T, dtype=bf), cu), {}, TypeError, "logp must be"),
        ((z(T), z(4, dtype=i32)), {}, ValueError, "even number"),
        ((z(T), z(5)), {}, TypeError, "cu_seqlens must be"),
        ((z(T), z(5, 1, dtype=i32)), {}, ValueError, "at least two"),
        ((z(T), cu, z(T + 1, dtype=u8)), {}, ValueError, "mask must have shape"),
        ((z(T), cu), dict(ref_logp=z(T + 1)), ValueError, "ref_logp must have shape"),
    ]:
        refused(lambda: kd.preference_loss(*a, **kw), err, match)


def test_clipping():
    gpu_only(lambda: kd.clip_grad_norm([z(3)], 1.0))
    refused(lambda: kd.clip_grad_norm([], 1.0), ValueError, "no tensors")
    refused(lambda: kd.clip_grad_norm([None], 1.0), ValueError, "no tensors")
    refused(lambda: kd.clip_grad_norm([z(3, dtype=f64)], 1.0), TypeError, "float32, bfloat16 or float16")
    refused(lambda: kd.clip_grad_norm([1.0], 1.0), TypeError, "torch.Tensors")


@pytest.mark.parametrize("t,dense", [
    (torch.zeros(4, 5), True), (torch.zeros(4, 5).t(), True), (torch.zeros(2, 3, 4).permute(2, 0, 1), True),
    (torch.zeros(4, 6)[:, :5], False), (torch.zeros(4, 6)[:, ::2], False), (torch.zeros(4, 1).expand(4, 3), False),
    (torch.zeros(()), True), (torch.zeros(0, 5), True), (torch.zeros(1, 7, 1), True), (torch.zeros(4, 6)[1:2, :3], True),
])
def test_dense(t, dense):
    assert B._dense(t) == dense

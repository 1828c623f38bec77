"""The C ABI of kdpolicy.h on the CPU: what the header declares is exported, workspaces are sized as documented, and
bad arguments are refused on the host before any HIP call."""
import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
kd = pytest.importorskip("chunked_kl_loss_logit_amd")
B = kd._policy_binding
vp = ctypes.c_void_p
F = 0x10000  # aligned to 256, never dereferenced: the calls fail before any HIP call


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kd.LIB_PATH):
        pytest.fail("libkdloss.so is not built (run __graft_entry__.build())")
    return B.plib()


def test_exports_every_declared_symbol(L):
    text = open(os.path.join(ROOT, "include", "kdpolicy.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(kd_[a-z0-9_]+)\s*\(", text)))
    assert sorted(kd.POLICY_EXPORTS) == names
    assert all(hasattr(L, n) for n in names)


def err():
    return kd.lib().kd_last_error().decode()


def size(L, fn, *args):
    out = ctypes.c_size_t()
    st = getattr(L, fn)(*args, ctypes.byref(out))
    return st, out.value


def test_sizes(L):
    assert size(L, "kd_token_logp_logits_size", 10, 264) == (0, 10 * 512 * 4)
    assert size(L, "kd_token_logp_workspace_size", 0, 128, 264, 1, 1, 0) == (0, 0)
    a = [size(L, "kd_token_logp_workspace_size", T, 2048, 128256, 1, 0, 0)[1] for T in (16384, 65536, 262144)]
    assert 0 < (a[2] - a[1]) / 196608 <= 16  # per token: the list of valid rows
    # a bf16 dW that adds up over chunks does so in float32
    f, b = (size(L, "kd_token_logp_workspace_size", 8192, 2048, 128256, 1, w, 0)[1] for w in (0, 1))
    assert b - f >= 2048 * 128256 * 4
    assert size(L, "kd_token_logp_workspace_size", 8, 128, 264, 0, 1, 0)[0] == 2
    assert size(L, "kd_token_logp_workspace_size", 8, 128, 264, 1, 7, 0)[0] == 1
    assert size(L, "kd_token_logp_workspace_size", 8, 128, 264, 1, 1, -1)[0] == 1
    assert size(L, "kd_policy_loss_workspace_size", 0, 0)[0] == 0
    assert size(L, "kd_policy_loss_workspace_size", -1, 0)[0] == 1
    assert size(L, "kd_policy_loss_workspace_size", 1 << 31, 0)[0] == 2
    assert size(L, "kd_preference_loss_workspace_size", 100, 0)[0] == 1
    assert size(L, "kd_preference_loss_workspace_size", 100, 3)[0] == 0
    n = (ctypes.c_int64 * 3)(5, 0, 100000)
    assert size(L, "kd_grad_norm_workspace_size", n, 3)[0] == 0
    assert size(L, "kd_grad_norm_workspace_size", (ctypes.c_int64 * 1)(-1), 1)[0] == 1
    assert size(L, "kd_grad_norm_workspace_size", (ctypes.c_int64 * 1)(1 << 50), 1)[0] == 2
    assert size(L, "kd_grad_norm_workspace_size", None, 0)[0] == 0


def logp_fwd(L, H=F, W=F, tok=F, tau=1.0, T=8, d=64, V=256, dt=1, logp=F, lse=F, ent=F, z=F, ws=F, wsb=0):
    return L.kd_token_logp_fwd(vp(H), vp(W), vp(tok), None, tau, T, d, V, dt, vp(logp), vp(lse), vp(ent), vp(z), vp(ws),
                               wsb, None)


def logp_bwd(L, H=F, W=F, tok=F, tau=1.0, T=8, d=64, V=256, dt=1, lse=F, ent=F, z=F, g=F, ge=F, dH=F, dW=F, dw=0,
             chunk=0, ws=F, wsb=0):
    return L.kd_token_logp_bwd(vp(H), vp(W), vp(tok), None, tau, T, d, V, dt, vp(lse), vp(ent), vp(z), vp(g), vp(ge),
                               vp(dH), vp(dW), dw, chunk, vp(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(H=0), 1), (dict(W=0), 1), (dict(tok=0), 1), (dict(logp=0), 1), (dict(lse=0), 1),
    (dict(ent=0), 4), (dict(z=0), 4), (dict(tau=0.0), 1), (dict(tau=math.nan), 1), (dict(T=-1), 1), (dict(d=60), 2),
    (dict(V=260), 2), (dict(V=1 << 25), 2), (dict(d=1 << 25), 2), (dict(dt=2), 1), (dict(T=1 << 31), 2), (dict(H=F + 8), 3), (dict(W=F + 2), 3), (dict(tok=F + 1), 3),
    (dict(z=F + 4), 3), (dict(ent=F + 1), 3), (dict(ws=0), 1), (dict(ws=F + 16, wsb=1 << 40), 3), (dict(T=0, H=0), 0),
])
def test_token_logp_fwd_refuses(L, kw, code):
    assert logp_fwd(L, **kw) == code
    assert code == 0 or err()


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(lse=0), 1), (dict(g=0, ge=0), 1), (dict(g=0), 4), (dict(ge=0, ent=0), 4), (dict(ent=0), 1),
    (dict(dH=0, dW=0), 1), (dict(dH=0), 4), (dict(dW=0), 4), (dict(dW=F + 8), 3), (dict(dH=F + 8), 3), (dict(dw=1), 4), (dict(dw=2), 1),
    (dict(dt=0, dw=1), 2), (dict(chunk=-1), 1), (dict(z=F + 8), 3), (dict(g=F + 2), 3), (dict(V=0), 1),
])
def test_token_logp_bwd_refuses(L, kw, code):
    assert logp_bwd(L, **kw) == code
    assert err()


def test_shard_calls_refuse(L):
    def fwd(v0=0, V=256, rec=F):
        return L.kd_token_logp_fwd_shard(vp(F), vp(F), vp(F), None, 1.0, 8, 64, V, v0, 1, vp(rec), None, vp(F), 0, None)

    assert [fwd(), fwd(v0=-1), fwd(v0=1 << 30), fwd(rec=0), fwd(rec=F + 4)] == [4, 1, 2, 1, 3]

    def comb(R=2, T=8, tau=1.0, rec=F, logp=F):
        return L.kd_token_logp_shard_combine(vp(rec), R, None, tau, T, vp(logp), vp(F), None, None)

    assert [comb(R=0), comb(T=-1), comb(tau=math.inf), comb(R=1 << 30), comb(rec=0), comb(rec=F + 8), comb(logp=0)] == \
        [1, 1, 1, 2, 1, 3, 1]
    assert comb(T=0, rec=0) == 0


def policy(L, T=100, logp=F, old=F, adv=F, stats=F, weights=F, ws=F, wsb=0, fn="fwd", **o):
    d = dict(ref_logp=0, entropy=0, cu_seqlens=0, S=0, per_sequence=0, reduction=1, kl_kind=3, clip_low=0.2,
             clip_high=0.2, dual_clip=0.0, kl_weight=0.0, entropy_weight=0.0)
    d.update(o)
    opts = B.KdPolicyOpts(*[d[k] for k, _ in B.KdPolicyOpts._fields_])
    if fn == "fwd":
        return L.kd_policy_loss_fwd(vp(logp), vp(old), vp(adv), None, opts, T, None, vp(stats), vp(weights), vp(ws), wsb,
                                    None)
    if fn == "bwd":
        return L.kd_policy_loss_bwd(vp(logp), vp(old), vp(adv), None, opts, T, vp(weights), vp(stats), vp(0), None, None)
    return L.kd_policy_loss_fwd_bwd(vp(logp), vp(old), vp(adv), None, opts, T, vp(stats), vp(weights), vp(0), None,
                                    vp(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(T=-1), 1), (dict(T=1 << 31), 2), (dict(logp=0), 1), (dict(old=0), 1), (dict(adv=0), 1),
    (dict(stats=0), 1), (dict(weights=0), 1), (dict(weights=F + 4), 3), (dict(logp=F + 2), 3),
    (dict(reduction=2), 1), (dict(reduction=3), 1), (dict(reduction=2, cu_seqlens=F, S=4), 4), (dict(cu_seqlens=F), 1),
    (dict(per_sequence=1), 1), (dict(S=-1), 1), (dict(kl_kind=0), 1), (dict(kl_kind=4), 1), (dict(clip_low=-0.1), 1),
    (dict(clip_low=1.1), 1), (dict(clip_low=math.nan), 1), (dict(clip_high=-1.0), 1), (dict(clip_high=math.inf), 4),
    (dict(dual_clip=1.0), 1), (dict(dual_clip=-2.0), 1), (dict(dual_clip=math.inf), 1), (dict(dual_clip=2.0), 4),
    (dict(kl_weight=0.1), 1), (dict(kl_weight=0.1, ref_logp=F), 4), (dict(kl_weight=math.nan, ref_logp=F), 1),
    (dict(entropy_weight=0.1), 1), (dict(entropy_weight=0.1, entropy=F), 4), (dict(entropy=F + 1), 3),
    (dict(ws=0), 1), (dict(fn="bwd"), 1), (dict(fn="bwd", T=0), 0), (dict(fn="fwd_bwd"), 1),
])
def test_policy_loss_refuses(L, kw, code):
    assert policy(L, **kw) == code
    assert code == 0 or err()


def pref(L, T=100, P=3, logp=F, cu=F, loss=F, rewards=F, sums=F, ws=F, wsb=0, **o):
    d = dict(ref_logp=0, kind=0, average=0, beta=0.1, label_smoothing=0.0, margin=0.0)
    d.update(o)
    opts = B.KdPrefOpts(*[d[k] for k, _ in B.KdPrefOpts._fields_])
    return L.kd_preference_loss_fwd(vp(logp), vp(cu), None, opts, T, P, vp(loss), vp(rewards), vp(sums), vp(ws), wsb,
                                    None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(P=0), 1), (dict(P=-1), 1), (dict(P=1 << 30), 2), (dict(T=-1), 1), (dict(cu=0), 1),
    (dict(cu=F + 2), 3), (dict(logp=0), 1), (dict(loss=0), 1), (dict(rewards=0), 1), (dict(sums=0), 1),
    (dict(sums=F + 4), 3), (dict(kind=3), 1), (dict(beta=0.0), 1), (dict(beta=math.inf), 1), (dict(beta=math.nan), 1),
    (dict(label_smoothing=0.5), 1), (dict(label_smoothing=-0.1), 1), (dict(label_smoothing=0.1, kind=1), 2),
    (dict(label_smoothing=0.1), 4), (dict(margin=math.nan), 1), (dict(margin=1.0, kind=2), 2), (dict(margin=1.0), 4),
])
def test_preference_loss_refuses(L, kw, code):
    assert pref(L, **kw) == code
    assert err()


def test_null_options_are_refused(L):
    assert L.kd_policy_loss_fwd(vp(F), vp(F), vp(F), None, None, 10, None, vp(F), vp(F), vp(F), 1 << 30, None) == 1
    assert L.kd_preference_loss_fwd(vp(F), vp(F), None, None, 10, 1, vp(F), vp(F), vp(F), vp(F), 1 << 30, None) == 1


def clip(L, ptrs, numel, types, outs=None, otypes=None, max_norm=1.0, sumsq=F, norm=F):
    n = len(ptrs)
    return L.kd_grad_clip((vp * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types), n,
                          (vp * n)(*(outs or ptrs)), (ctypes.c_int32 * n)(*(otypes or types)), vp(sumsq), max_norm,
                          vp(norm), None)


def test_grad_calls_refuse(L):
    A, C = F, F + 4096
    # every check but the last argument's: sumsq = NULL ends the calls that would be fine
    fine = dict(sumsq=0)
    assert clip(L, [A, C], [8, 8], [0, 1], **fine) == 1 and "sumsq" in err()
    assert clip(L, [A, C], [8, 8], [0, 3], **fine) == 1 and "type" in err()
    assert clip(L, [A, 0], [8, 8], [0, 1], **fine) == 1 and "NULL" in err()
    assert clip(L, [A, 0], [8, 0], [0, 1], **fine) == 1 and "sumsq" in err()
    assert clip(L, [A + 2, C], [8, 8], [0, 1], **fine) == 3
    assert clip(L, [A, C + 2], [8, 8], [0, 1], **fine) == 1 and "sumsq" in err()
    assert clip(L, [A], [8], [0], max_norm=-1.0, **fine) == 1 and "max_norm" in err()
    assert clip(L, [A], [8], [0], max_norm=math.nan, **fine) == 1 and "max_norm" in err()
    assert clip(L, [A], [-8], [0], **fine) == 1
    # overlaps: the same tensor twice in place, partly, an output over another input or output, another type in place
    assert clip(L, [A, A], [8, 8], [0, 0], **fine) == 1 and "overlaps" in err()
    assert clip(L, [A, A + 28], [8, 8], [0, 0], **fine) == 1 and "overlaps" in err()
    assert clip(L, [A, A + 32], [8, 8], [0, 0], **fine) == 1 and "sumsq" in err()
    assert clip(L, [A, A], [8, 8], [0, 0], outs=[C, C + 32], **fine) == 1 and "sumsq" in err()
    assert clip(L, [A, A + 64], [8, 8], [0, 0], outs=[C, C + 16], **fine) == 1 and "overlaps" in err()
    assert clip(L, [A, A + 64], [8, 8], [0, 0], outs=[C, A + 16], **fine) == 1 and "overlaps" in err()
    assert clip(L, [A, A + 4], [64, 1], [0, 0], outs=[C, A + 200], **fine) == 1 and "overlaps" in err()
    assert clip(L, [A], [8], [0], otypes=[1], **fine) == 1 and "same type" in err()
    n = (ctypes.c_int64 * 1)(8)
    t = (ctypes.c_int32 * 1)(0)
    assert L.kd_grad_sumsq((vp * 1)(A), n, t, 1, vp(0), vp(F), 1 << 20, None) == 1
    assert L.kd_grad_sumsq((vp * 1)(A), n, t, 1, vp(F + 4), vp(F), 1 << 20, None) == 3
    assert L.kd_grad_sumsq((vp * 1)(A), n, t, 1, vp(F), vp(F), 8, None) == 4
    assert L.kd_grad_sumsq((vp * 1)(A), n, t, -1, vp(F), vp(F), 8, None) == 1


@pytest.mark.parametrize("V", [2048, 2056])
def test_huge_chunks_are_cut(L, V):
    """A chunk's rows, in panels, keep within 32-bit offsets whatever chunk_rows asks for: 131072 rows of 16384 bf16
    are 4 GB."""
    s = [size(L, "kd_token_logp_workspace_size", 1 << 22, 16384, V, 1, 0, c) for c in (130560, 130816, 131072, 1 << 22)]
    assert s[0][0] == 0 and s[0][1] < s[1][1] and s[1] == s[2] == s[3]


def test_grad_clip_norm_refuses(L):
    n, t = (ctypes.c_int64 * 2)(8, 100000), (ctypes.c_int32 * 2)(0, 1)
    p, q = (vp * 2)(F, F + (1 << 20)), (vp * 2)(F, F + (1 << 21))

    def call(outs=p, max_norm=1.0, sumsq=F, norm=F, ws=F, wsb=0):
        return L.kd_grad_clip_norm(p, n, t, 2, outs, t, max_norm, vp(sumsq), vp(norm), vp(ws), wsb, None)

    assert [call(), call(outs=q), call(max_norm=-1.0), call(sumsq=0), call(norm=0), call(norm=F + 2), call(sumsq=F + 4),
            call(ws=0), call(ws=F + 8, wsb=1 << 20)] == [4, 4, 1, 1, 1, 3, 3, 1, 3]
    assert call(outs=(vp * 2)(F, F + 16)) == 1 and "overlaps" in err()

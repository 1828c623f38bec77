"""The C ABI of kdlayers.h on the CPU: what the header declares is exported, workspaces are sized as documented, and
bad arguments are refused on the host before any HIP call."""
import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
kd = pytest.importorskip("chunked_kl_loss_logit_amd")
B = kd._layers_binding
vp = ctypes.c_void_p
F = 0x10000  # aligned to 256, never dereferenced: the calls fail before any HIP call
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kd.LIB_PATH):
        pytest.fail("libkdloss.so is not built (run __graft_entry__.build())")
    return B.llib()


def test_exports_every_declared_symbol(L):
    text = open(os.path.join(ROOT, "include", "kdlayers.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(kd_[a-z0-9_]+)\s*\(", text)))
    assert sorted(kd.LAYERS_EXPORTS) == names
    assert all(hasattr(L, n) for n in names)


def err():
    return kd.lib().kd_last_error().decode()


def size(L, fn, *args):
    out = ctypes.c_size_t()
    st = getattr(L, fn)(*args, ctypes.byref(out))
    return st, out.value


def test_sizes(L):
    assert size(L, "kd_embedding_workspace_size", 0, 10, 8, 0) == (0, 0)
    for T, d in ((1, 8), (16384, 2048), (16385, 2048), (1 << 20, 512)):
        st, n = size(L, "kd_embedding_workspace_size", T, 32000, d, 0)
        assert st == 0 and 8 * T <= n <= T * (17 + d // 2) + 4 * 32000 + 2 * 4 * d + 1024 * 1024
        st, m = size(L, "kd_embedding_workspace_size", T, 32000, d, 1)
        assert st == 0 and min(4 * T * d, 1 << 29) <= m <= n + (1 << 30) + 1024
    a, b = (size(L, "kd_embedding_workspace_size", 10, 1 << 28, 1000, tied)[1] for tied in (0, 1))
    # a large vocabulary: slabs of as many columns as a launch takes (of the partial rows too, 2 for 10 tokens)
    assert b - a < 4 * 10 * 1000 - 2 * 4 * 1000
    assert size(L, "kd_embedding_workspace_size", -1, 10, 8, 1)[0] == 1
    assert size(L, "kd_embedding_workspace_size", 1 << 30, 10, 8, 1)[0] == 2
    assert size(L, "kd_embedding_workspace_size", 10, 0, 8, 1)[0] == 1
    assert size(L, "kd_embedding_workspace_size", 10, 10, 1 << 24, 1)[0] == 2
    assert size(L, "kd_layer_norm_workspace_size", 0, 100)[0] == 0
    assert size(L, "kd_layer_norm_workspace_size", 100, 0)[0] == 1
    a, b = (size(L, "kd_layer_norm_workspace_size", T, 4096)[1] for T in (1 << 16, 1 << 20))
    assert a == b  # a fixed number of partial rows
    assert size(L, "kd_int8_matmul_workspace_size", 4, 4096, 32000) == (0, 0)
    st, n = size(L, "kd_int8_matmul_workspace_size", 4096, 4096, 32000)
    assert st == 0 and n == 4096 * 4096
    assert size(L, "kd_int8_matmul_workspace_size", 1 << 24, 4096, 32000)[1] <= 1 << 30
    assert size(L, "kd_int8_matmul_workspace_size", 4, 4100, 32000)[0] == 2
    assert size(L, "kd_int8_matmul_workspace_size", 4, 1 << 17, 32000)[0] == 2
    assert L.kd_embedding_workspace_size(1, 1, 1, 0, None) == 1


def embed(L, tokens=F, table=F, scale=1.0, T=8, V=100, d=64, dt=1, tied=0, out=F):
    return L.kd_embedding_fwd(vp(tokens), vp(table), None, scale, T, V, d, dt, tied, vp(out), None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), 1), (dict(table=0), 1), (dict(out=0), 1), (dict(tokens=F + 2), 3), (dict(table=F + 1), 3),
    (dict(out=F + 1), 3), (dict(dt=0, table=F + 2), 3), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1),
    (dict(T=-1), 1), (dict(T=1 << 30), 2), (dict(V=0), 1), (dict(V=1 << 30), 2), (dict(d=0), 1), (dict(d=1 << 24), 2),
    (dict(dt=3), 1), (dict(T=0, tokens=0), 0),
])
def test_embedding_refuses(L, kw, code):
    assert embed(L, **kw) == code
    assert code == 0 or err()


def embed_bwd(L, grad=F, tokens=F, scale=1.0, T=8, V=100, d=64, dt=1, gdt=0, tied=0, acc=1, out=F, ws=F, wsb=0):
    return L.kd_embedding_bwd(vp(grad), vp(tokens), None, scale, T, V, d, dt, gdt, tied, acc, vp(out), vp(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(grad=0), 1), (dict(tokens=0), 1), (dict(out=0), 1), (dict(out=F + 2), 3), (dict(gdt=9), 1),
    (dict(dt=-1), 1), (dict(scale=math.nan), 1), (dict(T=-1), 1), (dict(V=0), 1), (dict(d=1 << 24), 2),
    (dict(ws=0), 1), (dict(ws=F + 16, wsb=BIG), 3), (dict(T=0, grad=0, tokens=0, ws=0), 0),
])
def test_embedding_bwd_refuses(L, kw, code):
    assert embed_bwd(L, **kw) == code
    assert code == 0 or err()


def rows(L, x=F, T=8, d=100, dt=1, kind=1, group=32, q=F, scale=F, back=False):
    if back:
        return L.kd_rows_dequantize(vp(q), vp(scale), T, d, kind, group, dt, vp(x), None)
    return L.kd_rows_quantize(vp(x), T, d, dt, kind, group, vp(q), vp(scale), None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(x=0), 1), (dict(x=F + 1), 3), (dict(q=0), 1), (dict(scale=0), 1), (dict(scale=F + 2), 3), (dict(kind=0), 1),
    (dict(kind=3), 1), (dict(group=16), 1), (dict(group=1024), 1), (dict(group=-32), 1), (dict(dt=4), 1),
    (dict(T=-1), 1), (dict(d=0), 1), (dict(T=1 << 30), 2), (dict(T=0, x=0, q=0), 0),
])
def test_rows_refuse(L, kw, code, back):
    assert rows(L, back=back, **kw) == code
    assert code == 0 or err()


def norm(L, x=F, w=F, b=F, eps=1e-5, T=8, d=100, dt=1, wdt=1, y=F, mean=F, rstd=F, kind=0, group=0, q=0, scale=0):
    return L.kd_layer_norm_fwd(vp(x), vp(w), vp(b), None, eps, T, d, dt, wdt, vp(y), vp(mean), vp(rstd), kind, group,
                               vp(q), vp(scale), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), 1), (dict(y=0), 1), (dict(x=F + 1), 3), (dict(w=F + 1), 3), (dict(b=F + 1), 3), (dict(mean=F + 2), 3),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(wdt=2), 2), (dict(dt=0, wdt=1), 2),
    (dict(wdt=5), 1), (dict(dt=5), 1), (dict(kind=1), 1), (dict(kind=1, q=F), 1), (dict(kind=7, q=F, scale=F), 1),
    (dict(kind=2, group=48, q=F, scale=F), 1), (dict(kind=2, group=32, q=F, scale=F + 1), 3), (dict(T=-1), 1),
    (dict(d=0), 1), (dict(d=1 << 24), 2), (dict(T=0, x=0, y=0), 0),
])
def test_layer_norm_refuses(L, kw, code):
    assert norm(L, **kw) == code
    assert code == 0 or err()


def norm_bwd(L, grad=F, x=F, w=F, mean=F, rstd=F, T=8, d=100, dt=1, wdt=0, kind=0, group=0, q=0, scale=0, dx=F, dw=F,
             db=F, ws=F, wsb=0):
    return L.kd_layer_norm_bwd(vp(grad), vp(x), vp(w), None, vp(mean), vp(rstd), T, d, dt, wdt, kind, group, vp(q),
                               vp(scale), vp(dx), vp(dw), vp(db), vp(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(grad=0), 1), (dict(x=0), 1), (dict(mean=0), 1), (dict(rstd=0), 1), (dict(dx=0, dw=0, db=0), 1),
    (dict(dx=0), 4), (dict(dw=0, db=0), 4), (dict(dx=F + 1), 3), (dict(dw=F + 2), 3), (dict(db=F + 1), 3),
    (dict(kind=1, x=0, q=F, scale=F), 4), (dict(kind=1, q=F, scale=F), 1), (dict(kind=1, x=0, q=F), 1),
    (dict(kind=1, x=0, scale=F), 1), (dict(kind=3, x=0, q=F, scale=F), 1), (dict(kind=1, group=8, x=0, q=F, scale=F), 1),
    (dict(wdt=2), 2), (dict(ws=0), 1), (dict(ws=F + 8, wsb=BIG), 3), (dict(T=-1), 1), (dict(T=0, dw=0, db=0, wsb=BIG), 0),
])
def test_layer_norm_bwd_refuses(L, kw, code):
    assert norm_bwd(L, **kw) == code
    assert code == 0 or err()


def int8(L, x=F, sx=F, w=F, sw=F, T=300, d=64, V=33000, dt=0, out=F, ws=F, wsb=0):
    return L.kd_int8_matmul(vp(x), vp(sx), vp(w), vp(sw), T, d, V, dt, vp(out), vp(ws), wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(), 4), (dict(x=0), 1), (dict(w=0), 1), (dict(sx=0), 1), (dict(sw=0), 1), (dict(out=0), 1), (dict(x=F + 8), 3),
    (dict(w=F + 1), 3), (dict(sx=F + 2), 3), (dict(sw=F + 1), 3), (dict(out=F + 2), 3), (dict(dt=3), 1),
    (dict(d=0), 1), (dict(d=24), 2), (dict(d=1 << 17), 2), (dict(V=0), 1), (dict(V=1 << 30), 2), (dict(T=-1), 1),
    (dict(T=1 << 30), 2), (dict(ws=0), 1), (dict(ws=F + 64, wsb=BIG), 3), (dict(T=0, x=0, out=0), 0),
])
def test_int8_matmul_refuses(L, kw, code):
    assert int8(L, **kw) == code
    assert code == 0 or err()

"""Sizes next to the limits of the policy operators' plans, on the CPU: what the library reports for a shape tells how
many rows a chunk has."""
import ctypes
import os
import sys

import pytest
import torch

kd = pytest.importorskip("chunked_kl_loss_logit_amd")
B = kd._policy_binding
BF16, F32 = 1, 0
REACH = (1 << 32) - 65537  # bytes that 32-bit offsets span, less what one load may reach beyond


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(kd.LIB_PATH):
        pytest.fail("libkdloss.so is not built (run __graft_entry__.build())")
    return B.plib()


def size(L, T, d, V, chunk, dt=BF16, dw=F32):
    out = ctypes.c_size_t()
    assert L.kd_token_logp_workspace_size(T, d, V, dt, dw, chunk, ctypes.byref(out)) == 0
    return out.value


def most_rows(L, T, d, V):
    """The rows of the largest chunk: the smallest chunk_rows that is given what any larger one is."""
    top = size(L, T, d, V, T)
    lo, hi = 1, T // 256  # in 256 rows
    while lo < hi:
        mid = (lo + hi) // 2
        if size(L, T, d, V, 256 * mid) == top:
            hi = mid
        else:
            lo = mid + 1
    return 256 * lo


def in_reach(rows, V):
    """dZ's columns in whole tiles, then four pieces of 32 for its tail and the zeros behind it, 2 bytes each."""
    return rows * (-(-V // 256) * 256 + 128) * 2 <= REACH


@pytest.mark.parametrize("d,V", [(64, 47368), (1024, 87048), (2048, 87048), (64, 37128), (256, 23560), (256, 22536),
                                 (1024, 1198088), (1024, 1397768), (64, 47360), (64, 47104), (2048, 2056)])
def test_dz_panels_keep_to_32_bits(L, d, V):
    rows = most_rows(L, 1 << 20, d, V)
    assert in_reach(rows, V), f"{rows} rows of {V}"


def test_dz_panels_keep_to_32_bits_everywhere(L):
    """Vocabularies whose last tile leaves the tail pieces no room of its own, and others beside them."""
    for V in list(range(8 * 1024, 300000, 1016)) + [256 * k + r for k in range(40, 1200, 7) for r in (8, 32, 128, 136, 248)]:
        rows = most_rows(L, 1 << 18, 512, V)
        assert in_reach(rows, V), f"{rows} rows of {V}"


def test_a_row_tile_too_large_for_the_ring(L):
    """256 rows of 16 M columns are 8 GB of dZ, beyond 32-bit offsets whatever the chunk: the register-fed tiles take
    them, with little beside dZ (the ring would keep 8 MB of dH parts)."""
    V = 1 << 24
    a, b = size(L, 128, 32, V, 256), size(L, 128, 32, V, 256, dw=BF16)
    assert a == b  # one chunk: a bf16 dW needs no float32 buffer
    dz = 256 * V * 2
    assert dz <= a < dz + (4 << 20)
    assert size(L, 300, 32, V, 0) < dz + (4 << 20)


@pytest.mark.parametrize("call", [lambda p: kd.clip_grad_norm_([p], 1.0), lambda p: kd.clip_grad_norm_(iter([p]), 1.0),
                                  lambda p: kd.clip_grad_norm_(p, 1.0),
                                  lambda p: kd.clip_grad_norm_([torch.ones(3), p], 1.0)])
def test_parameters_are_not_clipped(call):
    """Refused before anything is looked up on a device, in and out of grad mode."""
    p = torch.nn.Parameter(torch.full((3,), 5.0))
    with pytest.raises(ValueError, match=r"\.grad"):
        call(p)
    with torch.no_grad(), pytest.raises(ValueError, match=r"\.grad"):
        call(p)
    assert (p == 5.0).all()


def test_what_autograd_follows_is_not_clipped_in_grad_mode():
    x = torch.ones(3, requires_grad=True) * 2
    with pytest.raises(ValueError, match="must not require a gradient"):
        kd.clip_grad_norm_([x], 1.0)
    with torch.no_grad(), pytest.raises(ValueError, match="on the GPU"):  # accepted so far
        kd.clip_grad_norm_([x], 1.0)
    with pytest.raises(ValueError, match="on the GPU"):  # only read
        kd.clip_grad_norm([x], 1.0, out=[torch.ones(3)])


@pytest.mark.parametrize("chunk", [2 ** 63 - 1, 2 ** 63 - 254, 2 ** 63 - 255, 2 ** 63 - 256, 2 ** 62, 1000])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_any_number_of_chunk_rows_is_cut_to_the_rows_present(L, chunk, dt):
    """The largest numbers round up to beyond 63 bits."""
    for T, d, V in ((1000, 1024, 7016), (1000, 256, 1032), (1, 64, 64)):
        assert size(L, T, d, V, chunk, dt) == size(L, T, d, V, 1024, dt)
    sizes = [("kd_topk_kl_workspace_size", (1000, 1024, 7016, 16, dt)), ("kd_topk_kl_fwd_bwd_workspace_size", (1000, 1024, 7016, 16, dt)),
             ("kd_full_kl_workspace_size", (1000, 1024, 256, 7016, dt)), ("kd_full_kl_fwd_bwd_workspace_size", (1000, 1024, 256, 7016, dt))]
    for fn, args in sizes:
        got = []
        for c in (chunk, 1024):
            out = ctypes.c_size_t()
            assert getattr(L, fn)(*args, c, ctypes.byref(out)) == 0
            got.append(out.value)
        assert got[0] == got[1], fn


@pytest.mark.parametrize("T,d,V,dt", [(1500, 4096, 128256, BF16), (4096, 2048, 128256, BF16), (1, 4096, 128256, BF16),
                                      (100000, 2048, 32000, BF16), (777, 1024, 32000, F32), (20000, 64, 264, F32)])
def test_a_forward_alone_needs_no_dz(L, T, d, V, dt):
    """Its workspace is records (16 bytes a row and tile of at least 128 columns, of a chunk of up to 4096 rows), the
    chunk's rows of H and the list of valid rows."""
    out = ctypes.c_size_t()
    assert L.kd_token_logp_fwd_workspace_size(T, d, V, dt, ctypes.byref(out)) == 0
    rows, elem = min(4096, -(-T // 256) * 256), 2 if dt == BF16 else 4
    assert out.value <= -(-V // 128) * rows * 16 + rows * -(-d // 128) * 128 * elem + 4 * T + 2048
    assert out.value <= size(L, T, d, V, 0, dt)
    assert out.value < rows * V * elem / 3


def test_forward_size_refuses(L):
    out = ctypes.c_size_t()
    assert L.kd_token_logp_fwd_workspace_size(0, 64, 264, BF16, ctypes.byref(out)) == 0 and out.value == 0
    assert L.kd_token_logp_fwd_workspace_size(8, 60, 264, BF16, ctypes.byref(out)) == 2
    assert L.kd_token_logp_fwd_workspace_size(-1, 64, 264, BF16, ctypes.byref(out)) == 1
    assert L.kd_token_logp_fwd_workspace_size(8, 64, 264, 2, ctypes.byref(out)) == 1
    assert L.kd_token_logp_fwd_workspace_size(8, 64, 264, BF16, None) == 1

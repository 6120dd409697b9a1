"""Results and workspaces over what a call reads, and limits of sizes, on the host (no GPU needed: the addresses are made up).

Vectors (bias, row scales, norm weights, positions, frequencies) and the workspace, beside the rows that
test_linear.py and test_rotary.py cover.  A call that only touches its neighbours is not refused; without a GPU it
ends with the launch's error.
"""
from __future__ import annotations

import os

import pytest
import torch

import rmsnorm_qknorm_b200 as qk
from rmsnorm_qknorm_b200 import build as qbuild

OK, NULL, SHAPE, DTYPE, EPS, ALIGN, CUDA, TIMEOUT, UNSUP = range(9)
F32, BF16 = 0, 1
P = 0x100000  # made-up device addresses, a MiB apart; validation never dereferences them
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would launch on made-up addresses")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qk.library_path()):
        qbuild.build()
    return qk.load_library()


# M 8, N 64, K 32 bf16: y and preact 1024 bytes, x 512, W 4096, bias 128 (fp32 256), row scales 32
def linear(lib, y=3 * P, b=4 * P, bdt=BF16, inv=5 * P, z=6 * P, res=7 * P):
    return lib.linear_fused(P, 2 * P, y, 8, 64, 32, 32, 32, 64, b, bdt, 0, res, 64, inv, z, 64, None)


@pytest.mark.parametrize("kw", [dict(b=3 * P), dict(b=3 * P + 1008), dict(b=3 * P - 112), dict(b=3 * P - 240, bdt=F32),
                                dict(inv=3 * P + 1020), dict(inv=3 * P - 28), dict(b=6 * P + 512), dict(inv=6 * P),
                                dict(inv=6 * P + 1020)])
def test_linear_results_over_vectors_are_refused(lib, kw):
    assert linear(lib, **kw) == UNSUP
    assert "shares memory" in lib.qkn_last_error().decode()


@no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(b=3 * P + 1024), dict(b=3 * P - 128), dict(b=3 * P - 256, bdt=F32),
                                dict(inv=3 * P + 1024), dict(inv=6 * P - 32), dict(res=3 * P)])
def test_linear_results_beside_vectors_pass(lib, kw):
    assert linear(lib, **kw) == CUDA


# dy, preact [8, 64]; x [8, 32], W [64, 32] and their gradients; dbias 256 bytes
def linear_back(lib, ws, db=7 * P):
    need = lib.linear_fused_backward_workspace_bytes(8, 64, 32, 2)
    return lib.linear_fused_backward(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, db, 8, 64, 32, 64, 64, 32, 32, 32, 32, 2, ws, need,
                                     None)


@pytest.mark.parametrize("at,size", [(1, 1024), (2, 1024), (3, 512), (4, 4096), (5, 512), (6, 4096), (7, 256)])
def test_linear_workspace_over_others_is_refused(lib, at, size):
    need = lib.linear_fused_backward_workspace_bytes(8, 64, 32, 2)
    for ws in (at * P, at * P + size - 16, at * P - need // 16 * 16 + 16):
        assert linear_back(lib, ws) == UNSUP
        assert "workspace shares memory" in lib.qkn_last_error().decode()


@no_gpu
def test_linear_workspace_beside_others_passes(lib):
    need = lib.linear_fused_backward_workspace_bytes(8, 64, 32, 2)
    for ws in (8 * P, P + 1024, 7 * P + 256, 5 * P - (need + 15) // 16 * 16):
        assert linear_back(lib, ws) == CUDA


# T 4, q 128 and k 64 wide: rows of 1024 and 512 bytes in all, positions 32, 32 frequencies 256
def rotary(lib, qo=3 * P, ko=4 * P, pos=5 * P, freq=6 * P):
    return lib.rotary_apply(P, 2 * P, qo, ko, 4, 128, 64, 128, 64, 128, 64, 64, pos, 64, freq, 64, 0, 1.0, 0, BF16, None)


def qknorm(lib, qo=3 * P, ko=4 * P, pos=5 * P, freq=6 * P, wq=7 * P, wk=8 * P, r=64):
    return lib.qknorm_rotary(P, 2 * P, wq, wk, qo, ko, 4, 128, 64, 128, 64, 128, 64, 64, pos, 64, freq, r, 0, 1.0, BF16, BF16,
                             1e-6, None)


def back(lib, dq=3 * P, dk=4 * P, pos=5 * P, freq=6 * P, wq=7 * P, wk=8 * P, dwq=9 * P, dwk=10 * P, ws=11 * P):
    need = lib.qknorm_rotary_backward_workspace_bytes(4, 128, 64)
    return lib.qknorm_rotary_backward(12 * P, 13 * P, P, 2 * P, wq, wk, dq, dk, dwq, dwk, 4, 128, 64, 128, 64, 128, 64, 128,
                                      64, 64, pos, 64, freq, 64, 0, 1.0, BF16, BF16, 1e-6, ws, need, None)


@pytest.mark.parametrize("call", [rotary, qknorm, back])
@pytest.mark.parametrize("kw", [dict(pos=3 * P), dict(pos=3 * P + 1016), dict(pos=3 * P - 24), dict(pos=4 * P + 504),
                                dict(freq=3 * P + 8), dict(freq=4 * P - 248)])
def test_rotary_results_over_positions_and_frequencies_are_refused(lib, call, kw):
    assert call(lib, **kw) == UNSUP
    assert "positions or frequencies" in lib.qkn_last_error().decode()


@pytest.mark.parametrize("call", [qknorm, back])
@pytest.mark.parametrize("kw", [dict(wq=3 * P), dict(wq=4 * P + 510), dict(wk=3 * P - 126), dict(wk=4 * P)])
def test_rotary_results_over_weights_are_refused(lib, call, kw):
    assert call(lib, **kw) == UNSUP
    assert "shares memory with weights" in lib.qkn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(dwq=7 * P), dict(dwq=8 * P + 124), dict(dwk=7 * P - 252), dict(dwq=5 * P - 508),
                                dict(dwk=6 * P + 252)])
def test_weight_gradients_over_inputs_are_refused(lib, kw):
    assert back(lib, **kw) == UNSUP


@pytest.mark.parametrize("at,size", [(1, 1024), (2, 512), (3, 1024), (4, 512), (5, 32), (6, 256), (7, 256), (8, 128), (9, 512),
                                     (10, 256), (12, 1024), (13, 512)])
def test_rotary_workspace_over_others_is_refused(lib, at, size):
    need = lib.qknorm_rotary_backward_workspace_bytes(4, 128, 64)
    for ws in (at * P, at * P + size - 16, at * P - need // 16 * 16 + 16):
        assert back(lib, ws=ws) == UNSUP
        assert "workspace shares memory" in lib.qkn_last_error().decode()


@no_gpu
def test_rotary_results_beside_others_pass(lib):
    assert rotary(lib) == CUDA and rotary(lib, pos=3 * P + 1024, freq=4 * P - 256) == CUDA
    assert rotary(lib, qo=None, ko=None) == CUDA
    assert qknorm(lib, wq=3 * P + 1024, wk=4 * P - 128) == CUDA
    assert qknorm(lib, r=0, pos=3 * P, freq=3 * P) == CUDA  # not read without a rotation
    assert back(lib) == CUDA and back(lib, dwq=7 * P + 256, dwk=8 * P - 256) == CUDA
    assert back(lib, ws=3 * P + 1024) == CUDA and back(lib, ws=5 * P + 32) == CUDA


def meets(a, b):
    """Whether rows (start, rows, bytes, pitch) share a byte, byte by byte."""
    return bool(set(a[0] + i * a[3] + c for i in range(a[1]) for c in range(a[2]))
                & set(b[0] + i * b[3] + c for i in range(b[1]) for c in range(b[2])))


@no_gpu
def test_rows_under_other_pitches_against_every_byte(lib):
    # q's rows and k's result, both of small widths and pitches, among one another in all ways; the rest lies far away
    import random
    rng, met = random.Random(5), 0
    for _ in range(4000):
        T, dq, dk = rng.randint(1, 9), 2 * rng.randint(1, 5), 2 * rng.randint(1, 5)
        lq, lk = dq + rng.choice([0, 0, 1, 2, 7, rng.randint(0, 60)]), dk + rng.choice([0, 1, 2, 5, rng.randint(0, 60)])
        at = 64 * P + 2 * rng.randint(-T * lk - 4, T * lq + 4)
        st = lib.rotary_apply(64 * P, P, 2 * P, at, T, dq, dk, lq, dk, dq, lk, 2, 4 * P, 64, 5 * P, 2, 0, 1.0, 0, BF16, None)
        hit = meets((64 * P, T, 2 * dq, 2 * lq), (at, T, 2 * dk, 2 * lk))
        met += hit
        assert st == (UNSUP if hit else CUDA), (T, dq, dk, lq, lk, at - 64 * P)
    assert 400 < met < 3600


@no_gpu
def test_many_rows_under_two_pitches_are_checked_at_once(lib):
    # every 32 bytes against every 48, apart from one another (a walk over 2^28 rows takes seconds)
    import time
    T, A = 1 << 28, 1 << 40

    def call(at):
        return lib.rotary_apply(A, None, at, None, T, 2, 0, 16, 0, 24, 0, 2, 1 << 50, 64, 1 << 52, 2, 0, 1.0, 0, BF16, None)

    call(A)  # the first call looks for a device
    t0 = time.perf_counter()
    assert call(A + 8) == CUDA and time.perf_counter() - t0 < 1.0
    # the last row of q_out alone reaches the first one of q
    assert call(A + 8 - 48 * (T - 1)) == CUDA and call(A + 2 - 48 * (T - 1)) == UNSUP


@no_gpu
def test_the_widest_rows(lib):
    # the columns of q and k together, rounded up to the blocks that add up the weights' gradients, fit 31 bits
    A, W = 1 << 40, (1 << 30) - 16

    def call(dq, dk):
        at = [A + (i << 33) for i in range(13)]
        return lib.qknorm_rotary_backward(*at[:10], 1, dq, dk, dq, dk, dq, dk, dq, dk, 2, at[10], 64, at[11], 2, 0, 1.0, BF16,
                                          BF16, 1e-6, None, 0, None)

    assert call(W, W) == CUDA and call(W + 2, W) == SHAPE and call(W, W + 2) == SHAPE
    assert lib.qknorm_rotary_backward_workspace_bytes(1, W, W) >= 8 * W
    assert lib.qknorm_rotary_backward_workspace_bytes(1, W, W + 2) == 0

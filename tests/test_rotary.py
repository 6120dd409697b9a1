"""Rotary positions on the host: frequencies, and the refusals of the C entry points and the binding (no GPU needed)."""
from __future__ import annotations

import math
import os

import pytest
import torch

import rmsnorm_qknorm_b200 as qk
from rmsnorm_qknorm_b200 import build as qbuild

OK, NULL, SHAPE, DTYPE, EPS, ALIGN, CUDA, TIMEOUT, UNSUP = range(9)
F32, BF16 = 0, 1
P = 0x10000  # a fake 64 KiB-aligned device address; validation never dereferences it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qk.library_path()):
        qbuild.build()
    return qk.load_library()


def test_plain_linear_and_ntk_frequencies():
    f, m = qk.rotary_inv_freq(8, 10000.0, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    g, m = qk.rotary_inv_freq(8, 10000.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4) and m == 1.0
    n, _ = qk.rotary_inv_freq(8, 10000.0, scaling="ntk", factor=4.0, device="cpu")
    assert n[0] == 1.0 and abs(float(n[-1] / f[-1]) - 0.25) < 1e-15  # fastest kept, slowest slowed by the factor


def test_yarn_keeps_fast_pairs_and_slows_slow_ones():
    r, L, s = 128, 4096, 8.0
    f, _ = qk.rotary_inv_freq(r, device="cpu")
    y, m = qk.rotary_inv_freq(r, scaling="yarn", factor=s, original=L, device="cpu")
    assert m == pytest.approx(0.1 * math.log(8) + 1)
    turns = L * f / (2 * math.pi)
    assert torch.allclose(y[turns > 64], f[turns > 64], rtol=1e-15)
    assert torch.allclose(y[turns < 0.5], f[turns < 0.5] / s, rtol=1e-15)
    assert bool((y <= f).all()) and bool((y >= f / s * (1 - 1e-15)).all())
    same, m1 = qk.rotary_inv_freq(r, scaling="yarn", factor=1.0, original=L, device="cpu")
    assert torch.allclose(same, f, rtol=1e-15) and m1 == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0),
                                dict(rotary_dim=8, scaling="cubic"), dict(rotary_dim=8, factor=0.5),
                                dict(rotary_dim=8, scaling="yarn", factor=2.0),
                                dict(rotary_dim=2, scaling="ntk", factor=2.0),
                                dict(rotary_dim=8, scaling="yarn", original=64, fast=1.0, slow=2.0),
                                dict(rotary_dim=8, base=float("inf")), dict(rotary_dim=8, factor=float("nan"))])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        qk.rotary_inv_freq(device="cpu", **kw)


def rot(lib, q=P, k=P, qo=P, ko=P, T=4, dq=128, dk=64, ldq=None, ldk=None, ldqo=None, ldko=None, D=64, pos=P, bits=64,
        freq=P, r=64, layout=0, m=1.0, inverse=0, act=BF16):
    return lib.rotary_apply(q, k, qo, ko, T, dq, dk, ldq or dq, ldk or dk, ldqo or dq, ldko or dk, D, pos, bits, freq, r,
                            layout, m, inverse, act, None)


def test_rotary_refusals(lib):
    assert rot(lib, q=None) == NULL and rot(lib, k=None) == NULL and rot(lib, pos=None) == NULL
    assert rot(lib, freq=None) == NULL
    for kw in (dict(T=-1), dict(dq=0), dict(ldq=64), dict(ldqo=64), dict(r=0), dict(r=63), dict(r=66), dict(D=48),
               dict(D=1026, dq=1026, dk=1026, r=1026), dict(m=float("inf")), dict(m=float("nan")), dict(dk=96)):
        assert rot(lib, **kw) == SHAPE, kw
    assert rot(lib, layout=2) == UNSUP and rot(lib, bits=16) == DTYPE and rot(lib, act=3) == DTYPE
    for kw in (dict(q=P + 1), dict(ko=P + 1), dict(pos=P + 4), dict(freq=P + 4), dict(act=F32, q=P + 2)):
        assert rot(lib, **kw) == ALIGN, kw
    assert "aligned" in lib.qkn_last_error().decode()
    assert rot(lib, T=0, q=None, k=None, qo=None, ko=None, pos=None) == OK


def norm_rot(lib, q=P, k=P, wq=P, wk=P, T=4, dq=128, dk=64, ldq=None, D=64, pos=P, bits=64, freq=P, r=64, layout=0,
             m=1.0, act=BF16, wdt=BF16, eps=1e-6):
    return lib.qknorm_rotary(q, k, wq, wk, P, P, T, dq, dk, ldq or dq, dk or 1, dq, dk or 1, D, pos, bits, freq, r,
                             layout, m, act, wdt, eps, None)


def test_qknorm_rotary_refusals(lib):
    assert norm_rot(lib, wq=None) == NULL and norm_rot(lib, wk=None) == NULL and norm_rot(lib, pos=None) == NULL
    assert norm_rot(lib, eps=-1.0) == EPS and norm_rot(lib, eps=float("nan")) == EPS
    assert norm_rot(lib, r=2, D=0) == SHAPE and norm_rot(lib, ldq=100) == SHAPE
    assert norm_rot(lib, wdt=9) == DTYPE and norm_rot(lib, wdt=F32, wq=P + 2) == ALIGN
    assert norm_rot(lib, T=0, r=0, D=0, pos=None, freq=None, q=None, k=None) == OK


def back(lib, gq=P, q=P, wq=P, dqi=P, dwq=P, dwk=P, T=4, dq=128, dk=64, ldgq=None, r=64, eps=1e-6, ws=P, nbytes=1 << 30,
         act=BF16):
    return lib.qknorm_rotary_backward(gq, P, q, P, wq, P, dqi, P, dwq, dwk, T, dq, dk, ldgq or dq, dk, dq, dk, dq, dk, 64,
                                      P, 64, P, r, 0, 1.0, act, BF16, eps, ws, nbytes, None)


def test_backward_refusals(lib):
    for kw in (dict(gq=None), dict(q=None), dict(wq=None), dict(dqi=None), dict(dwq=None), dict(dwk=None)):
        assert back(lib, **kw) == NULL, kw
    assert back(lib, ldgq=8) == SHAPE and back(lib, r=2048) == SHAPE and back(lib, eps=-1.0) == EPS
    assert back(lib, dwq=P + 2) == ALIGN and back(lib, gq=P + 1) == ALIGN and back(lib, ws=P + 8) == ALIGN
    need = lib.qknorm_rotary_backward_workspace_bytes(4, 128, 64)
    assert need > 0 and back(lib, nbytes=need - 1) == SHAPE
    assert "workspace" in lib.qkn_last_error().decode()
    assert lib.qknorm_rotary_backward_workspace_bytes(4, 0, 64) == 0


def test_binding_refuses_cpu_tensors_and_wrong_arguments():
    x, f = torch.zeros(4, 64), torch.ones(32, dtype=torch.float64)
    pos = torch.arange(4)
    with pytest.raises(ValueError, match="CUDA"):
        qk.rotary_apply(x, None, pos, f, 64)
    with pytest.raises(ValueError, match="CUDA"):
        qk.qknorm_rotary(x, None, torch.ones(64), None, pos, f, 64)
    with pytest.raises(ValueError, match="CUDA"):
        qk.qknorm_rotary_backward(x, None, x, None, torch.ones(64), None, pos, f, 64)


def test_yarn_refuses_a_length_without_a_slow_turn():
    with pytest.raises(ValueError, match="original length"):
        qk.rotary_inv_freq(8, scaling="yarn", factor=2.0, original=6, device="cpu")


# Results over inputs, other than a result in place of its own operand.  Row width 128 (q) and 64 (k) bf16.
@pytest.mark.parametrize("kw", [dict(q=P, k=P, qo=None, ko=None),                  # one tensor twice, in place
                                dict(q=P, k=P + 128, qo=None, ko=None),            # k's columns among q's
                                dict(q=P, k=4 * P, qo=2 * P, ko=2 * P),            # one result for both
                                dict(q=P, k=4 * P, qo=4 * P, ko=8 * P),            # q's result over k
                                dict(q=P, k=4 * P, qo=P + 256, ko=8 * P),          # a row further down
                                dict(q=P, k=4 * P, qo=P, ldqo=136, ko=8 * P),      # in place with another pitch
                                dict(q=P, k=4 * P, qo=2 * P, ko=2 * P + 256, ldqo=256, ldko=200)])
def test_results_over_inputs_are_refused(lib, kw):
    assert rot(lib, **kw) == UNSUP
    assert "shares memory" in lib.qkn_last_error().decode()


def test_gradients_over_inputs_are_refused(lib):
    for kw in (dict(dqi=P), dict(gq=P, q=4 * P, dqi=4 * P), dict(gq=P, q=4 * P, dqi=P + 512)):
        assert back(lib, **kw) == UNSUP, kw


# gq, gk, q, k, dq_in, dk_in lie at P .. 6 P, the weights at 7 P and 8 P
@pytest.mark.parametrize("dwq,dwk", [(9 * P, 9 * P), (9 * P, 9 * P + 508), (6 * P + 4, 10 * P), (9 * P, P + 1020)])
def test_weight_gradients_over_others_are_refused(lib, dwq, dwk):
    assert lib.qknorm_rotary_backward(P, 2 * P, 3 * P, 4 * P, 7 * P, 8 * P, 5 * P, 6 * P, dwq, dwk, 4, 128, 64, 128, 64, 128,
                                      64, 128, 64, 64, 11 * P, 64, 12 * P, 64, 0, 1.0, BF16, BF16, 1e-6, 13 * P, 1 << 16,
                                      None) == UNSUP
    assert "gradient of weights" in lib.qkn_last_error().decode()

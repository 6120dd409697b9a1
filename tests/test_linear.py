"""Refusals of linear_fused and linear_fused_backward on the host (no GPU needed)."""
from __future__ import annotations

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


def lin(lib, x=P, W=P, y=P, M=8, N=64, K=32, ldx=None, ldw=None, ldy=None, b=None, bdt=BF16, act=0, res=None, ldr=0,
        inv=None, z=None, ldz=0):
    return lib.linear_fused(x, W, y, M, N, K, ldx or K, ldw or K, ldy or N, b, bdt, act, res, ldr, inv, z, ldz, None)


def test_forward_refusals(lib):
    for kw in (dict(x=None), dict(W=None), dict(y=None)):
        assert lin(lib, **kw) == NULL, kw
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(N=60), dict(K=36), dict(ldx=24), dict(ldw=36), dict(ldy=60),
               dict(res=P, ldr=32), dict(z=P, ldz=68), dict(M=1 << 31)):
        assert lin(lib, **kw) == SHAPE, kw
    assert lin(lib, act=5) == UNSUP and lin(lib, act=-1) == UNSUP and lin(lib, b=P, bdt=7) == DTYPE
    for kw in (dict(x=P + 8), dict(W=P + 2), dict(y=P + 4), dict(b=P + 8), dict(res=P + 8, ldr=64),
               dict(z=P + 8, ldz=64), dict(inv=P + 2)):
        assert lin(lib, **kw) == ALIGN, kw
    assert "16-byte" in lib.qkn_last_error().decode()
    assert lin(lib, M=0, x=None, W=None, y=None) == OK


def back(lib, dy=P, z=P, x=P, W=P, dx=P, dW=P, db=P, M=8, N=64, K=32, lddy=None, ldz=None, lddx=None, act=2, ws=P,
         nbytes=1 << 30):
    return lib.linear_fused_backward(dy, z, x, W, dx, dW, db, M, N, K, lddy or N, ldz or N, K, K, lddx or K, K, act, ws,
                                     nbytes, None)


def test_backward_refusals(lib):
    for kw in (dict(dy=None), dict(z=None), dict(x=None), dict(W=None)):
        assert back(lib, **kw) == NULL, kw
    for kw in (dict(M=-1), dict(N=60), dict(K=36), dict(lddy=60), dict(ldz=32), dict(lddx=8)):
        assert back(lib, **kw) == SHAPE, kw
    assert back(lib, act=9) == UNSUP
    for kw in (dict(dy=P + 8), dict(dW=P + 8), dict(db=P + 2), dict(ws=P + 8)):
        assert back(lib, **kw) == ALIGN, kw
    need = lib.linear_fused_backward_workspace_bytes(8, 64, 32, 2)
    assert need > 8 * 64 * 2 and back(lib, nbytes=need - 1) == SHAPE
    assert "workspace" in lib.qkn_last_error().decode()
    assert lib.linear_fused_backward_workspace_bytes(8, 0, 32, 2) == 0
    assert back(lib, dx=None, dW=None, db=None) == OK  # nothing asked for


def test_binding_refusals():
    x, W = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        qk.linear_fused(x, W)
    with pytest.raises(ValueError, match="CUDA"):
        qk.linear_fused_backward(torch.zeros(4, 64, dtype=torch.bfloat16), x, W)
    with pytest.raises(ValueError, match="act"):
        qk.linear_fused_backward_workspace_bytes(4, 64, 32, "tanh")


@pytest.mark.parametrize("kw", [dict(y=P), dict(W=4 * P, y=4 * P), dict(W=4 * P, y=8 * P, z=8 * P, ldz=64),
                                dict(W=4 * P, y=8 * P, res=8 * P + 16, ldr=64),     # a shifted residual
                                dict(W=4 * P, y=8 * P, res=8 * P, ldr=72),          # in place, another pitch
                                dict(W=4 * P, y=8 * P, z=P, ldz=64), dict(W=4 * P, y=8 * P, z=4 * P + 4000, ldz=64),
                                dict(W=4 * P, y=8 * P, z=16 * P, ldz=64, res=16 * P, ldr=64),
                                dict(x=P, ldx=128, W=4 * P, y=P + 32, ldy=128)])    # columns that cross x's
def test_results_over_inputs_are_refused(lib, kw):
    assert lin(lib, **kw) == UNSUP
    assert "shares memory" in lib.qkn_last_error().decode()


@pytest.mark.parametrize("kw", [dict(dx=P), dict(dx=2 * P, dW=P), dict(dx=2 * P, dW=2 * P), dict(dx=2 * P, dW=2 * P + 256),
                                dict(dx=2 * P, dW=4 * P, db=2 * P + 508), dict(dx=2 * P, dW=4 * P, db=P + 4)])
def test_gradients_over_inputs_are_refused(lib, kw):
    assert back(lib, **kw) == UNSUP

"""Every finite bf16 pre-activation through the linear layer's activations and their slopes.

Bounds as in test_linear_gpu.py: an activation and its slope are good to 2^-17 of their parts, which are at most
1 + |z| where the result is not saturated (beyond |z| = 128 it is z, 0 or 1 exactly), one factor 2 for their sum;
results below 10^-36 may become zero.  An activation is rounded to bf16 once, a slope (as the sum of one row) stays fp32.
"""
from __future__ import annotations

import pytest
import torch

import rmsnorm_qknorm_b200 as qk
from test_linear_gpu import ACTS, DEV, U, close, slope, value

pytestmark = pytest.mark.gpu


def finite():
    z = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    assert z.numel() == 65280 and float(z.max()) > 3e38
    return z


@pytest.mark.parametrize("act", ACTS)
def test_every_value(cuda_lib, act):
    z = finite()
    x, ref = z.view(-1, 8), value(z.double(), act).view(-1, 8)
    y = qk.linear_fused(x, torch.eye(8, device=DEV).bfloat16(), act=act)  # the other terms of a sum are 0 z
    close(y, ref, 2.0 ** -16 * ref.abs() * (1 + x.double().abs().clamp(max=128)) + 1e-36, act)


@pytest.mark.parametrize("act", ACTS)
def test_every_slope(cuda_lib, act):
    z = finite()[None]
    ref = slope(z.double(), act)
    got = qk.linear_fused_backward(torch.ones_like(z), None, None, z, act, need_dbias=True)[2]
    close(got[None], ref, 2.0 ** -16 * (1 + z.double().abs().clamp(max=128)), act, step=U)


@pytest.mark.parametrize("act", ACTS[1:])
def test_nan_stays(cuda_lib, act):
    z = torch.full((1, 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert torch.isnan(qk.linear_fused_backward(torch.ones_like(z), None, None, z, act, need_dbias=True)[2]).all()
    assert torch.isnan(qk.linear_fused(z, torch.eye(8, device=DEV).bfloat16(), act=act)).all()

"""Rows wider than 15 warps of two units a thread: four units a thread (bf16, forward calls), the element-wise kernels.

The limits of the kernels, per token of q and k together: 15360 elements (fp32, gradients, bf16 heads of 8-byte
chunks) or twice that (bf16 forward), less where q or k does not fill its last warp, and what shared memory holds.
"""
from __future__ import annotations

import pytest
import torch

import rmsnorm_qknorm_b200 as qk
import test_rotary_gpu as base

pytestmark = pytest.mark.gpu

# heads whose chunks lie in the row's order and in the units' own; parts of heads; q alone; rows that leave room for a
# single stage of shared memory; just below and above the limits
WIDTHS = [(128, 8, 128, 128), (256, 8, 64, 64), (120, 24, 128, 64), (200, 8, 96, 48), (150, 0, 128, 128), (220, 8, 128, 128),
          (112, 8, 128, 128), (240, 8, 128, 128), (192, 16, 80, 40)]
CASES = [(*w, torch.bfloat16) for w in WIDTHS] + [(*w, torch.float32) for w in ((128, 8, 128, 128), (112, 8, 128, 128))]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hk,D,r,dtype", CASES)
def test_wide_rows(cuda_lib, hq, hk, D, r, layout, dtype):
    base.test_rotary_parity(cuda_lib, hq, hk, D, r, layout, dtype)
    base.test_qknorm_rotary_parity(cuda_lib, hq, hk, D, r, layout, dtype, dtype)
    base.test_backward_parity(cuda_lib, hq, hk, D, r, layout, dtype, dtype)
    assert qk.load_library().qkn_check_device(None) == 0


@pytest.mark.parametrize("hq,hk,D,r", [(128, 8, 128, 0), (128, 8, 128, 128), (256, 8, 64, 64)])
def test_wide_rows_with_weights_of_another_type(cuda_lib, hq, hk, D, r):
    for a, w in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        base.test_qknorm_rotary_parity(cuda_lib, hq, hk, D, r, "half", a, w)
        base.test_backward_parity(cuda_lib, hq, hk, D, r, "half", a, w)


@pytest.mark.parametrize("hq,hk,D", [(128, 8, 128), (256, 8, 64), (220, 8, 128)])
def test_wide_rows_in_place_and_beside_others(cuda_lib, hq, hk, D):
    # columns of one buffer, more rows than the device has SMs several times over; the rest stays as it was
    T, dq, dk = 700, hq * D, hk * D
    s = base.dev(base.make(T, hq, hk, D, D, torch.bfloat16, seed=8))
    buf = torch.full((T, dq + 2 * dk + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    q, k = buf[:, :dq], buf[:, dq + 8: dq + 8 + dk]
    for norm in (False, True):
        rest = (s["pos"], s["freq"], D)
        call = (lambda a, b, **o: qk.qknorm_rotary(a, b, s["wq"], s["wk"], *rest, **o)) if norm else (
            lambda a, b, **o: qk.rotary_apply(a, b, *rest, **o))
        want = call(s["q"], s["k"])
        q.copy_(s["q"])
        k.copy_(s["k"])
        call(q, k, inplace=True)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        q.fill_(7.0)
        k.fill_(7.0)
        assert bool((buf == 7.0).all())
    assert qk.load_library().qkn_check_device(None) == 0

"""Weights of QK-Norm that are not finite: what does not depend on them keeps its bits.

k and its gradients do not depend on q's weights, nor q on k's; the weights' gradients (sum of g x inv) depend on no
weight at all; and of the forward results only the pairs change that hold such a weight.
"""
from __future__ import annotations

import pytest
import torch

import rmsnorm_qknorm_b200 as qk
from test_rotary_gpu import SHAPES, dev, make

pytestmark = pytest.mark.gpu

# beside the shapes of the parity tests: key rows of fewer units than their warps have places, in bf16 and fp32; heads
# whose units lie in their own order; q alone
WIDTHS = SHAPES + [(5, 4, 128, 128), (8, 3, 64, 64), (9, 1, 128, 128), (16, 1, 96, 96), (11, 0, 64, 64), (3, 1, 48, 32)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hk,D,r", WIDTHS)
def test_a_weight_that_is_not_finite_stays_in_its_tensor(cuda_lib, hq, hk, D, r, layout, dtype):
    for T in (1, 37):
        s = dev(make(T, hq, hk, D, r, dtype, seed=T + D + 3))

        def call():
            a = (s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], D)
            return (*qk.qknorm_rotary(*a, layout=layout),
                    *qk.qknorm_rotary_backward(s["gq"], s["gk"], *a, layout=layout))

        want = call()
        for which in (0, 1) if hk else (0,):
            w = s["wq" if which == 0 else "wk"]
            n = min(8, r // 2)  # the first chunk's weights, every second one infinite
            keep = w[:n].clone()
            w[:n:2], w[1:n:2] = float("inf"), float("nan")
            got = call()
            w[:n] = keep
            for i, name in ((0, "q"), (1, "k"), (2, "dq"), (3, "dk"), (4, "dwq"), (5, "dwk")):
                if want[i] is not None and (i >= 4 or i % 2 != which):
                    assert torch.equal(got[i], want[i]), f"{name} T={T} with weights of {'qk'[which]}"
            touched = torch.zeros(want[which].shape[1], dtype=torch.bool)
            for i in range(n):
                touched[i] = True
                touched[(i + r // 2 if i < r // 2 else i - r // 2) if layout == "half" else i ^ 1] = True
            rest = ~touched.to(got[which].device)
            assert torch.equal(got[which][:, rest], want[which][:, rest])

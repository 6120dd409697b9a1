"""Every kernel, tile and split that the linear layer's rules choose between, by the names and grids of the launches.

Which sizes reach which kernel follows from cost estimates and the device's number of SMs; the parity tests' sizes were
chosen for 148.  Here each of their products is traced, so that a combination that none of them reaches any more fails.
"""
from __future__ import annotations

import json
import re

import pytest
import torch

import rmsnorm_qknorm_b200 as qk
import test_linear_gpu as base

pytestmark = pytest.mark.gpu

# split over the pairs of a cluster: forward 128 columns in 4; dx 128 in 4, 256 in 2 and 4; dW 128 in 3, 256 in 2 and 4
FORWARD = [(272, 848, 11208), (3748, 8, 3048)]
BACKWARD = [(3797, 2344, 8), (69, 4720, 6656), (65, 5872, 3728), (1563, 4784, 8), (3936, 72, 7512), (6432, 72, 3320)]


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_forward_parity(cuda_lib, M, N, K, act):
    base.test_forward_parity(cuda_lib, M, N, K, act)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_backward_parity(cuda_lib, M, N, K, act):
    base.test_backward_parity(cuda_lib, M, N, K, act)


def launches(call, path):
    """(kernel, template arguments, blocks) of the products that a call launches."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        call()
        torch.cuda.synchronize()
    prof.export_chrome_trace(path)
    with open(path) as f:
        events = json.load(f)["traceEvents"]
    seen = []
    for e in sorted((e for e in events if e.get("cat") == "kernel"), key=lambda e: e["ts"]):
        m = re.search(r"linear_(rows|pair|split)_kernel<([^>]*)>", e["name"])
        if m:
            g = e["args"]["grid"]
            seen.append((m[1], [int({"true": 1, "false": 0}.get(a, a)) for a in m[2].replace(" ", "").split(",")], g[0] * g[1]))
    return seen


def label(launch, rows, cols):
    """The kernel, its tile's size and, split over pairs, their number."""
    kernel, args, blocks = launch
    if kernel == "rows":
        return kernel, args[0]
    tile = args[2]
    if kernel == "pair":
        return kernel, tile
    return kernel, tile, blocks // (2 * -(-rows // 256) * -(-cols // tile))


def test_the_sizes_reach_every_kernel(cuda_lib, tmp_path):
    if torch.cuda.get_device_properties(0).multi_processor_count != 148:
        pytest.skip("the sizes were chosen for 148 SMs")
    # (of calls with an activation; the rule takes them apart from plain ones)
    reached = {"forward": set(), "dx": set(), "dW": set()}
    sizes = base.SIZES + FORWARD + BACKWARD
    calls, shapes = [], []
    for M, N, K in sizes:
        x, W, dy = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (N, K), (M, N)))

        def call(x=x, W=W, dy=dy):
            qk.linear_fused(x, W, act="relu")
            qk.linear_fused_backward(dy, x, W)

        calls.append(call)
        shapes += [("forward", M, N), ("dx", M, K), ("dW", N, K)]
    seen = launches(lambda: [c() for c in calls], str(tmp_path / "trace.json"))
    if not seen:
        pytest.skip("the profiler gives no kernel trace here")
    assert len(seen) == len(shapes)
    for (what, rows, cols), launch in zip(shapes, seen):
        reached[what].add(label(launch, rows, cols))
    splits = {("split", 128, p) for p in (2, 3, 4)} | {("split", 256, p) for p in (2, 3, 4)}
    rows16 = {("rows", t) for t in (16, 32, 64, 128)}
    assert reached["forward"] == splits | rows16 | {("pair", t) for t in (128, 192, 256)}
    assert reached["dx"] == splits | rows16 | {("pair", t) for t in (128, 256)}
    assert reached["dW"] == splits | {("rows", t) for t in (64, 128)} | {("pair", t) for t in (128, 256)}

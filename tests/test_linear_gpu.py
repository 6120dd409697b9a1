"""GPU parity of linear_fused and linear_fused_backward.

The reference is fp64 on the exact bf16 inputs; the bounds count roundings
(u = 2^-24; half a step of bf16 is finfo.eps / 2 = 2^-8 relative to a value):

* a product of K terms accumulated in fp32 in any order: off by at most
  K u sum |x w| (the products of bf16 values are exact in fp32; tensor cores
  may truncate instead of rounding when they align terms: one more factor 2);
* z = r * p + b: 2 u of its parts; an activation has slope at most 1.13, its
  own fp32 evaluation is good to 2^-17 of its result (exp) plus 2^-17 |z|;
* y = act + residual: one more u; each result is rounded once to bf16;
* dz is rounded to bf16 for the products: half a step of each factor.
"""
from __future__ import annotations

import math

import pytest
import torch

import rmsnorm_qknorm_b200 as qk

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
H = torch.finfo(torch.bfloat16).eps / 2
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def value(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def close(got, ref, err, what, step=H):
    off = (got.double() - ref).abs() - (err + step * (ref.abs() + err) + 1e-30)
    assert not torch.isnan(got).any(), f"{what}: NaN"
    assert float(off.max()) <= 0, f"{what}: beyond the bound by {float(off.max()):.3e}"


def normal(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def check_forward(x, W, bias, act, res, inv, y, z, what=""):
    xd, wd = x.double(), W.double()
    p, size = xd @ wd.t(), xd.abs() @ wd.abs().t()
    K = x.shape[1]
    err = 2 * K * U * size
    if inv is not None:
        p, err = p * inv.double()[:, None], err * inv.double().abs()[:, None]
    b = bias.double() if bias is not None else torch.zeros(W.shape[0], device=DEV, dtype=torch.float64)
    ze = err + 2 * U * (p.abs() + b.abs())
    zr = p + b
    if z is not None:
        close(z, zr, ze, what + " preact")
    yr = value(zr, act)
    ye = 1.13 * ze + (0 if act == "none" else 2.0 ** -17 * (yr.abs() * (1 + zr.abs())))
    if res is not None:
        yr = yr + res.double()
        ye = ye + 2 * U * yr.abs()
    close(y, yr, ye, what + " y")


# From a single token to several tiles; widths of less than a tile, one tile and ragged ones.
SIZES = [(1, 64, 64), (1, 264, 1000), (2, 8, 8), (3, 128, 72), (17, 520, 136), (64, 256, 512), (100, 1032, 264),
         (128, 128, 128), (129, 264, 1000), (256, 256, 256), (257, 520, 64), (700, 776, 200), (1029, 2056, 1000),
         (1500, 4104, 1600)]
# One for each kernel and tile that the sizes choose between on 148 SMs: of the forward product the
# kernel for few rows with 32, 64 and 128 tokens per tile, then the pair kernel with 128 and 256
# columns (16 tokens are taken by the small ones above); the same of dx; of dW; the forward product
# with 192 columns; split over the pairs of a cluster, 128 columns and 2 and 3 pairs, 256 and 2, 3 and 4, the
# same of dx and dW.
SIZES += [(65, 3728, 8), (333, 2704, 8), (500, 3464, 8), (333, 3344, 264), (1000, 3464, 72),
          (65, 8, 3736), (500, 8, 1696), (65, 712, 3080), (333, 264, 3336), (1000, 72, 3816),
          (100, 8, 8), (1000, 3224, 8), (200, 3272, 264), (65, 3528, 912),
          (257, 4848, 1000), (129, 3736, 1000), (129, 2384, 2312), (65, 6336, 3952),
          (129, 4776, 1984), (65, 3736, 5264),
          (520, 800, 1216), (264, 2152, 2096), (136, 2256, 2360), (1001, 1632, 424), (3001, 280, 2096), (3001, 1216, 336)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward_parity(cuda_lib, M, N, K, act):
    x, W = normal(M, K, seed=M + K), normal(N, K, seed=N, scale=K ** -0.5)
    check_forward(x, W, None, act, None, None, qk.linear_fused(x, W, act=act), None, "bare")
    for dt in (torch.bfloat16, torch.float32):
        b, res = normal(N, seed=7, dtype=dt), normal(M, N, seed=8)
        inv = torch.rand(M, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV) + 0.5
        z = torch.full((M, N), 9.0, dtype=torch.bfloat16, device=DEV)
        y = qk.linear_fused(x, W, b, act, res, inv_rms=inv, preact_out=z)
        check_forward(x, W, b, act, res, inv, y, z, f"all {dt}")
    y = qk.linear_fused(x, W, b, act)
    check_forward(x, W, b, act, None, None, y, None, "bias")
    y = qk.linear_fused(x, W, None, act, res)
    check_forward(x, W, None, act, res, None, y, None, "residual")
    assert qk.load_library().qkn_check_device(None) == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_backward_parity(cuda_lib, M, N, K, act):
    x, W = normal(M, K, seed=M + K), normal(N, K, seed=N, scale=K ** -0.5)
    z, dy = normal(M, N, seed=3, scale=2.0), normal(M, N, seed=4)
    dx, dW, db = qk.linear_fused_backward(dy, x, W, z if act != "none" else None, act, need_dbias=True)
    s = slope(z.double(), act)
    dz = dy.double() * s
    # slopes in fp32: 2^-17 of each of their parts, which are at most 1 + |z|
    de = 0 if act == "none" else dy.double().abs() * 2.0 ** -17 * (1 + z.double().abs())
    dze = torch.zeros_like(dz) if act == "none" else de + H * (dz.abs() + de)
    wd, xd = W.double(), x.double()
    close(dx, dz @ wd, dze @ wd.abs() + 2 * N * U * (dz.abs() @ wd.abs()), "dx")
    close(dW, dz.t() @ xd, dze.t() @ xd.abs() + 2 * M * U * (dz.abs().t() @ xd.abs()), "dW")
    close(db, dz.sum(0), (de + M * U * dz.abs()).sum(0) if act != "none" else (M * U * dz.abs()).sum(0), "dbias", step=U)
    again = qk.linear_fused_backward(dy, x, W, z, act, need_dbias=True)
    assert all(torch.equal(a, b) for a, b in zip((dx, dW, db), again))
    # one at a time
    assert torch.equal(qk.linear_fused_backward(dy, None, W, z, act)[0], dx)
    only = qk.linear_fused_backward(dy, x, None, z, act)
    assert only[0] is None and only[2] is None and torch.equal(only[1], dW)
    assert torch.equal(qk.linear_fused_backward(dy, None, None, z, act, need_dbias=True)[2], db)
    assert qk.load_library().qkn_check_device(None) == 0


def test_gradients_against_differences(cuda_lib):
    # central differences of sum(y c) of the fp64 formula at bf16 inputs; z comes from the kernel
    M, N, K = 5, 16, 8
    x, W, b, c = normal(M, K, seed=1), normal(N, K, seed=2), normal(N, seed=3), normal(M, N, seed=4)
    z = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    for act in ACTS[2:]:
        qk.linear_fused(x, W, b, act, preact_out=z)
        dx, dW, db = qk.linear_fused_backward(c, x, W, z, act, need_dbias=True)
        h = 1e-6

        def total(xx, ww, bb):
            return float((value(xx @ ww.t() + bb, act) * c.double()).sum())

        args = [x.double(), W.double(), b.double()]
        for i, got in enumerate((dx, dW, db)):
            num = torch.zeros_like(args[i]).view(-1)
            for j in range(num.numel()):
                e = torch.zeros_like(num)
                e[j] = h
                hi = [a + (e.view_as(a) if k == i else 0) for k, a in enumerate(args)]
                lo = [a - (e.view_as(a) if k == i else 0) for k, a in enumerate(args)]
                num[j] = (total(*hi) - total(*lo)) / (2 * h)
            # z is rounded to bf16 (2^-8 of at most 8, slopes change by at most 0.8 per unit of z), dz and the
            # result to bf16; sums of at most 16 products of size up to 3
            size = {0: c.double().abs() @ W.double().abs(), 1: c.double().abs().t() @ x.double().abs(),
                    2: c.double().abs().sum(0)}[i].view(-1)
            zmax = float(z.float().abs().max())
            assert bool(((got.double().view(-1) - num).abs() <= size * (H * zmax * 0.8 + 2 * 1.13 * H) + 1e-6).all()), (act, i)


@pytest.mark.parametrize("M", [1, 9, 200, 300])
def test_pitches_guards_and_in_place_residual(cuda_lib, M):
    N, K = 136, 72
    xb, wb = normal(M, K + 24, seed=1), normal(N, K + 8, seed=2, scale=0.1)
    x, W = xb[:, 8: 8 + K], wb[:, :K]
    buf = torch.full((M + 2, N + 32), 7.0, dtype=torch.bfloat16, device=DEV)
    zb = buf.clone()
    y, z = buf[1: M + 1, 16: 16 + N], zb[1: M + 1, 8: 8 + N]
    res = normal(M, N, seed=3)
    y.copy_(res)
    out = qk.linear_fused(x, W, None, "gelu", y, preact_out=z, out=y)
    assert out.data_ptr() == y.data_ptr()
    check_forward(x.contiguous(), W.contiguous(), None, "gelu", res, None, y, z, "views")
    # the same bits as contiguous buffers
    assert torch.equal(qk.linear_fused(x.contiguous(), W.contiguous(), None, "gelu", res), y)
    y.fill_(7.0)
    z.fill_(7.0)
    assert bool((buf == 7.0).all()) and bool((zb == 7.0).all())
    dyb = normal(M, N + 8, seed=4)
    dxb = torch.full((M, K + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    dwb = torch.full((N, K + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    zz = normal(M, N, seed=5)
    dx, dW, _ = qk.linear_fused_backward(dyb[:, :N], x, W, zz, "silu", dx_out=dxb[:, 8: 8 + K], dW_out=dwb[:, 8: 8 + K])
    a = qk.linear_fused_backward(dyb[:, :N].contiguous(), x.contiguous(), W.contiguous(), zz, "silu")
    assert torch.equal(dx, a[0]) and torch.equal(dW, a[1])
    for t in (dxb, dwb):
        t[:, 8: 8 + K] = 7.0
        assert bool((t == 7.0).all())


def test_rows_do_not_depend_on_the_batch_and_nan_stays(cuda_lib):
    N, K = 264, 512
    x, W = normal(300, K, seed=1), normal(N, K, seed=2, scale=0.05)
    y = qk.linear_fused(x, W, act="silu")
    bad = x.clone()
    bad[5, 7], bad[200, 0] = float("nan"), float("inf")
    b = qk.linear_fused(bad, W, act="silu")
    keep = torch.ones(300, dtype=torch.bool, device=DEV)
    keep[5] = keep[200] = False
    assert torch.equal(b[keep], y[keep]) and torch.isnan(b[5]).all()
    big = torch.tensor([[-3e4, -100.0, -20.0, -0.0, 0.0, 20.0, 100.0, 3e4]], device=DEV).bfloat16()
    eye = torch.eye(8, device=DEV).bfloat16()
    for act in ACTS:  # saturated arguments stay finite
        got = qk.linear_fused(big, eye, act=act)
        close(got, value(big.double(), act), torch.full((1, 8), 1e-30, device=DEV, dtype=torch.float64)
              + 2.0 ** -16 * value(big.double(), act).abs() * (1 + big.double().abs().clamp(max=128)), act)
        g = qk.linear_fused_backward(torch.ones_like(big), None, None, big, act, need_dbias=True)[2]
        close(g[None], slope(big.double(), act), 2.0 ** -16 * (1 + big.double().abs().clamp(max=128)), act, step=U)


def test_empty_batch(cuda_lib):
    x, W = normal(4, 64)[:0], normal(32, 64)
    assert qk.linear_fused(x, W).shape == (0, 32)
    dx, dW, db = qk.linear_fused_backward(normal(4, 32)[:0], x, W, need_dbias=True)
    assert dx.shape == (0, 64) and bool((dW == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("M", [4, 600])
def test_other_stream_graph_and_two_calls_at_once(cuda_lib, M):
    N, K = 520, 256
    x, W, b, res = normal(M, K, seed=1), normal(N, K, seed=2, scale=0.1), normal(N, seed=3), normal(M, N, seed=4)
    z, dy = normal(M, N, seed=5), normal(M, N, seed=6)
    want = qk.linear_fused(x, W, b, "gelu", res)
    wg = qk.linear_fused_backward(dy, x, W, z, "gelu", need_dbias=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(qk.linear_fused(x, W, b, "gelu", res, stream=s),
             *qk.linear_fused_backward(dy, x, W, z, "gelu", need_dbias=True, stream=s)) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, (want, *wg)))
    # two graphs that share a workspace, replayed one after the other with new inputs
    ws = torch.empty(qk.linear_fused_backward_workspace_bytes(M, N, K, "gelu"), dtype=torch.uint8, device=DEV)
    got, graphs = [], []
    for _ in range(2):
        o = [torch.empty_like(t) for t in (want, *wg)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qk.linear_fused(x, W, b, "gelu", res, out=o[0])
            qk.linear_fused_backward(dy, x, W, z, "gelu", dx_out=o[1], dW_out=o[2], dbias_out=o[3], workspace=ws)
        got.append(o)
        graphs.append(g)
    x.copy_(normal(M, K, seed=11))
    dy.copy_(normal(M, N, seed=12))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    fresh = (qk.linear_fused(x, W, b, "gelu", res), *qk.linear_fused_backward(dy, x, W, z, "gelu", need_dbias=True))
    for o in got:
        assert all(torch.equal(p, q) for p, q in zip(o, fresh))
    assert qk.load_library().qkn_check_device(None) == 0


def test_refusals_of_the_binding(cuda_lib):
    x, W, b, z = normal(4, 64), normal(32, 64), normal(32), normal(4, 32)
    for kw in (dict(x=x[:1].expand(4, -1)), dict(W=W[:, :32]), dict(bias=b[:16]), dict(act="tanh"), dict(residual=z[:1]),
               dict(residual=z[:1].expand(4, -1)), dict(residual=z.float()), dict(inv_rms=torch.ones(4, device=DEV).bfloat16()),
               dict(preact_out=z[:, :16]), dict(out=z[:3]), dict(W=W.cpu()), dict(x=x.t()), dict(out=x[:, :32])):
        a = dict(x=x, W=W) | kw
        with pytest.raises((ValueError, TypeError)):
            qk.linear_fused(a.pop("x"), a.pop("W"), **a)
    with pytest.raises(qk.QKNormError, match="SHAPE"):
        qk.linear_fused(x[:, :60].contiguous(), W[:, :60].contiguous())
    with pytest.raises(qk.QKNormError, match="ALIGN"):
        qk.linear_fused(normal(4, 72)[:, 1:65], W)
    for args, kw in (((z, x, W, None, "gelu"), {}), ((z, None, None), {}), ((z, x[:3], W), {}),
                     ((z, x, W), dict(dx_out=z)), ((z, x, None), dict(dx_out=x))):
        with pytest.raises(ValueError):
            qk.linear_fused_backward(*args, **kw)


@pytest.mark.parametrize("M,N,K", [(9, 136, 72), (333, 3344, 264)])  # the kernel for few rows, the pair kernel
def test_offsets_beyond_32_bits(cuda_lib, M, N, K):
    # every operand but W is a block of columns of one buffer whose rows lie so far apart that the
    # last ones pass 2^32 bytes; the same bits as contiguous operands
    pitch = (2 ** 31 // (M - 1) + 64) // 8 * 8
    buf = torch.empty(M, pitch, dtype=torch.bfloat16, device=DEV)
    x, dx = buf[:, :K], buf[:, 512: 512 + K]
    dy, y, z = (buf[:, c: c + N] for c in (1024, 5120, 9216))
    assert M * pitch * 2 > 2 ** 32
    W = normal(N, K, seed=2)
    x.copy_(normal(M, K, seed=1))
    dy.copy_(normal(M, N, seed=3))
    y.copy_(dy)
    qk.linear_fused(x, W, None, "gelu", y, preact_out=z, out=y)
    _, dW, _ = qk.linear_fused_backward(dy, x, W, z, "gelu", dx_out=dx)
    xc, dyc, zc = x.contiguous(), dy.contiguous(), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    assert torch.equal(qk.linear_fused(xc, W, None, "gelu", dyc, preact_out=zc), y) and torch.equal(z, zc)
    gx, gW, _ = qk.linear_fused_backward(dyc, xc, W, zc, "gelu")
    assert torch.equal(dx, gx) and torch.equal(dW, gW)


def test_a_long_sum_of_ones_is_exact(cuda_lib):
    # 2^24 rows: every partial sum of ones is an integer that fp32 holds, in whatever order
    M = 2 ** 24
    dy, x = (torch.ones(M, 8, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _, dW, db = qk.linear_fused_backward(dy, x, None, need_dbias=True)
    assert bool((dW == M).all()) and bool((db == M).all())


def test_results_of_columns_beside_the_inputs(cuda_lib):
    # columns of one buffer under two pitches (every row of one, every other row of the other)
    M, N, K = 6, 64, 64
    buf = normal(2 * M, 256, seed=1)
    x, W = buf[::2, :K], normal(N, K, seed=2, scale=0.1)
    ref = qk.linear_fused(x.contiguous(), W)
    y = buf[:M, 128: 128 + N]
    assert torch.equal(qk.linear_fused(x, W, out=y), ref)
    with pytest.raises(qk.QKNormError, match="shares memory"):
        qk.linear_fused(x, W, out=buf[:M, 56: 56 + N])


@pytest.mark.parametrize("M,N,K", [(129, 3736, 1000), (300, 4096, 8192)])  # split over two pairs, 128 and 256 columns
def test_split_products_on_views(cuda_lib, M, N, K):
    x, W, b, res = normal(M, K, seed=1), normal(N, K, seed=2, scale=K ** -0.5), normal(N, seed=3), normal(M, N, seed=4)
    inv = torch.rand(M, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV) + 0.5
    z = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    want = qk.linear_fused(x, W, b, "silu", res, inv_rms=inv, preact_out=z)
    buf = torch.full((M + 2, 2 * N + 48), 7.0, dtype=torch.bfloat16, device=DEV)
    y, zv = buf[1: M + 1, 8: 8 + N], buf[1: M + 1, N + 24: 2 * N + 24]
    y.copy_(res)
    xv = torch.empty(M, K + 8, dtype=torch.bfloat16, device=DEV)[:, :K].copy_(x)
    for _ in range(3):  # the same bits every time
        qk.linear_fused(xv, W, b, "silu", y, inv_rms=inv, preact_out=zv, out=y)
        assert torch.equal(y, want) and torch.equal(zv, z)
        y.copy_(res)
    y.fill_(7.0)
    zv.fill_(7.0)
    assert bool((buf == 7.0).all())
    bad = x.clone()
    bad[M - 2] = float("nan")
    got = qk.linear_fused(bad, W, b, "silu", res, inv_rms=inv)
    assert torch.isnan(got[M - 2]).all() and torch.equal(got[:M - 2], want[:M - 2]) and torch.equal(got[M - 1], want[M - 1])

"""GPU parity of rotary_apply, qknorm_rotary and qknorm_rotary_backward.

The reference is a plain fp64 restatement (angles in extended precision), the
bounds count roundings.  With u = 2^-24 and per pair (a, b) of fp32 values:

* cos and sin: the reduced angle is rounded once in units of half a turn
  (pi u absolute at most), the function is good to 2 ulp, the product with
  mscale rounds once: at most (pi + 2 * 2 + 1) u < 9 u absolute, times mscale;
  the fp64 angle itself is off by at most 2^-51 of its size;
* a c - b s: two products and a sum, 2 u of |a| + |b| more: 11 u in all;
* an fp32 sum of n terms of one sign in any order is off by at most n u
  relative (per row n = d); x * inv * w rounds inv (rsqrt: 2 ulp, half of the
  sum's error, a division, a sum: 4 u) and two products;
* the result is rounded once, half a step of its type.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import rmsnorm_qknorm_b200 as qk

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def turn(positions, freq, mscale):
    """(cos, sin, error) per token and pair, fp64."""
    theta = np.asarray(positions, dtype=np.longdouble)[:, None] * freq.astype(np.longdouble)[None, :]
    return ((np.cos(theta) * mscale).astype(np.float64), (np.sin(theta) * mscale).astype(np.float64),
            mscale * (9 * U + np.abs(theta).astype(np.float64) * 2.0 ** -51))


def pair_index(heads, D, r, layout):
    """Element indices (a, b) of every pair [heads, r/2]."""
    i = np.arange(r // 2)
    a, b = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
    base = np.arange(heads)[:, None] * D
    return base + a, base + b


def rotate(x, err, positions, freq, mscale, D, layout, sign):
    """Rotation of fp64 rows x known to +-err; returns (y, error before the final rounding)."""
    y, e = x.copy(), err.copy()
    r = 2 * len(freq)
    if r == 0:
        return y, e
    a, b = pair_index(x.shape[1] // D, D, r, layout)
    c, s, ce = (v[:, None, :] for v in turn(positions, freq, mscale))
    s = sign * s
    xa, xb, ea, eb = x[:, a], x[:, b], err[:, a], err[:, b]
    y[:, a], y[:, b] = xa * c - xb * s, xb * c + xa * s
    size = np.abs(xa) + np.abs(xb)
    pair_err = size * (ce + 2 * U * mscale) + (ea + eb) * mscale
    e[:, a], e[:, b] = pair_err, pair_err
    return y, e


def norm(x, w, eps):
    d = x.shape[1]
    inv = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    rel = (d / 2 + 4) * U
    y = x * inv * w
    return y, np.abs(y) * (rel + 2 * U)


def norm_back(x, w, g, ge, eps):
    """(dx, error), (dw, error) for the gradient g +- ge of RMSNorm's result."""
    T, d = x.shape
    inv = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    rel = (d / 2 + 4) * U
    P = (w * g * x).sum(1, keepdims=True)
    Pe = (np.abs(w * x) * (ge + np.abs(g) * (d + 3) * U)).sum(1, keepdims=True)
    dx = inv * (w * g - x * inv ** 2 * P / d)
    dxe = inv * np.abs(w) * (ge + np.abs(g) * (rel + 3 * U)) + np.abs(x) * inv ** 3 / d * (Pe + np.abs(P) * (3 * rel + 6 * U))
    dw = (g * x * inv).sum(0)
    dwe = (np.abs(x * inv) * (ge + np.abs(g) * (rel + 3 * U + T * U))).sum(0)
    return dx, dxe, dw, dwe


def close(got, ref, err, dtype, what):
    g = f64(got)
    bound = err + half_step(dtype) * (np.abs(ref) + err) + 1e-30
    off = np.abs(g - ref) - bound
    assert not np.isnan(g).any(), f"{what}: NaN"
    assert off.max(initial=-1.0) <= 0, f"{what}: off by {np.abs(g - ref).flat[off.argmax()]:.3e}, bound {bound.flat[off.argmax()]:.3e}"


def make(T, hq, hk, D, r, dtype, seed=0, span=5000, pos_dtype=torch.int64, scaling=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = dict(q=n(T, hq * D).to(dtype), k=n(T, hk * D).to(dtype) if hk else None,
             gq=n(T, hq * D).to(dtype), gk=n(T, hk * D).to(dtype) if hk else None,
             wq=(1 + 0.1 * n(hq * D)).to(dtype), wk=(1 + 0.1 * n(hk * D)).to(dtype) if hk else None,
             pos=torch.randint(0, span, (T,), generator=g).to(pos_dtype))
    s["freq"], s["m"] = (qk.rotary_inv_freq(r, scaling=scaling, factor=4.0, original=2048, device="cpu") if r
                         else (None, 1.0))
    return s


def dev(s):
    return {n: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for n, v in s.items()}


def freqs(s):
    return s["freq"].numpy() if s["freq"] is not None else np.zeros(0)


# (heads of q, of k, head width, rotated elements): whole heads, part of them, heads
# without a multiple of 16 bytes (element-wise kernel), one head, rows of several widths
SHAPES = [(2, 1, 64, 64), (5, 2, 128, 64), (32, 8, 128, 128), (3, 3, 80, 32), (1, 0, 256, 256), (4, 1, 96, 48),
          (3, 2, 20, 12), (2, 2, 6, 2), (40, 40, 128, 128), (7, 1, 24, 16), (1, 1, 16, 16), (3, 0, 32, 16)]
# in bf16 16-byte rows of which only 8-byte pieces divide the heads and their rotated parts
SHAPES += [(3, 2, 80, 40), (20, 4, 80, 40), (64, 64, 80, 40), (4, 2, 20, 8), (2, 2, 12, 8), (1, 1, 40, 24)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hk,D,r", SHAPES)
def test_rotary_parity(cuda_lib, hq, hk, D, r, layout, dtype):
    for T, inverse, pd in ((1, False, torch.int64), (37, True, torch.int32), (700, False, torch.int64)):
        s = make(T, hq, hk, D, r, dtype, seed=T + D, pos_dtype=pd)
        d = dev(s)
        qo, ko = qk.rotary_apply(d["q"], d["k"], d["pos"], d["freq"], D, layout=layout, mscale=1.25, inverse=inverse)
        for n, got in (("q", qo), ("k", ko)):
            if got is None:
                continue
            x = f64(s[n])
            ref, err = rotate(x, np.zeros_like(x), s["pos"].numpy(), freqs(s), 1.25, D, layout, -1 if inverse else 1)
            close(got, ref, err, dtype, f"{n} T={T}")
            if r < D:  # the rest of a head is copied bit for bit
                rest = np.arange(x.shape[1]) % D >= r
                assert np.array_equal(f64(got)[:, rest], x[:, rest])


@pytest.mark.parametrize("dtype,wdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                          (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hk,D,r", SHAPES + [(5, 2, 128, 0), (3, 1, 20, 0)])
def test_qknorm_rotary_parity(cuda_lib, hq, hk, D, r, layout, dtype, wdtype):
    for T in (1, 300):
        s = make(T, hq, hk, D, r, dtype, seed=T + D + 1)
        s["wq"] = s["wq"].to(wdtype)
        s["wk"] = s["wk"].to(wdtype) if hk else None
        d = dev(s)
        qo, ko = qk.qknorm_rotary(d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D, 1e-5, layout=layout,
                                  mscale=0.75)
        for n, got in (("q", qo), ("k", ko)):
            if got is not None:
                y, e = norm(f64(s[n]), f64(s["w" + n]), 1e-5)
                ref, err = rotate(y, e, s["pos"].numpy(), freqs(s), 0.75, D, layout, 1)
                close(got, ref, err, dtype, f"{n} T={T}")


@pytest.mark.parametrize("dtype,wdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                          (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("hq,hk,D,r", SHAPES + [(5, 2, 128, 0), (3, 1, 20, 0)])
def test_backward_parity(cuda_lib, hq, hk, D, r, layout, dtype, wdtype):
    for T in (1, 300):
        s = make(T, hq, hk, D, r, dtype, seed=T + D + 2)
        s["wq"] = s["wq"].to(wdtype)
        s["wk"] = s["wk"].to(wdtype) if hk else None
        d = dev(s)
        got = qk.qknorm_rotary_backward(d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D,
                                        1e-5, layout=layout, mscale=0.75)
        for n, dx, dw in (("q", got[0], got[2]), ("k", got[1], got[3])):
            if dx is None:
                assert n == "k" and dw is None and not hk
                continue
            g = f64(s["g" + n])
            g, ge = rotate(g, np.zeros_like(g), s["pos"].numpy(), freqs(s), 0.75, D, layout, -1)
            ref, err, dwr, dwe = norm_back(f64(s[n]), f64(s["w" + n]), g, ge, 1e-5)
            close(dx, ref, err, dtype, f"d{n} T={T}")
            close(dw, dwr, dwe, torch.float32, f"dw{n} T={T}")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_backward_against_differences(cuda_lib, layout):
    # central differences of sum(y * c) in fp64 through the plain form; the kernel's gradients in fp32
    T, hq, D, r, eps = 3, 2, 16, 8, 1e-5
    s = make(T, hq, 0, D, r, torch.float32, seed=5)
    d = dev(s)
    dq, _, dwq, _ = qk.qknorm_rotary_backward(d["gq"], None, d["q"], None, d["wq"], None, d["pos"], d["freq"], D, eps,
                                              layout=layout)
    c = f64(s["gq"])

    def value(x, w):
        return (rotate(norm(x, w, eps)[0], np.zeros_like(x), s["pos"].numpy(), freqs(s), 1.0, D, layout, 1)[0] * c).sum()

    x, w, h = f64(s["q"]), f64(s["wq"]), 1e-6
    num = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        e = np.zeros_like(x)
        e[i] = h
        num[i] = (value(x + e, w) - value(x - e, w)) / (2 * h)
    numw = np.array([(value(x, w + h * e) - value(x, w - h * e)) / (2 * h) for e in np.eye(len(w))])
    # differences: truncation of order h^2 and rounding 1e-15 * |value| / h, both below 1e-7; kernel below 1e-5
    assert np.abs(f64(dq) - num).max() < 2e-5 and np.abs(f64(dwq) - numw).max() < 2e-5


def test_far_and_negative_positions(cuda_lib):
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 7, -(2 ** 24) - 1, 2 ** 31 + 5, 10 ** 8], dtype=torch.int64)
    for scaling in (None, "linear", "ntk", "yarn"):
        s = make(len(pos), 4, 2, 64, 64, torch.float32, seed=3, scaling=scaling)
        s["pos"] = pos
        d = dev(s)
        qo, ko = qk.rotary_apply(d["q"], d["k"], d["pos"], d["freq"], 64, mscale=s["m"])
        for n, got in (("q", qo), ("k", ko)):
            x = f64(s[n])
            ref, err = rotate(x, np.zeros_like(x), pos.numpy(), freqs(s), s["m"], 64, "half", 1)
            close(got, ref, err, torch.float32, f"{n} {scaling}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,shift", [(128, 0), (128, 1), (40, 0)])  # shift 1: rows off the 16-byte grid
def test_views_in_place_and_guards(cuda_lib, dtype, D, shift):
    # q | k | v of one fused buffer, rotated (and normalised) in place: v and the
    # columns before and behind stay as they were, and the bits are those of the
    # out-of-place call on the same views
    T, hq, hk, r = 67, 4, 2, 32
    dq, dk, wide = hq * D, hk * D, (hq + 2 * hk) * D + 16
    g = torch.Generator().manual_seed(11)
    buf = torch.randn(T, wide, generator=g).to(dtype).to(DEV)
    s = make(T, hq, hk, D, r, dtype, seed=12)
    d = dev(s)
    qv, kv = buf[:, shift: shift + dq], buf[:, shift + dq: shift + dq + dk]
    for call in (lambda **o: qk.rotary_apply(qv, kv, d["pos"], d["freq"], D, **o),
                 lambda **o: qk.qknorm_rotary(qv, kv, d["wq"], d["wk"], d["pos"], d["freq"], D, **o)):
        before = buf.clone()
        qo, ko = call()
        outer = torch.full((T, wide), 7.0, dtype=dtype, device=DEV)
        call(q_out=outer[:, shift: shift + dq], k_out=outer[:, shift + dq: shift + dq + dk])
        assert torch.equal(outer[:, shift: shift + dq], qo) and torch.equal(outer[:, shift + dq: shift + dq + dk], ko)
        outer[:, shift: shift + dq + dk] = 7.0
        assert bool((outer == 7.0).all())
        assert torch.equal(buf, before)
        call(inplace=True)
        assert torch.equal(qv, qo) and torch.equal(kv, ko)
        assert torch.equal(buf[:, shift + dq + dk:], before[:, shift + dq + dk:])
        assert torch.equal(buf[:, :shift], before[:, :shift])


def test_rows_are_independent_and_repeatable(cuda_lib):
    # a row's bits depend neither on the rows beside it nor on the run; NaN and Inf stay in their row,
    # and without a norm in their pair
    T, hq, hk, D = 513, 8, 4, 64
    s = make(T, hq, hk, D, 64, torch.bfloat16, seed=21)
    d = dev(s)
    a = qk.qknorm_rotary(d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D)
    b = qk.qknorm_rotary(d["q"][200:201], d["k"][200:201], d["wq"], d["wk"], d["pos"][200:201], d["freq"], D)
    assert torch.equal(a[0][200:201], b[0]) and torch.equal(a[1][200:201], b[1])
    alone, _ = qk.qknorm_rotary(d["q"], None, d["wq"], None, d["pos"], d["freq"], D)
    ref, err = norm(f64(s["q"]), f64(s["wq"]), 1e-6)
    ref, err = rotate(ref, err, s["pos"].numpy(), freqs(s), 1.0, D, "half", 1)
    close(alone, ref, err, torch.bfloat16, "q alone")
    g1 = qk.qknorm_rotary_backward(d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D)
    g2 = qk.qknorm_rotary_backward(d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D)
    assert all(torch.equal(x, y) for x, y in zip(g1, g2))
    bad = d["q"].clone()
    bad[7, 3], bad[9, 70] = float("nan"), float("inf")
    n, kn = qk.qknorm_rotary(bad, d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D)
    assert torch.isnan(n[7]).all() and torch.equal(kn, a[1])
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[7] = keep[9] = False
    assert torch.equal(n[keep], a[0][keep])
    r0, _ = qk.rotary_apply(d["q"], None, d["pos"], d["freq"], D)
    r1, _ = qk.rotary_apply(bad, None, d["pos"], d["freq"], D)
    differ = (r0 != r1).nonzero().tolist()
    assert {tuple(i) for i in differ} <= {(7, 3), (7, 35), (9, 70), (9, 102)}


def test_zero_rows_and_zero_tokens(cuda_lib):
    s = make(4, 2, 1, 64, 64, torch.bfloat16, seed=1)
    d = dev(s)
    z = torch.zeros_like(d["q"])
    o, _ = qk.qknorm_rotary(z, None, d["wq"], None, d["pos"], d["freq"], 64)
    assert bool((o == 0).all())
    e = {n: (v[:0] if n in ("q", "k", "gq", "gk", "pos") else v) for n, v in d.items()}
    assert qk.rotary_apply(e["q"], e["k"], e["pos"], e["freq"], 64)[0].shape == (0, 128)
    assert qk.qknorm_rotary(e["q"], e["k"], e["wq"], e["wk"], e["pos"], e["freq"], 64)[1].shape == (0, 64)
    dw = torch.full((128,), 5.0, device=DEV)
    got = qk.qknorm_rotary_backward(e["gq"], e["gk"], e["q"], e["k"], e["wq"], e["wk"], e["pos"], e["freq"], 64, dwq_out=dw)
    assert got[0].shape == (0, 128) and bool((dw == 0).all()) and bool((got[3] == 0).all())


@pytest.mark.parametrize("T", [1, 5, 8, 13, 2500])
def test_narrow_rows_share_a_warp(cuda_lib, T):
    # rows of a few chunks go several tokens to a warp; the last ones may be missing, and with
    # eps = 0 nothing of the places without a token may reach the weights' gradients
    for hq, hk, D, r, dtype in ((1, 1, 16, 16, torch.bfloat16), (1, 1, 64, 64, torch.bfloat16), (2, 1, 64, 32, torch.float32),
                                (1, 1, 128, 128, torch.bfloat16), (1, 0, 64, 64, torch.float32)):
        s = make(T, hq, hk, D, r, dtype, seed=T)
        d = dev(s)
        args = (d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], D, 0.0)
        fwd = qk.qknorm_rotary(*args)
        got = qk.qknorm_rotary_backward(d["gq"], d["gk"], *args)
        for n, o, dx, dw in (("q", fwd[0], got[0], got[2]), ("k", fwd[1], got[1], got[3])):
            if o is None:
                continue
            y, e = norm(f64(s[n]), f64(s["w" + n]), 0.0)
            ref, err = rotate(y, e, s["pos"].numpy(), freqs(s), 1.0, D, "half", 1)
            close(o, ref, err, dtype, n)
            g = f64(s["g" + n])
            g, ge = rotate(g, np.zeros_like(g), s["pos"].numpy(), freqs(s), 1.0, D, "half", -1)
            ref, err, dwr, dwe = norm_back(f64(s[n]), f64(s["w" + n]), g, ge, 0.0)
            close(dx, ref, err, dtype, "d" + n)
            close(dw, dwr, dwe, torch.float32, "dw" + n)


def test_norm_without_rotation_is_qknorm(cuda_lib):
    # the same statistic in another order of summation: bf16 results at most one step apart
    s = make(300, 8, 4, 128, 0, torch.bfloat16, seed=31)
    d = dev(s)
    a = qk.qknorm_rotary(d["q"], d["k"], d["wq"], d["wk"], None, None, 0)
    b = qk.qknorm_fused(d["q"], d["k"], d["wq"], d["wk"])
    for x, y in zip(a, b):
        assert float(((x.float() - y.float()).abs() / y.float().abs().clamp(min=1e-30)).max()) <= 2.0 ** -7


def test_other_stream_graph_and_workspace(cuda_lib):
    s = make(400, 8, 2, 128, 128, torch.bfloat16, seed=41)
    d = dev(s)
    args = (d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], 128)
    want = qk.qknorm_rotary_backward(*args)
    fwd = qk.qknorm_rotary(*args[2:])
    need = qk.qknorm_rotary_backward_workspace_bytes(400, 1024, 256)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for got in (qk.qknorm_rotary_backward(*args, workspace=ws),
                qk.qknorm_rotary_backward(*args, stream=side),
                qk.qknorm_rotary_backward(*args, stream=side.cuda_stream, workspace=ws)):
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    # captured and replayed with other inputs in the same buffers
    outs = [torch.empty_like(t) for t in (*want, *fwd)]

    def both():
        qk.qknorm_rotary_backward(*args, dq_out=outs[0], dk_out=outs[1], dwq_out=outs[2], dwk_out=outs[3], workspace=ws)
        qk.qknorm_rotary(*args[2:], q_out=outs[4], k_out=outs[5])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in (42, 43):
        new = dev(make(400, 8, 2, 128, 128, torch.bfloat16, seed=seed))
        for n in ("q", "k", "gq", "gk", "pos"):
            d[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        seen = [t.clone() for t in outs]
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(seen, outs))


def test_long_batch_keeps_every_row(cuda_lib):
    # more rows than any grid holds at once, rows of one head: every row against the rotation of a repeated block
    T, D = 200003, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    base = torch.randn(1000, D, generator=g, device=DEV).bfloat16()
    q = base.repeat(201, 1)[:T].contiguous()
    pos = torch.arange(1000, device=DEV).repeat(201)[:T].contiguous()
    freq, _ = qk.rotary_inv_freq(D)
    w = torch.ones(D, device=DEV).bfloat16()
    one = qk.qknorm_rotary(base, None, w, None, pos[:1000].contiguous(), freq, D)[0]
    assert torch.equal(qk.qknorm_rotary(q, None, w, None, pos, freq, D)[0], one.repeat(201, 1)[:T])
    one = qk.rotary_apply(base, None, pos[:1000].contiguous(), freq, D)[0]
    assert torch.equal(qk.rotary_apply(q, None, pos, freq, D)[0], one.repeat(201, 1)[:T])


def test_rows_as_wide_as_the_norm_takes(cuda_lib):
    # wider than shared memory: the element-wise kernel serves them
    s = make(3, 300, 1, 256, 256, torch.float32, seed=51)
    d = dev(s)
    qo, ko = qk.qknorm_rotary(d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], 256)
    got = qk.qknorm_rotary_backward(d["gq"], d["gk"], d["q"], d["k"], d["wq"], d["wk"], d["pos"], d["freq"], 256)
    y, e = norm(f64(s["q"]), f64(s["wq"]), 1e-6)
    ref, err = rotate(y, e, s["pos"].numpy(), freqs(s), 1.0, 256, "half", 1)
    close(qo, ref, err, torch.float32, "q")
    g = f64(s["gq"])
    g, ge = rotate(g, np.zeros_like(g), s["pos"].numpy(), freqs(s), 1.0, 256, "half", -1)
    ref, err, dwr, dwe = norm_back(f64(s["q"]), f64(s["wq"]), g, ge, 1e-6)
    close(got[0], ref, err, torch.float32, "dq")
    close(got[2], dwr, dwe, torch.float32, "dwq")


def test_refusals_of_the_binding(cuda_lib):
    s = make(4, 2, 1, 64, 64, torch.bfloat16, seed=1)
    d = dev(s)
    q, k, pos, f = d["q"], d["k"], d["pos"], d["freq"]
    for bad in (dict(q=q[:1].expand(4, -1)), dict(k=k[:3]), dict(k=k.float()), dict(pos=pos.float()), dict(pos=pos[:3]),
                dict(f=f.float()), dict(f=None), dict(layout="both"), dict(q_out=q[:, :64]), dict(q=q.t()),
                dict(q_out=q[:1].expand(4, -1)), dict(inplace=True, q_out=torch.empty_like(q)), dict(f=f.cpu()), dict(pos=pos.cpu())):
        a = dict(q=q, k=k, pos=pos, f=f) | bad
        with pytest.raises((ValueError, TypeError)):
            qk.rotary_apply(a.pop("q"), a.pop("k"), a.pop("pos"), a.pop("f"), 64, **a)
    with pytest.raises(qk.QKNormError, match="SHAPE"):
        qk.rotary_apply(q, k, pos, f, 48)
    back = (d["gq"], d["gk"], q, k, d["wq"], d["wk"], pos, f, 64)
    for kw in (dict(dq_out=d["gq"]), dict(dq_out=q), dict(dwq_out=torch.empty(128, device=DEV).bfloat16())):
        with pytest.raises(ValueError):
            qk.qknorm_rotary_backward(*back, **kw)
    with pytest.raises(qk.QKNormError, match="workspace"):
        qk.qknorm_rotary_backward(*back, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="gk"):
        qk.qknorm_rotary_backward(d["gq"], None, *back[2:])


@pytest.mark.parametrize("shift", [0, 1])  # the unit kernel, the element-wise kernels
def test_offsets_beyond_32_bits(cuda_lib, shift):
    # the rows of every operand are columns of one buffer, so far apart that the last ones pass 2^32 bytes
    T, hq, hk, D = 9, 4, 2, 64
    s = make(T, hq, hk, D, 64, torch.bfloat16, seed=5)
    d = dev(s)
    pitch = 2 ** 28 + 8 + shift
    buf = torch.empty(T, pitch, dtype=torch.bfloat16, device=DEV)
    at = lambda c, w: buf[:, c: c + w]  # noqa: E731
    v = {n: at(512 * i, d[n].shape[1]) for i, n in enumerate(("q", "k", "gq", "gk"))}
    o = [at(512 * i, w * D) for i, w in ((4, hq), (5, hk), (6, hq), (7, hk))]
    for n, t in v.items():
        t.copy_(d[n])
    # the same alignment in a small buffer: the same kernel, the same bits
    small = {n: torch.empty(T, 512 + shift, dtype=torch.bfloat16, device=DEV)[:, : t.shape[1]].copy_(t) for n, t in v.items()}
    rest = (d["pos"], d["freq"], D)
    for call in (lambda a, **kw: qk.rotary_apply(a["q"], a["k"], *rest, **kw),
                 lambda a, **kw: qk.qknorm_rotary(a["q"], a["k"], d["wq"], d["wk"], *rest, **kw)):
        got, want = call(v, q_out=o[0], k_out=o[1]), call(small)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = qk.qknorm_rotary_backward(small["gq"], small["gk"], small["q"], small["k"], d["wq"], d["wk"], *rest)
    got = qk.qknorm_rotary_backward(v["gq"], v["gk"], v["q"], v["k"], d["wq"], d["wk"], *rest, dq_out=o[2], dk_out=o[3])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_one_tensor_twice_is_refused_in_place(cuda_lib):
    s = dev(make(5, 2, 2, 64, 64, torch.bfloat16, seed=6))
    with pytest.raises(qk.QKNormError, match="shares memory"):
        qk.rotary_apply(s["q"], s["q"], s["pos"], s["freq"], 64, inplace=True)
    a, b = qk.rotary_apply(s["q"], s["q"], s["pos"], s["freq"], 64)
    assert torch.equal(a, b)

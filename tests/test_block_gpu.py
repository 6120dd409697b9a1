"""The calls around QK-Norm run together, as a transformer block uses them: serving (a prefill and
single tokens, with the norms folded) and the gradients of a training step, against fp64 torch.

Bounds: every call rounds its result to bf16 once, half a step (finfo.eps / 2 = 2^-8 of the value)
at most; along the longest chain of a test n results are rounded one after the other and the calls
between them do not enlarge a relative error of a whole tensor (products with random weights, norms,
sums with the residual stream), so the relative Frobenius error stays below n 2^-8.
"""
from __future__ import annotations

import math

import pytest
import torch

import rmsnorm_qknorm_b200 as qk

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = torch.finfo(torch.bfloat16).eps / 2
HQ, HK, D = 4, 2, 64
DM, DF = 256, 520


def normal(*shape, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).bfloat16()


def weights():
    nqkv = (HQ + 2 * HK) * D
    w = dict(w1=1 + normal(DM, seed=1, scale=0.1), w2=1 + normal(DM, seed=2, scale=0.1),
             Wqkv=normal(DM, nqkv, seed=3, scale=DM ** -0.5), wq=1 + normal(HQ * D, seed=4, scale=0.1),
             wk=1 + normal(HK * D, seed=5, scale=0.1), Wo=normal(DM, HQ * D, seed=6, scale=(HQ * D) ** -0.5),
             Wup=normal(DM, DF, seed=7, scale=DM ** -0.5), bup=normal(DF, seed=8, scale=0.1),
             Wdown=normal(DM, DF, seed=9, scale=DF ** -0.5))
    return w


def rel(a, ref):
    return float((a.double() - ref).norm() / ref.norm())


def rms(x, w, eps):
    return x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w


def turn(x, pos, freq, m):
    v = x.view(x.shape[0], -1, D)
    a, b = v[..., : D // 2], v[..., D // 2:]
    t = pos.double()[:, None, None] * freq
    c, s = t.cos() * m, t.sin() * m
    return torch.cat((a * c - b * s, b * c + a * s), -1).view_as(x)


def attend(q, k, v, causal_from):
    """q [T, HQ D] over k, v [S, HK D]; query t sees keys 0 .. causal_from + t."""
    T, S = q.shape[0], k.shape[0]
    q, k, v = (t.view(t.shape[0], -1, D).transpose(0, 1) for t in (q, k, v))
    k, v = k.repeat_interleave(HQ // HK, 0), v.repeat_interleave(HQ // HK, 0)
    s = q @ k.transpose(1, 2) / math.sqrt(D)
    mask = torch.arange(S, device=DEV)[None] <= causal_from + torch.arange(T, device=DEV)[:, None]
    return (s.masked_fill(~mask, -math.inf).softmax(-1) @ v).transpose(0, 1).reshape(T, HQ * D)


class Served:
    """A block with its weights laid out once and a cache of keys and values."""

    def __init__(self, w, fused):
        self.w, self.fused = w, fused
        self.Wqkv = qk.flashnorm_fold_weights(w["w1"], w["Wqkv"])
        self.Wup = qk.flashnorm_fold_weights(w["w2"], w["Wup"])
        self.freq, self.m = qk.rotary_inv_freq(D, scaling="yarn", factor=2.0, original=64)
        self.k = torch.zeros(128, HK * D, device=DEV, dtype=torch.bfloat16)
        self.v = torch.zeros_like(self.k)

    def __call__(self, x, pos):
        w, nq, nk, n0 = self.w, HQ * D, HK * D, int(pos[0])
        if self.fused:
            qkv = qk.qkv_proj_qknorm(x, self.Wqkv, nq, nk, nk, w["wq"], w["wk"])
            q, k = qk.rotary_apply(qkv[:, :nq], qkv[:, nq: nq + nk], pos, self.freq, D, mscale=self.m, inplace=True)
        else:
            qkv = qk.flashnorm_proj(x, self.Wqkv)
            q, k = qk.qknorm_rotary(qkv[:, :nq], qkv[:, nq: nq + nk], w["wq"], w["wk"], pos, self.freq, D,
                                    mscale=self.m, inplace=True)
        n1 = n0 + x.shape[0]
        self.k[n0:n1], self.v[n0:n1] = k, qkv[:, nq + nk:]
        a = attend(q.float(), self.k[:n1].float(), self.v[:n1].float(), n0).bfloat16()
        x1 = qk.linear_fused(a, w["Wo"], residual=x)
        h = qk.linear_fused(x1, self.Wup, w["bup"], "gelu", inv_rms=qk.flashnorm_inv_rms(x1))
        return qk.linear_fused(h, w["Wdown"], residual=x1, out=x1)  # the stream updated in place


def block64(x, w, freq, m):
    w = {n: t.double() for n, t in w.items()}
    nq, nk = HQ * D, HK * D
    qkv = rms(x, w["w1"], 1e-6) @ w["Wqkv"]
    pos = torch.arange(x.shape[0], device=DEV)
    q = turn(rms(qkv[:, :nq], w["wq"], 1e-6), pos, freq, m)
    k = turn(rms(qkv[:, nq: nq + nk], w["wk"], 1e-6), pos, freq, m)
    x1 = x + attend(q, k, qkv[:, nq + nk:], 0) @ w["Wo"].t()
    z = rms(x1, w["w2"], 1e-6) @ w["Wup"] + w["bup"]
    return x1 + (0.5 * z * torch.special.erfc(-z / math.sqrt(2))) @ w["Wdown"].t()


@pytest.mark.parametrize("fused", [False, True])
def test_serving_block(cuda_lib, fused):
    # a prefill of 67 tokens, then single tokens through the same block
    w = weights()
    x = normal(72, DM, seed=20)
    served = Served(w, fused)
    ref = block64(x.double(), w, served.freq, served.m)
    pos = torch.arange(72, device=DEV)
    parts = [served(x[:67].contiguous(), pos[:67])] + [served(x[i: i + 1], pos[i: i + 1]) for i in range(67, 72)]
    # rounded one after the other: W', qkv, q / k, (k, v in the cache: the same), attention, x1, W'up, h, x2
    for part, r in ((parts[0], ref[:67]), (torch.cat(parts[1:]), ref[67:])):
        assert rel(part, r) < 9 * HALF
    assert cuda_lib.load_library().qkn_check_device(None) == 0


@pytest.mark.parametrize("T", [1, 67, 300])
def test_training_step(cuda_lib, T):
    # x -> q, k -> QK-Norm + rotary -> (q with k repeated) -> linear with activation + residual
    w = weights()
    x, dy = normal(T, DM, seed=30), normal(T, DM, seed=31)
    Wq, Wk = normal(HQ * D, DM, seed=32, scale=DM ** -0.5), normal(HK * D, DM, seed=33, scale=DM ** -0.5)
    bo = normal(DM, seed=34, scale=0.2)
    pos = torch.arange(T, device=DEV) + 1000
    freq, m = qk.rotary_inv_freq(D)

    q, k = qk.linear_fused(x, Wq), qk.linear_fused(x, Wk)
    qr, kr = qk.qknorm_rotary(q, k, w["wq"], w["wk"], pos, freq, D)
    s = qr + kr.view(T, HK, D).repeat_interleave(HQ // HK, 1).reshape(T, -1)
    z = torch.empty(T, DM, device=DEV, dtype=torch.bfloat16)
    y = qk.linear_fused(s, w["Wo"], bo, "silu", x, preact_out=z)
    ds, dWo, dbo = qk.linear_fused_backward(dy, s, w["Wo"], z, "silu", need_dbias=True)
    dkr = ds.view(T, HK, HQ // HK, D).sum(2).reshape(T, -1)  # the key heads are shared
    dq, dk, dwq, dwk = qk.qknorm_rotary_backward(ds, dkr, q, k, w["wq"], w["wk"], pos, freq, D)
    dxq, dWq, _ = qk.linear_fused_backward(dq, x, Wq)
    dxk, dWk, _ = qk.linear_fused_backward(dk, x, Wk)
    dx = dxq + dxk + dy

    leaves = [t.double().requires_grad_() for t in (x, Wq, Wk, w["wq"], w["wk"], w["Wo"], bo)]
    X, Q, K, NQ, NK, O, B = leaves
    qd = turn(rms(X @ Q.t(), NQ, 1e-6), pos, freq, m)
    kd = turn(rms(X @ K.t(), NK, 1e-6), pos, freq, m)
    sd = qd + kd.view(T, HK, D).repeat_interleave(HQ // HK, 1).reshape(T, -1)
    zd = sd @ O.t() + B
    yd = zd * torch.sigmoid(zd) + X
    ref = torch.autograd.grad(yd, leaves, dy.double())
    # rounded one after the other: q, q turned, s, z (its slope's error: 0.5 per unit of z, z about 1), y: 5;
    # then dz, ds, dkr, dq, and the result: 10
    assert rel(y, yd.detach()) < 5 * HALF
    for name, got, r in zip(("dx", "dWq", "dWk", "dwq", "dwk", "dWo", "dbo"), (dx, dWq, dWk, dwq, dwk, dWo, dbo), ref):
        assert rel(got, r) < 10 * HALF, name
    assert cuda_lib.load_library().qkn_check_device(None) == 0


def test_decode_step_in_a_graph(cuda_lib):
    # one token's calls captured once and replayed on new inputs give the bits of the eager calls
    w = weights()
    Wup = qk.flashnorm_fold_weights(w["w2"], w["Wup"])
    freq, m = qk.rotary_inv_freq(D)
    x, qkv = normal(3, DM, seed=40), normal(3, (HQ + 2 * HK) * D, seed=41)
    pos = torch.tensor([5, 70, 9000], device=DEV)
    nq, nk = HQ * D, HK * D
    inv = torch.empty(3, device=DEV)
    h, x1 = torch.empty(3, DF, device=DEV, dtype=torch.bfloat16), torch.empty(3, DM, device=DEV, dtype=torch.bfloat16)
    q, k = torch.empty(3, nq, device=DEV, dtype=torch.bfloat16), torch.empty(3, nk, device=DEV, dtype=torch.bfloat16)

    def step():
        qk.qknorm_rotary(qkv[:, :nq], qkv[:, nq: nq + nk], w["wq"], w["wk"], pos, freq, D, q_out=q, k_out=k)
        qk.linear_fused(q, w["Wo"], residual=x, out=x1)
        qk.flashnorm_inv_rms(x1, out=inv)
        qk.linear_fused(x1, Wup, w["bup"], "gelu_tanh", inv_rms=inv, out=h)
        qk.linear_fused(h, w["Wdown"], residual=x1, out=x1)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (50, 60):
        x.copy_(normal(3, DM, seed=seed))
        qkv.copy_(normal(3, (HQ + 2 * HK) * D, seed=seed + 1))
        pos += 1
        step()
        want = [t.clone() for t in (q, k, h, x1)]
        for t in (q, k, h, x1, inv):
            t.fill_(3.0)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((q, k, h, x1), want))

"""The operators around QK-Norm in a transformer block, as cases to be measured.

Rotary positions on query and key rows, QK-Norm followed by rotary positions
(forward and gradients), and a matrix product with bias, activation and
residual in its epilogue (forward and gradients).  Each operator has a plain
form in elementary torch operations (``own`` false) and the call a user makes
of the library (``own`` true).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest batch of fp32 rows: a call whose latency counts
        dict(name="rotary_tiny_f32", op="rotary", T=64, hq=32, hk=32, D=128, r=128, layout="half",
             scaling="none", dtype="f32", inverse=False, span=4096),
        # a prefill of grouped-query rows with frequencies scaled for a longer context
        dict(name="rotary_prefill_gqa", op="rotary", T=16384, hq=40, hk=8, D=128, r=128, layout="half",
             scaling="yarn", dtype="bf16", inverse=False, span=131072),
        # gradient of rotary positions on part of each head, a ragged batch, far positions
        dict(name="rotary_gradient_partial", op="rotary", T=5003, hq=16, hk=4, D=80, r=32, layout="interleaved",
             scaling="linear", dtype="f32", inverse=True, span=1048576),
        # one decode step of a serving batch
        dict(name="qknorm_rotary_decode", op="qknorm_rotary", T=256, hq=40, hk=40, D=128, r=128, layout="half",
             scaling="none", dtype="bf16", span=131072),
        # a long context at once, the largest of the norm's workloads
        dict(name="qknorm_rotary_long", op="qknorm_rotary", T=131072, hq=32, hk=32, D=128, r=128, layout="half",
             scaling="none", dtype="bf16", span=131072),
        # gradients of a small model's rows in fp32, half of each head rotated, a ragged batch
        dict(name="qknorm_rotary_grad_narrow", op="qknorm_rotary_backward", T=1029, hq=8, hk=8, D=128, r=64,
             layout="interleaved", scaling="none", dtype="f32", span=4096),
        # gradients of a training batch of grouped-query rows
        dict(name="qknorm_rotary_grad_gqa", op="qknorm_rotary_backward", T=16384, hq=40, hk=8, D=128, r=128,
             layout="half", scaling="none", dtype="bf16", span=16384),
        # one token through an up projection: the weights are the traffic
        dict(name="linear_one_token", op="linear", M=1, K=4096, N=12288, act="gelu", bias="bf16", residual=False,
             scale=False, preact=False),
        # a decode batch through a down projection added to the residual stream
        dict(name="linear_decode_residual", op="linear", M=64, K=12288, N=4096, act="none", bias="none",
             residual=True, scale=False, preact=False),
        # ragged sizes with every part of the epilogue, rows scaled by a deferred norm
        dict(name="linear_ragged_all", op="linear", M=1029, K=1000, N=2056, act="silu", bias="f32", residual=True,
             scale=True, preact=False),
        # a prefill or training batch through an up projection, pre-activations kept for the gradients
        dict(name="linear_prefill_preact", op="linear", M=8192, K=4096, N=12288, act="gelu_tanh", bias="bf16",
             residual=False, scale=False, preact=True),
        # gradients of that projection
        dict(name="linear_grad", op="linear_backward", M=4096, K=4096, N=12288, act="gelu_tanh", bias="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "qknorm_rotary", "qknorm_rotary_backward", "linear", "linear", "linear_backward"])
    if op.startswith("linear"):
        while True:
            M = _log_uniform(rng, 1, 8192) if op == "linear" else _log_uniform(rng, 64, 4096)
            K = 8 * _log_uniform(rng, 8, 1536)
            N = 8 * _log_uniform(rng, 8, 1536)
            if M * K * N <= (8192 if op == "linear" else 4096) * 4096 * 12288:
                break
        c = dict(op=op, M=M, K=K, N=N, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                 bias=rng.choice(["none", "bf16", "f32"]))
        if op == "linear":
            c.update(residual=rng.random() < 0.5, scale=rng.random() < 0.3, preact=rng.random() < 0.3)
        return c
    D = rng.choice([64, 80, 96, 128, 128, 128, 256])
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = hk * rng.choice([1, 1, 2, 4, 5])
    while (hq + hk) * D > 10240:
        hq, hk = max(1, hq // 2), max(1, hk // 2)
    r = rng.choice([D, D, D // 2])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 131072 * 8192 * 2 // ((hq + hk) * D * (4 if dtype == "f32" else 2))
    if op == "qknorm_rotary_backward":
        most = most // 2
    c = dict(op=op, T=_log_uniform(rng, 1, min(131072, most)), hq=hq, hk=hk, D=D, r=r,
             layout=rng.choice(["half", "interleaved"]), dtype=dtype, span=rng.choice([4096, 131072, 1048576]),
             scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
    if op == "rotary":
        c["inverse"] = rng.random() < 0.3
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _frequencies(r, scaling):
    """The frequencies of r / 2 pairs in float64, and the factor on cos and sin."""
    base, factor, original = 10000.0, 8.0, 16384
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    inv = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling == "yarn":
        turns = [32.0, 1.0]  # pairs that turn more often than the first keep their frequency, less than the second are slowed
        low, high = [r * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in turns]
        low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
        ramp = ((torch.arange(r // 2, dtype=torch.float64, device="cuda") - low) / max(high - low, 0.001)).clamp(0, 1)
        return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return inv, 1.0


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"].startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        bf = torch.bfloat16

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        s["x"] = normal(M, K).to(bf)
        s["W"] = (normal(N, K) / math.sqrt(K)).to(bf)
        s["b"] = None if case["bias"] == "none" else (0.5 * normal(N)).to(DTYPES[case["bias"]])
        if case["op"] == "linear":
            s["res"] = normal(M, N).to(bf) if case["residual"] else None
            s["inv"] = 0.5 + torch.rand(M, generator=g, device="cuda") if case["scale"] else None
        else:
            s["z"] = normal(M, N).to(bf)
            s["dy"] = (normal(M, N) / math.sqrt(N)).to(bf)
        return s
    T, D = case["T"], case["D"]
    dq, dk, dt = case["hq"] * D, case["hk"] * D, DTYPES[case["dtype"]]
    s["q"] = torch.randn(T, dq, generator=g, device="cuda").to(dt)
    s["k"] = torch.randn(T, dk, generator=g, device="cuda").to(dt)
    # rows of packed sequences: runs of consecutive positions from random starts
    run_len = min(T, 512)
    starts = torch.randint(0, case["span"], (-(-T // run_len),), generator=g, device="cuda")
    s["pos"] = (starts[:, None] + torch.arange(run_len, device="cuda")).reshape(-1)[:T].contiguous()
    s["freq"], s["mscale"] = _frequencies(case["r"], case["scaling"])
    if case["op"] != "rotary":
        s["wq"] = (1 + 0.1 * torch.randn(dq, generator=g, device="cuda")).to(dt)
        s["wk"] = (1 + 0.1 * torch.randn(dk, generator=g, device="cuda")).to(dt)
        s["eps"] = 1e-6
    if case["op"] == "qknorm_rotary_backward":
        s["gq"] = torch.randn(T, dq, generator=g, device="cuda").to(dt)
        s["gk"] = torch.randn(T, dk, generator=g, device="cuda").to(dt)
    return s


# ---------------------------------------------------------------- plain forms

def _cos_sin(s):
    angle = s["pos"].double()[:, None, None] * s["freq"]  # 64 bits: positions reach far
    return (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()


def _rotate(x, s, cos, sin):
    """x [T, heads * D] in float32, the first r of each head rotated."""
    r = s["r"]
    v = x.view(x.shape[0], -1, s["D"])
    out = v.clone()
    if s["layout"] == "half":
        a, b = v[..., : r // 2], v[..., r // 2 : r]
        out[..., : r // 2] = a * cos - b * sin
        out[..., r // 2 : r] = b * cos + a * sin
    else:
        a, b = v[..., 0:r:2], v[..., 1:r:2]
        out[..., 0:r:2] = a * cos - b * sin
        out[..., 1:r:2] = b * cos + a * sin
    return out.view_as(x)


def _norm_back(x, w, g, eps):
    """Gradients of RMSNorm(x; w) for the gradient g of its result, all in float32."""
    inv = torch.rsqrt((x * x).mean(1, keepdim=True) + eps)
    h = x * inv
    wg = g * w
    return inv * (wg - h * (wg * h).mean(1, keepdim=True)), (g * h).sum(0)


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _activation(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * _sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = _sigmoid(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = _sigmoid(c * (z + 0.044715 * z * z * z))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain(s):
    op = s["op"]
    if op == "linear":
        z = s["x"].float() @ s["W"].float().t()
        if s["inv"] is not None:
            z = z * s["inv"][:, None]
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _activation(z, s["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        out = {"y": y.bfloat16()}
        if s["preact"]:
            out["preact"] = z.bfloat16()
        return out
    if op == "linear_backward":
        dz = s["dy"].float() * _slope(s["z"].float(), s["act"])
        out = {"dx": (dz @ s["W"].float()).bfloat16(), "dW": (dz.t() @ s["x"].float()).bfloat16()}
        if s["b"] is not None:
            out["dbias"] = dz.sum(0)
        return out
    cos, sin = _cos_sin(s)
    dt = s["q"].dtype
    if op == "rotary":
        sin = -sin if s["inverse"] else sin
        return {n: _rotate(s[n].float(), s, cos, sin).to(dt) for n in ("q", "k")}
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s["w" + n].float()
        if op == "qknorm_rotary":
            h = x * torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"]) * w
            out[n] = _rotate(h, s, cos, sin).to(dt)
        else:
            dx, dw = _norm_back(x, w, _rotate(s["g" + n].float(), s, cos, -sin), s["eps"])
            out["d" + n], out["dw" + n] = dx.to(dt), dw
    return out


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import rmsnorm_qknorm_b200 as qk
    op = s["op"]
    if op == "linear":
        z = torch.empty((s["M"], s["N"]), dtype=torch.bfloat16, device="cuda") if s["preact"] else None
        y = qk.linear_fused(s["x"], s["W"], s["b"], s["act"], s["res"], inv_rms=s["inv"], preact_out=z)
        return {"y": y, "preact": z} if s["preact"] else {"y": y}
    if op == "linear_backward":
        dx, dW, db = qk.linear_fused_backward(s["dy"], s["x"], s["W"], s["z"] if s["act"] != "none" else None,
                                              s["act"], need_dbias=s["b"] is not None)
        out = {"dx": dx, "dW": dW}
        if db is not None:
            out["dbias"] = db
        return out
    how = dict(layout=s["layout"], mscale=s["mscale"])
    if op == "rotary":
        q, k = qk.rotary_apply(s["q"], s["k"], s["pos"], s["freq"], s["D"], inverse=s["inverse"], **how)
        return {"q": q, "k": k}
    if op == "qknorm_rotary":
        q, k = qk.qknorm_rotary(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], s["D"], s["eps"], **how)
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = qk.qknorm_rotary_backward(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"],
                                                 s["freq"], s["D"], s["eps"], **how)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits, by another route

def _turned(x, s, back):
    """x [T, heads * D] (64 bits) with each pair, as a complex number, turned by its angle."""
    r, T = s["r"], x.shape[0]
    v = x.reshape(T, -1, s["D"]).clone()
    part = v[..., :r]
    pairs = part.reshape(T, v.shape[1], 2, r // 2).transpose(2, 3) if s["layout"] == "half" else \
        part.reshape(T, v.shape[1], r // 2, 2)
    angle = torch.outer(s["pos"].double(), s["freq"])
    turn = torch.polar(torch.full_like(angle, s["mscale"]), -angle if back else angle)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None, :])
    v[..., :r] = (z.transpose(2, 3) if s["layout"] == "half" else z).reshape(T, v.shape[1], r)
    return v.reshape(T, -1)


def _exact_rows(s, op, n):
    """Results of the row operators for tensor n (q or k), a block of rows at a time."""
    x, T = s[n], s["q"].shape[0]
    outs, dw = [], 0
    for i in range(0, T, 8192):
        b = dict(s, pos=s["pos"][i : i + 8192])
        v = x[i : i + 8192].double()
        if op == "rotary":
            outs.append(_turned(v, b, s["inverse"]))
            continue
        w = s["w" + n].double()
        rms = (v.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt()
        if op == "qknorm_rotary":
            outs.append(_turned(v / rms * w, b, False))
            continue
        g = _turned(s["g" + n][i : i + 8192].double(), b, True)
        inner = (g * w * v).sum(1, keepdim=True) / v.shape[1]
        outs.append(g * w / rms - v * inner / rms**3)
        dw = dw + (g * v / rms).sum(0)
    return torch.cat(outs), dw


def _exact_slope_and_value(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        return z * torch.special.expit(z), torch.special.expit(z) * (1 + z * torch.special.expit(-z))
    if act == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z**3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z**2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = torch.nn.functional.linear(s["x"].double(), s["W"].double())
        if s["inv"] is not None:
            z *= s["inv"].double()[:, None]
        if s["b"] is not None:
            z += s["b"].double()
        y = _exact_slope_and_value(z, s["act"])[0]
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y, "preact": z} if s["preact"] else {"y": y}
    if op == "linear_backward":
        dz = _exact_slope_and_value(s["z"].double(), s["act"])[1] * s["dy"].double()
        out = {"dx": dz @ s["W"].double(), "dW": torch.einsum("mn,mk->nk", dz, s["x"].double())}
        if s["b"] is not None:
            out["dbias"] = dz.sum(0)
        return out
    out = {}
    for n in ("q", "k"):
        v, dw = _exact_rows(s, op, n)
        if op == "qknorm_rotary_backward":
            out["d" + n], out["dw" + n] = v, dw
        else:
            out[n] = v
    return out


def work(case):
    if case["op"].startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        b = {"none": 0, "bf16": 2, "f32": 4}[case["bias"]] * N
        if case["op"] == "linear":
            moved = 2 * (M * K + N * K + M * N * (1 + case["residual"] + case["preact"])) + b + 4 * M * case["scale"]
            return {"bytes": moved, "flops": 2 * M * N * K}
        moved = 2 * (2 * M * K + 2 * N * K + M * N * (1 + (case["act"] != "none"))) + (4 * N if b else 0)
        return {"bytes": moved, "flops": 4 * M * N * K}
    es = 4 if case["dtype"] == "f32" else 2
    d = (case["hq"] + case["hk"]) * case["D"]
    T = case["T"]
    extra = 8 * T + 4 * case["r"]
    if case["op"] == "rotary":
        return {"bytes": 2 * T * d * es + extra, "flops": 3 * T * d}
    if case["op"] == "qknorm_rotary":
        return {"bytes": 2 * T * d * es + d * es + extra, "flops": 7 * T * d}
    return {"bytes": 3 * T * d * es + d * (es + 4) + extra, "flops": 14 * T * d}

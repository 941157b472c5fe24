"""Measured cases of the dense layers on MXFP4 weights and of their gradients.

With W the values of the prepared weights, Q(x) those of the quantized rows
and f an activation:

`linear`  z = Q(x) W^T + bias, y = f(z) + residual; gated: y = f(first half of
          z's columns) * second half + residual; z kept for the gradients or not
`pre`     dz from dy and the kept z, and the bias' gradient
`input`   dx = dz W
`weight`  dW = dz^T Q(x)

Each case runs either in its plain form (elementary torch operations in 32
bits, `own` false) or through the framework's entry points (`own` true), on
the same inputs.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "": 0}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ---- cases -------------------------------------------------------------------

def _linear(**c):
    return {**dict(op="linear", act="none", gated=False, bias="", residual=False, pre=False, y="bf16"), **c}


def listed():
    return [
        # the output projection of one token in decoding, with its bias and the residual stream: latency of one call
        _linear(name="linear_token", M=1, N=4096, K=4096, bias="bf16", residual=True),
        # a small decode batch, odd row count, a classic feed-forward up projection with f32 output
        _linear(name="linear_batch13", M=13, N=2112, K=7168, bias="f32", act="gelu", y="f32"),
        # a short prompt in training: the pre-activations kept, a row count next to a power of two
        _linear(name="linear_short257", M=257, N=4096, K=2048, bias="bf16", act="gelu_tanh", pre=True),
        # the down projection of a long prompt onto the residual stream
        _linear(name="linear_prompt", M=8192, N=4096, K=8192, bias="bf16", residual=True),
        # the gated up projection of one token in decoding
        _linear(name="gated_token", M=1, N=16384, K=4096, act="silu", gated=True),
        # the gated up projection of a training batch, with what its backward pass needs
        _linear(name="gated_batch", M=8192, N=16384, K=4096, act="silu", gated=True, pre=True),
        # backward of activation and bias: a short ragged batch, f32 gradient
        dict(name="pre_ragged771", op="pre", M=771, N=2112, act="gelu", gated=False, bias=True, dy="f32"),
        # ... and of a gated training batch
        dict(name="pre_batch", op="pre", M=8192, N=16384, act="silu", gated=True, bias=False, dy="bf16"),
        # the input's gradient for a few rows (tuning a prompt through frozen weights)
        dict(name="input_few", op="input", M=24, N=4096, K=4096, dx="bf16"),
        # ... and for the training batch of the gated projection
        dict(name="input_batch", op="input", M=8192, N=16384, K=4096, dx="bf16"),
        # the weights' gradient of a short ragged batch
        dict(name="weight_ragged771", op="weight", M=771, N=2112, K=704, dw="bf16"),
        # ... and of the training batch, into f32
        dict(name="weight_batch", op="weight", M=8192, N=16384, K=4096, dw="f32"),
    ]


def _log(rng, lo, hi):
    """An integer between lo and hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "pre", "input", "weight"])
    m = _log(rng, 1, 8192)
    act = rng.choice(ACTS)
    if op in ("linear", "gated"):
        gated = op == "gated"
        n = 32 * _log(rng, 4, 512) if gated else 16 * _log(rng, 4, 512)
        return _linear(M=m, N=n, K=32 * _log(rng, 4, 128 if gated else 256), act=act, gated=gated,
                       bias=rng.choice(["", "bf16", "f32"]), residual=rng.random() < 0.4, pre=rng.random() < 0.5,
                       y=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "pre":
        gated = rng.random() < 0.5
        return dict(op="pre", M=m, N=32 * _log(rng, 4, 512), act=act, gated=gated, bias=rng.random() < 0.6,
                    dy=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "input":
        return dict(op="input", M=m, N=16 * _log(rng, 4, 1024), K=32 * _log(rng, 4, 128),
                    dx=rng.choice(["bf16", "bf16", "f16", "f32"]))
    return dict(op="weight", M=m, N=16 * _log(rng, 4, 1024), K=32 * _log(rng, 4, 128),
                dw=rng.choice(["f32", "f32", "bf16", "f16"]))


def work(c):
    m, n = c["M"], c["N"]
    cols = n // 2 if c.get("gated") else n
    if c["op"] == "pre":
        z = 2 * m * n if c["gated"] or c["act"] != "none" else 0
        return {"bytes": m * cols * SIZE[c["dy"]] + z + 2 * m * n + (4 * n if c["bias"] else 0), "flops": 10 * m * n}
    k = c["K"]
    w = n * k * 17 // 32
    if c["op"] == "linear":
        b = 2 * m * k + w + m * cols * SIZE[c["y"]] * (2 if c["residual"] else 1) + (2 * m * n if c["pre"] else 0)
        return {"bytes": b + n * SIZE[c["bias"]], "flops": 2 * m * n * k}
    if c["op"] == "input":
        return {"bytes": 2 * m * n + w + m * k * SIZE[c["dx"]], "flops": 2 * m * n * k}
    return {"bytes": 2 * m * n + 2 * m * k + n * k * SIZE[c["dw"]], "flops": 2 * m * n * k}


# ---- the format, in elementary operations --------------------------------------

def _quantize(x):
    """f32 [..., K] -> (code of each element, 0..15; scale byte of each group of 32)."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    bits = g.abs().amax(-1).view(torch.int32)
    s = (((bits + 0x200000) >> 23) - 2).clamp(0, 254)
    v = g.abs() * torch.where(s < 254, (254 - s) << 23, 0x400000).to(torch.int32).view(torch.float32).unsqueeze(-1)
    lo = torch.round(v * 2)
    mid = torch.round(v) + 2
    hi = torch.clamp(torch.round(v * 0.5) + 4, max=7)
    code = torch.where(v < 2, lo, torch.where(v < 4, mid, hi)).to(torch.uint8)
    code = code | (torch.signbit(g).to(torch.uint8) << 3)
    return code.reshape(x.shape), s.to(torch.uint8)


def _values(code, s):
    """What codes and scale bytes stand for, in f32."""
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float32, device=code.device)
    v = t[code.int()].reshape(*s.shape, 32)
    p = torch.where(s > 0, s.int() << 23, 0x400000).to(torch.int32).view(torch.float32)
    return (v * p.unsqueeze(-1)).reshape(code.shape)


def _dequantize(q, s):
    return _values(torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1), s)


def _weights(gen, N, K):
    """A matrix as a checkpoint holds it (packed codes, scale bytes) and as the framework prepares it."""
    code, s = _quantize(torch.randn((N, K), generator=gen, device="cuda") * (1.5 / math.sqrt(K)))
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    bw = q.view(N // 16, 16, K // 32, 16).permute(0, 2, 1, 3).reshape(N // 16, K * 8).contiguous()
    G = K // 32
    rows, gp = -(-N // 256) * 256, -(-G // 8) * 8
    pad = torch.full((rows, gp), 127, dtype=torch.uint8, device="cuda")
    pad[:N, :G] = s
    # byte of (row, group) in its 32-row block: row bit 4, group bit 2, row bits 0-3, group bits 0-1, the rest of the group
    bs = pad.view(rows // 32, 2, 16, gp // 8, 2, 4).permute(0, 3, 5, 2, 4, 1).reshape(rows // 32, gp * 32)
    return q, s, bw, bs.contiguous()


# ---- inputs --------------------------------------------------------------------

def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2 + 1)

    def normal(rows, cols, scale, dtype):
        """Rows of unlike size, as activations and gradients are."""
        size = scale * torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda"))
        return (torch.randn((rows, cols), generator=gen, device="cuda") * size).to(dtype)

    st = dict(c)
    M, N = c["M"], c["N"]
    cols = N // 2 if c.get("gated") else N
    if c["op"] in ("linear", "input"):
        st["q"], st["s"], st["bw"], st["bs"] = _weights(gen, N, c["K"])
    if c["op"] in ("linear", "weight"):
        st["xv"] = normal(M, c["K"], 1.0, torch.bfloat16)
    if c["op"] in ("input", "weight"):
        st["dz"] = normal(M, N, 0.01, torch.bfloat16)
    if c["op"] == "linear":
        y = DT[c["y"]]
        st["b"] = (torch.randn(N, generator=gen, device="cuda") * 0.2).to(DT[c["bias"]]) if c["bias"] else None
        st["res"] = normal(M, cols, 1.0, y) if c["residual"] else None
        st["out"] = torch.empty((M, cols), dtype=y, device="cuda")
        st["z"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda") if c["pre"] else None
    elif c["op"] == "pre":
        st["dyv"] = normal(M, cols, 0.01, DT[c["dy"]])
        st["z"] = normal(M, N, 1.5, torch.bfloat16) if c["gated"] or c["act"] != "none" else None
        st["out"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "input":
        st["out"] = torch.empty((M, c["K"]), dtype=DT[c["dx"]], device="cuda")
    else:
        st["out"] = torch.empty((N, c["K"]), dtype=DT[c["dw"]], device="cuda")
    return st


# ---- the operators ---------------------------------------------------------------

def _act(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
    return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)


def _plain_linear(st):
    z = _values(*_quantize(st["xv"].float())) @ _dequantize(st["q"], st["s"]).t()
    if st["b"] is not None:
        z = z + st["b"].float()
    if st["gated"]:
        g, u = z.chunk(2, dim=-1)
        y = _act(st["act"], g) * u
    else:
        y = _act(st["act"], z)
    if st["res"] is not None:
        y = y + st["res"].float()
    y = y.to(DT[st["y"]])
    return (y, z.to(torch.bfloat16)) if st["pre"] else y


def _plain_pre(st):
    dy = st["dyv"].float()
    z = st["z"].float() if st["z"] is not None else dy
    if st["gated"]:
        g, u = z.chunk(2, dim=-1)
        dz = torch.cat([dy * u * _act_slope(st["act"], g), dy * _act(st["act"], g)], -1)
    else:
        dz = dy * _act_slope(st["act"], z)
    out = dz.to(torch.bfloat16)
    return (out, dz.double().sum(0).float()) if st["bias"] else out


def _plain_input(st):
    return (st["dz"].float() @ _dequantize(st["q"], st["s"])).to(DT[st["dx"]])


def _plain_weight(st):
    return (st["dz"].float().t() @ _values(*_quantize(st["xv"].float()))).to(DT[st["dw"]])


def run(st):
    op = st["op"]
    if not own:
        return {"linear": _plain_linear, "pre": _plain_pre, "input": _plain_input, "weight": _plain_weight}[op](st)
    import block_scaled_mxfp4_bf16_amd as mx
    if op == "linear":
        return mx.linear(st["xv"], st["bw"], st["bs"], st["N"], bias=st["b"], activation=st["act"], gated=st["gated"],
                         residual=st["res"], pre=st["z"], out=st["out"])
    if op == "pre":
        return mx.linear_grad_pre(st["dyv"], st["z"], activation=st["act"], gated=st["gated"], bias=st["bias"],
                                  out=st["out"])
    if op == "input":
        return mx.linear_grad_input(st["dz"], st["bw"], st["bs"], st["K"], out=st["out"])
    return mx.linear_grad_weight(st["dz"], st["xv"], out=st["out"])


# ---- the definitions in 64 bits ----------------------------------------------------

def _exact_weight(q, s):
    """f64 [N, K] from packed codes [N, K/2] and scale bytes [N, K/32]: sign * (1 + m/2) * 2^(e-1), or m/2 where e is 0."""
    n = torch.empty((q.shape[0], q.shape[1] * 2), dtype=torch.float64, device=q.device)
    n[:, 0::2] = (q % 16).double()
    n[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double()
    sign = torch.where(n >= 8, -1.0, 1.0).double()
    mag = torch.remainder(n, 8)
    ex, m = torch.floor(mag / 2), torch.remainder(mag, 2)
    v = torch.where(ex == 0, m / 2, (1 + m / 2) * torch.exp2(ex - 1)) * sign
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, dim=-1)


def _exact_activation(a):
    """f64 values that the rows stand for once quantized: the nearest of the grid, halfway cases to the even code."""
    x = a.double()
    top = x.abs().reshape(x.shape[0], -1, 32).amax(-1)
    ex = torch.frexp(top).exponent.double() - 1  # top = (1..2) * 2^ex
    ex = torch.where(top / torch.exp2(ex) >= 1.75, ex + 1, ex)
    scale = torch.exp2((ex - 2).clamp_min(-127)).repeat_interleave(32, dim=-1)
    scale = torch.where(top.repeat_interleave(32, dim=-1) == 0, 1.0, scale)
    v = x.abs() / scale
    grid = torch.tensor(E2M1, dtype=torch.float64, device=a.device)
    best = torch.zeros_like(v)
    for i in range(1, 8):
        half = (grid[i - 1] + grid[i]) / 2
        best = torch.where((v > half) | ((v == half) & (i % 2 == 0)), grid[i], best)
    return best * scale * torch.sign(x)


def _exact_act(act, z):
    """f(z) and f'(z) of each element, in f64."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), torch.heaviside(z, torch.zeros_like(z))
    if act == "silu":
        s = torch.special.expit(z)
        return z * s, s * (1 + z * torch.special.expit(-z))
    if act == "gelu":
        p = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3)))
    du = math.sqrt(2 / math.pi) * (1 + 0.134145 * z.square())
    return z / 2 * (1 + t), (1 + t) / 2 + z / 2 * (1 - t.square()) * du


def exact(c, seed):
    st = prepare(c, seed)
    n = c["N"] // 2
    if c["op"] == "linear":
        z = _exact_activation(st["xv"]).matmul(_exact_weight(st["q"], st["s"]).t())
        if c["bias"]:
            z += st["b"].double()
        y = _exact_act(c["act"], z[:, :n])[0] * z[:, n:] if c["gated"] else _exact_act(c["act"], z)[0]
        if c["residual"]:
            y = y + st["res"].double()
        return (y, z) if c["pre"] else y
    if c["op"] == "pre":
        dy = st["dyv"].double()
        if c["gated"]:
            f, slope = _exact_act(c["act"], st["z"][:, :n].double())
            dz = torch.empty((c["M"], c["N"]), dtype=torch.float64, device="cuda")
            dz[:, :n] = dy * st["z"][:, n:].double() * slope
            dz[:, n:] = dy * f
        else:
            dz = dy if st["z"] is None else dy * _exact_act(c["act"], st["z"].double())[1]
        return (dz, torch.ones(c["M"], dtype=torch.float64, device="cuda") @ dz) if c["bias"] else dz
    if c["op"] == "input":
        return st["dz"].double().matmul(_exact_weight(st["q"], st["s"]))
    return st["dz"].double().t().matmul(_exact_activation(st["xv"]))

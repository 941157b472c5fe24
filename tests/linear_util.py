"""64-bit forms of the dense layer and its gradients, and how far f32 arithmetic may be from them."""
import math

import numpy as np
import torch

import oracle
from tests.expert_util import HALF_STEP, SMALLEST, bf16_bits, dequant, dtype_of

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


class Matrix:
    """A weight matrix: prepared by the oracle on the device, and its f64 values."""

    def __init__(self, seed, N, K, scale=1.5, scales=None):
        r = np.random.default_rng(seed)
        q, s = oracle.quantize(bf16_bits(r.standard_normal((N, K)) * scale / math.sqrt(K)))
        if scales is not None:  # scale bytes of the caller's
            s = scales(r, s)
        self.N, self.K = N, K
        self.Bw = torch.from_numpy(oracle.preshuffle_b(q).reshape(N // 16, K * 8)).cuda()
        self.Bs = torch.from_numpy(oracle.shuffle_scales(s, N, K).reshape(-1, ((K // 32 + 7) // 8) * 32)).cuda()
        self.values = torch.from_numpy(dequant(q, s)).cuda()


def quantized(x):
    """f64 values of Q(x), by the oracle; x a bf16 tensor [M, K]."""
    if x.shape[0] == 0:
        return x.double()
    bits = np.ascontiguousarray(x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
    return torch.from_numpy(dequant(*oracle.quantize(bits))).cuda()


def rows(seed, M, cols, dtype="bf16", scale=1.0, pad=0):
    """Rows of unlike size; with `pad` a view into rows that are longer by it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    size = scale * torch.exp(0.5 * torch.randn((M, 1), generator=g, device="cuda"))
    t = (torch.randn((M, cols + pad), generator=g, device="cuda") * size).to(dtype_of(torch, dtype))
    return t[:, :cols]


def act(name, z):
    """f(z) and f'(z) in f64."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "silu":
        s = torch.special.expit(z)
        return z * s, s * (1 + z * torch.special.expit(-z))
    if name == "gelu":
        p = 0.5 * torch.erfc(z * -math.sqrt(0.5))
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    v = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)
    s = torch.special.expit(v)
    return z * s, s + z * s * torch.special.expit(-v) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def exponent(name, z):
    """Size of the argument of the exponential that the activation takes."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    if name == "silu":
        return z.abs()
    if name == "gelu":
        return z * z / 2
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3).abs()


def act_error(name, z):
    """How far f(z) and f'(z) may be off in f32, for the z that it is given.

    The argument v of the exponential has at most 4 roundings, 2^-22 |v|, which
    the exponential turns into a relative error; it, the reciprocal, the fitted
    tail of gelu (7e-8) and the products around them add less than 16 steps of
    2^-23.  What is below 2^-126 may be flushed: an s (or tail) that small takes
    z s with it in f, and s + z s v' in the slope.  In a slope z s (1 - s) v' the
    difference 1 - s is off by s (1 - s) times the exponential's error and by
    four steps of 2^-24 absolutely."""
    f, _ = act(name, z)
    if name in ("none", "relu"):
        return torch.zeros_like(z), torch.zeros_like(z)
    v = exponent(name, z).clamp_max(110)
    rel = (2 * v + 16) * 2.0**-23
    tiny = 2.0**-126 * (1 + z.abs())
    if name == "gelu":
        p, e = 0.5 * torch.erfc(z * -math.sqrt(0.5)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return rel * f.abs() + tiny, rel * (p + (z * e).abs()) + tiny
    s = torch.special.expit(z if name == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3))
    dv = torch.ones_like(z) if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    slope = rel * (s + (z * s * (1 - s) * dv).abs()) + (z * s * dv).abs() * (s * (1 - s) * rel + 2.0**-22)
    return rel * f.abs() + tiny, slope + 2.0**-126 * (1 + (z * dv).abs())


def rounded(ref, err, name):
    """The allowed difference of a value that is off by err and then rounded to the type."""
    return err + HALF_STEP[name] * (ref.abs() + err) + SMALLEST[name]


def sum_error(a, b):
    """An f32 sum of K products, in any order, each addition rounding or truncating: K 2^-23 sum |a b|."""
    return a.shape[1] * 2.0**-23 * (a.abs() @ b.abs().t())


def linear_limit(x, w, y_type, bias=None, activation="none", gated=False, residual=None):
    """(y, allowed difference), (z, allowed difference) of the layer on bf16 x and f64 weights [N, K]."""
    q = quantized(x)
    z, ez = q @ w.t(), sum_error(q, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0**-23 * (z.abs() + ez)
    g, eg = z, ez
    if gated:
        n = z.shape[1] // 2
        g, u, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
    f, _ = act(activation, g)
    own, _ = act_error(activation, g)
    y, ey = f, 1.13 * eg + own  # 1.13: no slope is larger
    if gated:
        y = f * u
        ey = ey * (u.abs() + eu) + f.abs() * eu + 2.0**-23 * y.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0**-23 * (y.abs() + ey)
    return (y, rounded(y, ey, y_type)), (z, rounded(z, ez, "bf16"))


def grad_pre_limit(dy, pre, activation="none", gated=False):
    """(dz, allowed difference), (dbias, allowed difference)."""
    dy = dy.double()
    if pre is None:
        dz, e = dy, torch.zeros_like(dy)
    else:
        z = pre.double()
        n = dy.shape[1]
        g = z[:, :n]
        f, slope = act(activation, g)
        ef, es = act_error(activation, g)
        if gated:
            u = z[:, n:]
            dz = torch.cat([dy * u * slope, dy * f], 1)
            e = torch.cat([(dy * u).abs() * es, dy.abs() * ef], 1) + 2.0**-22 * dz.abs()
        else:
            dz, e = dy * slope, dy.abs() * es + 2.0**-23 * (dy * slope).abs()
    db, edb = dz.sum(0), e.sum(0) + max(1, dz.shape[0]) * 2.0**-23 * dz.abs().sum(0)
    return (dz, rounded(dz, e, "bf16")), (db, edb + 2.0**-24 * db.abs() + 2.0**-149)


def product_limit(p, t, out_type):
    """(p @ t, allowed difference) for bf16 p [I, J] and f64 t [J, K]."""
    p = p.double()
    ref = p @ t
    return ref, rounded(ref, sum_error(p, t.t().contiguous()), out_type)


def assert_within(got, want, what):
    """|got - ref| <= limit; a reference that lies further past the largest number of got's type rounds to infinity."""
    ref, limit = want
    past = ref.abs() - limit > torch.finfo(got.dtype).max
    got = got.detach().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= limit) & ~(past & (got == ref.sign() * math.inf))
    if bool(bad.any()):
        at = bad.nonzero()[:4].tolist()
        raise AssertionError("%s: %d of %d outside; first %s" % (
            what, int(bad.sum()), bad.numel(),
            ["%s: %r, not %r +- %r" % (i, got[tuple(i)].item(), ref[tuple(i)].item(), limit[tuple(i)].item()) for i in at]))

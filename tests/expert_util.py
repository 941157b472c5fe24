"""Plain 64-bit forms of the expert operators and the inputs of their tests."""
import numpy as np

import oracle

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])

# Half a step of each output type, relative to the value, and the size below
# which a type's steps stop shrinking.
HALF_STEP = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}
SMALLEST = {"bf16": 2.0**-133, "f16": 2.0**-24, "f32": 2.0**-149}


def dtype_of(torch, name):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def bf16_bits(x):
    """f32 array -> bf16 bits, nearest even (finite values)."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def dequant(q, s):
    """f64 values of packed codes [..., K/2] and raw scale bytes [..., K/32]."""
    code = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=-1)


class Weights:
    """E matrices: prepared by the oracle on the device, and their f64 values."""

    def __init__(self, torch, seed, E, N, K, scale=1.0):
        r = np.random.default_rng(seed)
        qs, ss, self.values = [], [], []
        for _ in range(E):
            q, s = oracle.quantize(bf16_bits(r.standard_normal((N, K)) * scale / np.sqrt(K)))
            qs.append(oracle.preshuffle_b(q).reshape(N // 16, K * 8))
            ss.append(oracle.shuffle_scales(s, N, K).reshape(-1, ((K // 32 + 7) // 8) * 32))
            self.values.append(dequant(q, s))
        self.E, self.N, self.K = E, N, K
        self.Bw = torch.from_numpy(np.stack(qs)).cuda()
        self.Bs = torch.from_numpy(np.stack(ss)).cuda()


def gated(h):
    """silu(first half of the columns) * second half, in f64."""
    n = h.shape[-1] // 2
    g, u = h[..., :n], h[..., n:]
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def product_limit(x, w, out, is_gated):
    """(reference, allowed difference) of x [M, K] times w [N, K]^T, f64.

    An f32 sum of K products, in any order and whether each addition rounds
    or truncates, is off by at most K * 2^-23 * sum |x w|.  The gate passes
    its own difference on with a slope of at most 1.1, and its exponential,
    quotient and product add (|g| + 8) * 2^-22 relative.  The result is
    rounded once."""
    ref = x @ w.T
    err = w.shape[1] * 2.0**-23 * (np.abs(x) @ np.abs(w).T)
    if is_gated:
        n = ref.shape[1] // 2
        g, u = ref[:, :n], ref[:, n:]
        eg, eu = err[:, :n], err[:, n:]
        y = gated(ref)
        silu = np.abs(g / (1 + np.exp(-g)))
        err = 1.1 * eg * (np.abs(u) + eu) + silu * eu + (np.abs(g) + 8) * 2.0**-22 * np.abs(y)
        ref = y
    return ref, err + HALF_STEP[out] * (np.abs(ref) + err) + SMALLEST[out]


def assert_within(got, ref, limit, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= limit)
    if bad.any():
        at = np.argwhere(bad)[:4]
        raise AssertionError("%s: %d of %d outside; first %s" % (
            what, int(bad.sum()), bad.size,
            ["%s: %r, not %r +- %r" % (tuple(map(int, i)), got[tuple(i)], ref[tuple(i)], limit[tuple(i)]) for i in at]))

"""The dense layer value by value: each scale byte at its own size, slopes against differences of the layer itself,
infinities and NaN in bias, residual, dy and the kept z."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.linear_util import ACTS, Matrix, act, act_error, assert_within, linear_limit, rows

pytestmark = pytest.mark.gpu

# one row quantized on the way, rows quantized before, and the large tiles
FORMS = [(2, 256, 128), (100, 256, 128), (2100, 4112, 96)]


@pytest.mark.parametrize("M,N,K", FORMS)
def test_each_scale_byte_at_its_own_size(M, N, K):
    """Each row of weights has one scale byte, 0 to 254, in all its groups, so a column of y is as large as its byte
    makes it.  Rows of x lie 2^60 apart, and every column is looked at where f32 holds it far from its ends."""
    def scales(r, s):
        return np.repeat(np.arange(s.shape[0])[:, None] % 255, s.shape[1], 1).astype(np.uint8)
    w = Matrix(11, N, K, scales=scales)
    size = torch.exp2(torch.tensor([-40.0, 40.0], device="cuda").repeat((M + 1) // 2)[:M, None])
    x = (rows(12, M, K) * size).to(torch.bfloat16)
    (ref, limit), _ = linear_limit(x, w.values, "f32")
    sums = x.double().abs() @ w.values.abs().t()
    held = (sums > 2.0**-110) & (sums < 2.0**125)
    assert bool(held.any(0).all()), "a scale byte that no row of x shows"
    y = mx.linear(x, w.Bw, w.Bs, N, out_dtype=torch.float32)
    assert_within(y[held], (ref[held], limit[held]), "y")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", ACTS)
def test_bias_gradient_against_differences_at_the_same_z(activation, gated):
    """(L(b + h) - L(b - h)) / 2h of L = sum dy * y, with rows of zeros and a bias that bf16 holds, so that the kept z
    is exactly the z of the forward pass.

    The difference is off from the slope by what the 64-bit function itself is at this h, and by the two values'
    errors over 2h: act_error, one rounding of the product with up and one of y.  dbias is off by act_error of the slope,
    by up to three roundings of each term, and by M of its sum."""
    M, N, K, h = 5, 64, 32, 2.0**-6
    cols = N // 2 if gated else N
    w = Matrix(21, N, K)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    b = torch.linspace(-7, 7, N, device="cuda")
    b = b[torch.randperm(N, generator=torch.Generator().manual_seed(5)).cuda()].to(torch.bfloat16).float()
    dy = rows(22, M, cols, "f32")

    def outputs(bias):
        return mx.linear(x, w.Bw, w.Bs, N, bias=bias, activation=activation, gated=gated, out_dtype=torch.float32).double()

    _, z = mx.linear(x, w.Bw, w.Bs, N, bias=b, activation=activation, gated=gated, pre=True)
    assert torch.equal(z, b.to(torch.bfloat16).expand(M, N))
    _, db = mx.linear_grad_pre(dy, z, activation=activation, gated=gated, bias=True)
    g = b[:cols].double()
    u = b[cols:].double() if gated else torch.ones_like(g)
    hi, lo = (outputs(torch.cat([b[:cols] + s, b[cols:]])) for s in (h, -h))
    weight = dy.double().abs().sum(0)
    noise = sum((act_error(activation, g + s)[0] + 2.0**-23 * act(activation, g + s)[0].abs()) * u.abs() for s in (h, -h))
    exact = (act(activation, g + h)[0] - act(activation, g - h)[0]) / (2 * h)
    f, slope = act(activation, g)
    slack = weight * u.abs() * ((exact - slope).abs() + act_error(activation, g)[1]) + weight * noise / (2 * h) \
        + (M + 3) * 2.0**-23 * weight * (slope * u).abs()
    diff = ((hi - lo) * dy.double()).sum(0) / (2 * h)
    # Far less than a term of the slope that could be missing, but at relu's corner.  It is largest for gelu_tanh at
    # |z| = 7, where the exponential's argument is 36: two values of 7, off by (2 * 36 + 16) 2^-23 each, over 2h = 2^-5
    # are 2 * 88 * 7 * 2^-18 = 0.0047 of dy u.
    near = (activation == "relu") & (g.abs() < h)
    assert bool((slack <= weight * (1 + u.abs()) * 2.0**-7)[~near].all())
    bad = (db[:cols].double() - diff).abs() > slack
    assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), db[:cols][bad][:4].tolist(), diff[bad][:4].tolist())
    if gated:  # y is linear in up: no error of the step itself
        hi, lo = (outputs(torch.cat([b[:cols], b[cols:] + s])) for s in (h, -h))
        diff = ((hi - lo) * dy.double()).sum(0) / (2 * h)
        ef = act_error(activation, g)[0]
        slack = weight * ef + weight * (2 * ef * (u.abs() + h) + 2 * 2.0**-23 * f.abs() * (u.abs() + h)) / (2 * h) \
            + (M + 2) * 2.0**-23 * weight * f.abs()
        assert bool(((db[cols:].double() - diff).abs() <= slack).all())


def same(got, ref, limit, what):
    """NaN and infinities where the definition has them, and finite values within the limit."""
    ref = ref.expand(got.shape)
    assert torch.equal(got.isnan(), ref.isnan()), what
    inf = ref.isinf()
    assert torch.equal(got[inf].double(), ref[inf]), what
    fin = ref.isfinite()
    assert_within(got[fin], (ref[fin], limit.expand(got.shape)[fin]), what)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M,N,K", FORMS)
def test_infinities_and_nan_in_bias_and_residual(M, N, K, activation, gated):
    """They touch their own column, and element, as the formulas say: v / (1 + exp(-v)) and v Phi(v) are NaN at -infinity."""
    N = N // 64 * 64
    cols = N // 2 if gated else N
    w = Matrix(31, N, K)
    x, b, r = rows(32, M, K), torch.randn(N, device="cuda") * 0.3, rows(33, M, cols, "f32")
    odd = torch.tensor([float("inf"), -float("inf"), float("nan")], device="cuda")
    (_, limit), (zref, zlimit) = linear_limit(x, w.values, "f32", b, activation, gated, r)
    b2, r2 = b.clone(), r.clone()
    b2[5:8] = odd
    if gated:
        b2[cols + 20:cols + 23] = odd
    r2[M // 2, 9:12] = odd
    y, z = mx.linear(x, w.Bw, w.Bs, N, bias=b2, activation=activation, gated=gated, residual=r2, pre=True,
                     out_dtype=torch.float32)
    plain_z = zref + (b2 - b).double()
    same(z, plain_z, zlimit, "pre")
    f = act(activation, plain_z[:, :cols])[0]
    want = (f * plain_z[:, cols:] if gated else f) + r2.double()
    assert int((~want.isfinite()).sum()) > 2
    if gated:  # f below 2^-126 may be flushed (act_error), and 0 times an infinite up is NaN where a tiny f is not
        either = plain_z[:, cols:].isinf() & (f.abs() <= act_error(activation, plain_z[:, :cols])[0])
        y = torch.where(either, 0.0, y)
        want = torch.where(either, 0.0, want)
    same(y, want, limit, "y")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", ACTS)
@pytest.mark.parametrize("M", [4, 1000])
def test_infinities_and_nan_in_the_activation_gradient(M, activation, gated):
    """dy and up as they are; the gate's slope at infinities and NaN is NaN, but for relu, where it is 1, 0 and 0."""
    cols = 48
    dy, z = rows(41, M, cols, "f32", 0.1), rows(42, M, 2 * cols if gated else cols, "bf16", 1.5)
    plain, plain_db = mx.linear_grad_pre(dy, z, activation=activation, gated=gated, bias=True)
    odd = torch.tensor([float("inf"), -float("inf"), float("nan")], device="cuda")
    dy[1, 5:8] = odd
    z[2, 20:23] = odd.to(torch.bfloat16)
    if gated:
        z[3, cols + 30:cols + 33] = odd.to(torch.bfloat16)
    dz, db = mx.linear_grad_pre(dy, z, activation=activation, gated=gated, bias=True)
    touched = torch.zeros(dz.shape, dtype=torch.bool, device="cuda")
    touched[1, 5:8] = touched[2, 20:23] = True
    if gated:
        touched[:, cols:] |= touched[:, :cols]
        touched[3, 30:33] = True
    assert torch.equal(dz[~touched], plain[~touched])
    clean = ~touched.any(0)
    assert torch.equal(db[clean], plain_db[clean])
    g = z[:, :cols].double()
    f, slope = act(activation, g)
    if activation == "none":
        assert torch.equal(dz[2, 20:23], (dy[2, 20:23] * (z[2, cols + 20:cols + 23].float() if gated else 1)).to(torch.bfloat16))
    elif activation == "relu":
        want = dy[2, 20:23] * torch.tensor([1.0, 0.0, 0.0], device="cuda")
        assert torch.equal(dz[2, 20:23], (want * z[2, cols + 20:cols + 23].float() if gated else want).to(torch.bfloat16))
    else:
        assert bool(dz[2, 20:23].isnan().all())
    assert not bool(torch.isfinite(dz[1, 5:8]).any()) or activation == "relu"
    assert torch.equal(dz[1, 5:8].isnan(), (dy[1, 5:8].double() * (z[1, cols + 5:cols + 8].double() if gated else 1)
                                            * slope[1, 5:8]).isnan())
    if gated:
        assert torch.equal(dz[2, cols + 20:cols + 23].isnan(), (dy[2, 20:23].double() * f[2, 20:23]).isnan())
        assert torch.equal(dz[3, 30:33].isnan(), (dy[3, 30:33].double() * z[3, cols + 30:cols + 33].double()
                                                  * slope[3, 30:33]).isnan())

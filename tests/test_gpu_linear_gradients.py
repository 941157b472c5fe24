"""The gradients of the dense layer against their 64-bit forms, against differences, and used together."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import dtype_of
from tests.linear_util import ACTS, Matrix, assert_within, grad_pre_limit, product_limit, quantized, rows

pytestmark = pytest.mark.gpu

TYPES = ["bf16", "f32", "f16"]


# ---- activation, gate and bias ----------------------------------------------------

@pytest.mark.parametrize("M,cols", [(1, 16), (1, 4096), (2, 48), (7, 2112), (16, 272), (17, 256), (65, 1040), (333, 96),
                                    (1000, 512), (4099, 64)])
@pytest.mark.parametrize("gated", [False, True])
def test_grad_pre_sizes(M, cols, gated):
    for i, activation in enumerate(ACTS):
        t = TYPES[(i + M) % 3]
        dy = rows(M + i, M, cols, t, 0.1)
        z = rows(M + i + 50, M, 2 * cols if gated else cols, "bf16", 1.5)
        want_dz, want_db = grad_pre_limit(dy, z, activation, gated)
        dz, db = mx.linear_grad_pre(dy, z, activation=activation, gated=gated, bias=True)
        assert_within(dz, want_dz, "dz of %s" % activation)
        assert_within(db, want_db, "dbias of %s" % activation)
        assert torch.equal(dz, mx.linear_grad_pre(dy, z, activation=activation, gated=gated))


def test_grad_pre_into_a_given_dbias():
    dy = rows(1, 700, 96, "f32", 0.1)
    want = mx.linear_grad_pre(dy, None, bias=True)[1]
    db = torch.full((96,), 7.0, device="cuda")
    assert mx.linear_grad_pre(dy, None, bias=db)[1] is db
    assert torch.equal(db, want)


@pytest.mark.parametrize("t", TYPES)
def test_grad_pre_without_activation_needs_no_pre(t):
    dy = rows(1, 37, 80, t, 0.1)
    want_dz, want_db = grad_pre_limit(dy, None)
    dz, db = mx.linear_grad_pre(dy, None, bias=True)
    assert_within(dz, want_dz, "dz")
    assert_within(db, want_db, "dbias")


def test_grad_pre_far_arguments_and_zeros():
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 20.0, -20.0, 100.0, -100.0, 1e10, -1e10, 1e25, -1e25, 3e38,
                      -3e38], device="cuda").to(torch.bfloat16).reshape(1, 16)
    dy = torch.ones((1, 16), device="cuda")
    for activation in ACTS:
        want, _ = grad_pre_limit(dy, z.clamp(-1e4, 1e4), activation)  # the slopes are 0 or 1 from there on
        assert_within(mx.linear_grad_pre(dy, z, activation=activation), want, activation)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
def test_grad_pre_strides_and_in_place(pad, gated):
    M, cols = 45, 96
    N = 2 * cols if gated else cols
    dy, z = rows(1, M, cols, "f32", 0.1, pad=pad), rows(2, M, N, "bf16", 1.5, pad=pad)
    want, want_db = grad_pre_limit(dy, z, "silu", gated)
    whole = torch.full((M + 2, N + 2 * pad), 777.0, dtype=torch.bfloat16, device="cuda")
    dz = whole[1:M + 1, pad:pad + N]
    got, db = mx.linear_grad_pre(dy, z, activation="silu", gated=gated, bias=True, out=dz)
    assert got is dz
    assert_within(dz, want, "dz")
    assert_within(db, want_db, "dbias")
    plain = dz.clone()
    dz.fill_(777.0)
    assert bool((whole == 777.0).all())
    mx.linear_grad_pre(dy, z, activation="silu", gated=gated, out=z)
    assert torch.equal(z, plain)


# ---- the two products -------------------------------------------------------------

SIZES = [(1, 16, 32), (1, 2112, 704), (2, 48, 96), (9, 4096, 64), (16, 16, 4096), (17, 112, 160), (24, 1024, 1024),
         (33, 272, 288), (64, 64, 128), (127, 528, 224), (129, 1040, 96), (255, 32, 1056), (257, 304, 544), (300, 768, 256),
         (771, 144, 416), (1030, 1296, 320), (2051, 80, 64)]


@pytest.mark.parametrize("i,size", enumerate(SIZES))
def test_grad_input_sizes(i, size):
    M, N, K = size
    t = TYPES[i % 3]
    w = Matrix(i, N, K)
    dz = rows(i + 100, M, N, "bf16", 0.1)
    want = product_limit(dz, w.values, t)
    assert_within(mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=dtype_of(torch, t)), want, "dx")


@pytest.mark.parametrize("i,size", enumerate(SIZES))
def test_grad_weight_sizes(i, size):
    M, N, K = size
    t = TYPES[(i + 1) % 3]
    dz, x = rows(i + 200, M, N, "bf16", 0.1), rows(i + 300, M, K)
    want = product_limit(dz.t().contiguous(), quantized(x), t)
    assert_within(mx.linear_grad_weight(dz, x, out_dtype=dtype_of(torch, t)), want, "dw")


@pytest.mark.parametrize("M,N,K", [(4096, 2048, 512), (520, 4096, 1056), (24, 4096, 4096), (2, 8192, 96), (700, 16384, 64)])
def test_larger_products(M, N, K):
    """Sizes at which tiles are many, or where a tile's sum is split over workgroups and joined."""
    w = Matrix(M, N, K)
    dz, x = rows(1, M, N, "bf16", 0.1), rows(2, M, K)
    assert_within(mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=torch.float32), product_limit(dz, w.values, "f32"), "dx")
    assert_within(mx.linear_grad_weight(dz, x), product_limit(dz.t().contiguous(), quantized(x), "f32"), "dw")


@pytest.mark.parametrize("pad", [8, 24])
@pytest.mark.parametrize("left,right", [(8, 8), (1, 2), (4, 1)])
@pytest.mark.parametrize("M", [5, 300])
def test_strides_and_what_lies_around(M, left, right, pad):
    """Strided inputs whose gaps hold NaN, and outputs inside longer rows."""
    N, K = 176, 160
    w = Matrix(1, N, K)

    def gapped(t):
        whole = torch.full((t.shape[0] + 1, t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        whole[:-1, :t.shape[1]] = t
        return whole[:-1, :t.shape[1]]

    dz, x = gapped(rows(3, M, N, "bf16", 0.1)), gapped(rows(4, M, K))
    for t in ("bf16", "f32"):
        for shape, call, want in (
                ((M, K), lambda o: mx.linear_grad_input(dz, w.Bw, w.Bs, K, out=o), product_limit(dz, w.values, t)),
                ((N, K), lambda o: mx.linear_grad_weight(dz, x, out=o), product_limit(dz.t().contiguous(), quantized(x), t))):
            whole = torch.full((shape[0] + 2, left + shape[1] + right), 777.0, dtype=dtype_of(torch, t), device="cuda")
            out = whole[1:-1, left:left + shape[1]]
            assert call(out) is out
            assert_within(out, want, "out")
            out.fill_(777.0)
            assert bool((whole == 777.0).all()), "something outside the rows was written"


def test_no_rows():
    w = Matrix(1, 64, 96)
    dz, x = (torch.empty((0, n), dtype=torch.bfloat16, device="cuda") for n in (64, 96))
    assert mx.linear_grad_input(dz, w.Bw, w.Bs, 96).shape == (0, 96)
    dw = torch.full((64, 96), 7.0, device="cuda")
    assert bool((mx.linear_grad_weight(dz, x, out=dw) == 0).all())
    empty, db = mx.linear_grad_pre(dz, dz, activation="silu", bias=True)
    assert empty.shape == (0, 64) and bool((db == 0).all())


def test_rows_of_nan_and_infinity_touch_their_own_row_only():
    M, N, K = 70, 96, 64
    w = Matrix(2, N, K)
    dz = rows(3, M, N, "bf16", 0.1)
    clean = mx.linear_grad_input(dz, w.Bw, w.Bs, K)
    dz[5, 3], dz[40] = float("inf"), float("nan")
    dirty = mx.linear_grad_input(dz, w.Bw, w.Bs, K)
    same = torch.ones(M, dtype=torch.bool, device="cuda")
    same[[5, 40]] = False
    assert torch.equal(dirty[same], clean[same])
    assert not bool(torch.isfinite(dirty[40]).any())


@pytest.mark.parametrize("M", [3, 140])
def test_scale_bytes_and_subnormal_gradients(M):
    """Each row group of weights with another scale byte, 0 to 252; gradients down to bf16's smallest."""
    def scales(r, s):
        return np.repeat(r.integers(0, 253, (s.shape[0], 1)), s.shape[1], 1).astype(np.uint8)
    N, K = 256, 64
    w = Matrix(5, N, K, scales=scales)
    one = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(M, device="cuda") % N
    one[torch.arange(M, device="cuda"), at] = 1.0
    got = mx.linear_grad_input(one, w.Bw, w.Bs, K, out_dtype=torch.float32)
    assert torch.equal(got.double(), w.values[at])  # one term each: exact
    w = Matrix(6, N, K, scale=64.0)
    tiny = one * 2.0**-133
    got = mx.linear_grad_input(tiny, w.Bw, w.Bs, K, out_dtype=torch.float32)
    assert torch.equal(got.double(), w.values[at] * 2.0**-133)


@pytest.mark.parametrize("M,N,K", [(20, 4096, 256), (300, 512, 512), (2048, 96, 64)])
def test_same_bits_every_time(M, N, K):
    w = Matrix(1, N, K)
    dz, x = rows(2, M, N, "bf16", 0.1), rows(3, M, K)
    first = mx.linear_grad_input(dz, w.Bw, w.Bs, K), mx.linear_grad_weight(dz, x), mx.linear_grad_pre(dz, None, bias=True)[1]
    for _ in range(20):
        again = mx.linear_grad_input(dz, w.Bw, w.Bs, K), mx.linear_grad_weight(dz, x), mx.linear_grad_pre(dz, None, bias=True)[1]
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    mx.mxfp4_set_quant_mode(1)
    try:
        assert torch.equal(first[1], mx.linear_grad_weight(dz, x))
    finally:
        mx.mxfp4_set_quant_mode(0)


# ---- against differences, and together -----------------------------------------------

@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", ACTS)
def test_bias_gradient_against_differences(activation, gated):
    """(L(b + h) - L(b - h)) / 2h of L = sum dy * y, with y in f32.

    z is kept in bf16 (2^-8 relative to a z of up to about 5: the slope, whose own
    slope is at most 1.2, is off by 0.025 times u), y is off by about 2^-22 of
    its size, which h = 2^-6 raises to 2^-16, and the difference itself by h^2 / 6
    of the third derivative, less than 2^-13."""
    M, N, K, h = 6, 64, 96, 2.0**-6
    w = Matrix(21, N, K)
    x = rows(22, M, K)
    cols = N // 2 if gated else N
    b = torch.randn(N, device="cuda") * 0.3
    dy = torch.randn((M, cols), device="cuda")

    def outputs(bias):
        return mx.linear(x, w.Bw, w.Bs, N, bias=bias, activation=activation, gated=gated, out_dtype=torch.float32).double()

    _, z = mx.linear(x, w.Bw, w.Bs, N, bias=b, activation=activation, gated=gated, pre=True)
    _, db = mx.linear_grad_pre(dy, z, activation=activation, gated=gated, bias=True)
    size = float(z.abs().max())
    for n in range(0, N, 5):
        c = n % cols
        if activation == "relu" and not (gated and n >= cols) and float(z[:, c].abs().min()) < 2 * h:
            continue  # the corner lies within the step
        step = torch.zeros(N, device="cuda")
        step[n] = h
        diff = ((outputs(b + step) - outputs(b - step)) * dy).sum(0)[c] / (2 * h)
        slack = float(dy[:, c].abs().sum()) * (1 + size) * (0.025 + 2.0**-13)
        assert abs(float(db[n]) - float(diff)) <= slack, (n, float(db[n]), float(diff))


@pytest.mark.parametrize("M,N,K", [(30, 160, 96), (400, 512, 288)])
def test_products_are_adjoint(M, N, K):
    """<dz W, v> = <dz, v W^T> = <dz^T v, W> for rows v that quantization leaves as they are."""
    w = Matrix(31, N, K)
    v = quantized(rows(32, M, K)).to(torch.bfloat16)
    assert torch.equal(quantized(v), v.double())
    dz = rows(33, M, N, "bf16", 0.1)
    y = mx.linear(v, w.Bw, w.Bs, N, out_dtype=torch.float32).double()
    dx = mx.linear_grad_input(dz, w.Bw, w.Bs, K, out_dtype=torch.float32).double()
    dw = mx.linear_grad_weight(dz, v).double()
    a, b, c = (dz.double() * y).sum(), (dx * v.double()).sum(), (dw * w.values).sum()
    size = (dz.double().abs() * (v.double().abs() @ w.values.abs().t())).sum()
    slack = float(size) * max(M, N, K) * 2.0**-23
    assert abs(float(a - b)) <= slack and abs(float(a - c)) <= slack


def test_workspaces_streams_and_graphs():
    """A whole backward pass on a side stream, captured and replayed with a workspace of its own, and eager."""
    M, N, K = 260, 512, 256
    w = Matrix(41, N, K)
    x, dy = rows(42, M, K), rows(43, M, N // 2, "bf16", 0.1)
    need = max(mx.mxfp4_linear_workspace_bytes(M, N, K), mx.mxfp4_linear_grad_pre_workspace_bytes(M, N),
               mx.mxfp4_linear_grad_input_workspace_bytes(M, N, K), mx.mxfp4_linear_grad_weight_workspace_bytes(M, N, K))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(**how):
        y, z = mx.linear(x, w.Bw, w.Bs, N, activation="silu", gated=True, pre=True, **how)
        dz, db = mx.linear_grad_pre(dy, z, activation="silu", gated=True, bias=True, **how)
        return y, dz, db, mx.linear_grad_input(dz, w.Bw, w.Bs, K, **how), mx.linear_grad_weight(dz, x, **how)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(workspace=ws)
    for seed in range(4):
        x.copy_(rows(50 + seed, M, K))
        dy.copy_(rows(60 + seed, M, N // 2, "bf16", 0.1))
        want = step()
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    for call, size in ((lambda s: mx.linear_grad_weight(out[1], x, workspace=s),
                        mx.mxfp4_linear_grad_weight_workspace_bytes(M, N, K)),
                       (lambda s: mx.linear_grad_pre(dy, None, bias=True, workspace=s),
                        mx.mxfp4_linear_grad_pre_workspace_bytes(M, N // 2))):
        with pytest.raises(RuntimeError, match="workspace"):
            call(ws[:size - 1])

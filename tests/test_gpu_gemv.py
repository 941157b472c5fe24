"""mxfp4_gemv against the product in 64 bits: row counts around the tile
sizes, odd N and K, every type of x and y, one matrix and one per row,
strides, rows without a matrix, non-finite rows, streams and graphs."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights, assert_within, dtype_of, product_limit
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def rows(torch, seed, M, K, xt, scale=1.0):
    r = np.random.default_rng(seed)
    return torch.from_numpy((r.standard_normal((M, K)) * scale).astype(np.float32)).to(dtype_of(torch, xt)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32"),
                                   ("f32", "bf16")])
@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (1, 4096, 512), (1, 2112, 1120), (2, 96, 160), (5, 160, 96),
                                   (16, 224, 640), (17, 64, 2048), (33, 96, 288), (64, 480, 1024), (65, 32, 64),
                                   (130, 32, 416)])
def test_matches_the_product_in_64_bits(M, N, K, xt, yt, gated):
    torch = torch_cuda()
    w = Weights(torch, M * 7 + N + K, 1, N, K)
    x = rows(torch, M + K, M, K, xt)
    y = mx.gemv(x, w.Bw, w.Bs, N, gated=gated, out_dtype=dtype_of(torch, yt))
    assert y.shape == (M, N // 2 if gated else N) and y.dtype == dtype_of(torch, yt)
    ref, limit = product_limit(f64(x), w.values[0], yt, gated)
    assert_within(y, ref, limit, "%dx%dx%d %s->%s" % (M, N, K, xt, yt))


@pytest.mark.parametrize("N", [16, 48, 2096])
def test_odd_groups_of_columns(N):
    torch = torch_cuda()
    w = Weights(torch, N, 1, N, 352)
    for M in (1, 18, 50):
        x = rows(torch, M, M, 352, "bf16")
        ref, limit = product_limit(f64(x), w.values[0], "f32", False)
        assert_within(mx.gemv(x, w.Bw, w.Bs, N, out_dtype=torch.float32), ref, limit, "M %d N %d" % (M, N))


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,K,tokens,repeat", [(4, 96, 160, 3, 2), (7, 64, 1056, 1, 5), (3, 32, 32, 9, 3)])
def test_one_matrix_per_row(E, N, K, tokens, repeat, gated, xt):
    torch = torch_cuda()
    w = Weights(torch, E + N, E, N, K)
    x = rows(torch, 5, tokens, K, xt)
    r = np.random.default_rng(E * K)
    ids = r.integers(0, E, tokens * repeat).astype(np.int32)
    ids[0] = -1  # rows without a matrix
    if ids.size > 3:
        ids[3] = E
    out = torch.full((tokens * repeat, N // 2 if gated else N), 7.0, device="cuda")
    y = mx.gemv(x, w.Bw, w.Bs, N, ids=torch.from_numpy(ids).cuda(), repeat=repeat, gated=gated, out=out)
    assert y is out
    for i, e in enumerate(ids):
        if 0 <= e < E:
            ref, limit = product_limit(f64(x)[i // repeat][None], w.values[e], "f32", gated)
            assert_within(y[i][None], ref, limit, "row %d" % i)
        else:
            assert not y[i].any()


def test_one_matrix_per_row_equals_that_row_alone():
    torch = torch_cuda()
    w = Weights(torch, 3, 5, 224, 576)
    x = rows(torch, 4, 6, 576, "bf16")
    ids = torch.tensor([4, 0, 2, 2, 1, 3], dtype=torch.int32, device="cuda")
    y = mx.gemv(x, w.Bw, w.Bs, 224, ids=ids)
    for i, e in enumerate(ids.tolist()):
        assert torch.equal(y[i:i + 1], mx.gemv(x[i:i + 1], w.Bw[e], w.Bs[e], 224))


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
def test_strided_rows(xt):
    torch = torch_cuda()
    M, N, K = 19, 96, 224
    w = Weights(torch, 8, 1, N, K)
    wide = rows(torch, 9, M, K + 40, xt)
    x = wide[:, 8:8 + K]
    out = torch.full((M, N + 5), 3.0, device="cuda")
    mx.gemv(x, w.Bw, w.Bs, N, out=out[:, 2:2 + N])
    ref, limit = product_limit(f64(x), w.values[0], "f32", False)
    assert_within(out[:, 2:2 + N], ref, limit, "strided")
    assert bool((out[:, :2] == 3).all()) and bool((out[:, 2 + N:] == 3).all())


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_scales_far_from_one(xt, power):
    """Weights that f16 could not hold are exact all the same."""
    torch = torch_cuda()
    w = Weights(torch, 11, 1, 64, 192, scale=2.0**power)
    x = rows(torch, 12, 3, 192, xt)
    ref, limit = product_limit(f64(x), w.values[0], "f32", False)
    assert_within(mx.gemv(x, w.Bw, w.Bs, 64, out_dtype=torch.float32), ref, limit, "2^%d" % power)


def test_f32_rows_keep_all_their_bits():
    """With one weight of 1 per column the product is x itself, to the last bit."""
    torch = torch_cuda()
    K = 64
    eye = np.zeros((K, K), dtype=np.float32)
    np.fill_diagonal(eye, 1.0)
    b = torch.from_numpy(eye).to(torch.bfloat16).cuda()
    Bw, Bs = mx.prepare_b(b)
    x = rows(torch, 13, 5, K, "f32", scale=1e3)
    assert torch.equal(mx.gemv(x, Bw, Bs, K), x)


@pytest.mark.parametrize("xt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_stays_alone(xt, bad):
    torch = torch_cuda()
    N, K = 96, 320
    w = Weights(torch, 14, 1, N, K)
    x = rows(torch, 15, 18, K, xt)
    clean = mx.gemv(x, w.Bw, w.Bs, N)
    x[4, 77] = bad
    y = mx.gemv(x, w.Bw, w.Bs, N)
    others = [i for i in range(18) if i != 4]
    assert torch.equal(y[others], clean[others])
    column = w.values[0][:, 77]
    with np.errstate(invalid="ignore"):
        want = np.where(column == 0, np.nan, bad * np.sign(column))
    assert np.array_equal(f64(y[4]), want, equal_nan=True)


def test_offsets_beyond_32_bits():
    """The last of many matrices, whose codes start past 2^31 bytes."""
    torch = torch_cuda()
    N = K = 8192
    E = (1 << 31) // (N * K // 2) + 2
    small = Weights(torch, 16, 1, N, 64)
    Bw = torch.zeros((E, N // 16, K * 8), dtype=torch.uint8, device="cuda")
    Bs = torch.full((E, N // 32, K), 127, dtype=torch.uint8, device="cuda")
    Bw[E - 1, :, :64 * 8] = small.Bw[0]  # the first 64 of K; the other codes stand for zero
    Bs[E - 1, :, :256] = small.Bs[0].reshape(N // 32, 256)
    x = rows(torch, 17, 2, K, "bf16")
    y = mx.gemv(x, Bw, Bs, N, ids=torch.tensor([E - 1, 0], dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    ref, limit = product_limit(f64(x)[:1, :64], small.values[0], "f32", False)
    assert_within(y[:1], ref, limit, "last matrix")
    assert not y[1].any()


def test_same_bits_every_time_and_on_other_streams():
    torch = torch_cuda()
    w = Weights(torch, 18, 1, 160, 2016)
    x = rows(torch, 19, 7, 2016, "bf16")
    first = mx.gemv(x, w.Bw, w.Bs, 160)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = [mx.gemv(x, w.Bw, w.Bs, 160) for _ in range(8)]
    s.synchronize()
    assert all(torch.equal(first, y) for y in again)


def test_captured_into_a_graph():
    torch = torch_cuda()
    w = Weights(torch, 20, 3, 96, 512)
    x = rows(torch, 21, 4, 512, "bf16")
    ids = torch.tensor([2, 1, 0, 2], dtype=torch.int32, device="cuda")
    y = torch.empty((4, 48), dtype=torch.bfloat16, device="cuda")
    mx.gemv(x, w.Bw, w.Bs, 96, ids=ids, gated=True, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.gemv(x, w.Bw, w.Bs, 96, ids=ids, gated=True, out=y)
    for k in range(4):
        x.copy_(rows(torch, 30 + k, 4, 512, "bf16"))
        ids.copy_(torch.tensor([k % 3, 0, 1, 2], dtype=torch.int32))
        want = mx.gemv(x, w.Bw, w.Bs, 96, ids=ids, gated=True)
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)

"""mxfp4_moe_combine against the sum in 64 bits: types, odd widths, strides and
alignments, choices that add nothing, a residual in place, streams and graphs."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import HALF_STEP, SMALLEST, assert_within, dtype_of
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def randn(torch, seed, shape, t):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(dtype_of(torch, t)).cuda()


def reference(y, w, pos, res, out):
    """(sum, allowed difference): k products and k + 1 additions in f32, one rounding of the result."""
    y, w = y.double().cpu().numpy(), w.double().cpu().numpy()
    T, k = w.shape
    p = np.arange(T * k).reshape(T, k) if pos is None else pos.cpu().numpy()
    ok = (p >= 0) & (p < y.shape[0])
    terms = np.where(ok[..., None], y[np.where(ok, p, 0)] * w[..., None], 0.0) if y.shape[0] else np.zeros((T, k, y.shape[1]))
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    if res is not None:
        res = res.double().cpu().numpy()
        ref, size = ref + res, size + np.abs(res)
    err = (2 * k + 1) * 2.0**-24 * size
    return ref, err + HALF_STEP[out] * (np.abs(ref) + err) + SMALLEST[out]


@pytest.mark.parametrize("yt,ot", [("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 7168), (4, 8, 264), (33, 3, 129), (5, 9, 2048), (2, 20, 40),
                                   (300, 6, 520), (1030, 2, 8)])
def test_matches_the_sum_in_64_bits(T, k, N, with_res, yt, ot):
    torch = torch_cuda()
    rows = T * k + 3
    y = randn(torch, T + N, (rows, N), yt)
    r = np.random.default_rng(k)
    w = torch.from_numpy(r.random((T, k)).astype(np.float32)).cuda()
    pos = torch.from_numpy(r.permutation(rows)[:T * k].reshape(T, k).astype(np.int32)).cuda()
    res = randn(torch, 9, (T, N), ot) if with_res else None
    for p in (None, pos):
        got = mx.moe_combine(y, w, pos=p, residual=res, out_dtype=dtype_of(torch, ot))
        assert_within(got, *reference(y, w, p, res, ot), "%d x %d of %d" % (T, N, k))


def test_choices_that_add_nothing():
    torch = torch_cuda()
    y = randn(torch, 1, (10, 64), "bf16")
    y[3] = float("nan")
    w = torch.ones((4, 3), device="cuda")
    pos = torch.tensor([[0, -1, 2], [-1, -1, -1], [10, 9, 1 << 30], [4, 4, -(1 << 31)]], dtype=torch.int32, device="cuda")
    res = randn(torch, 2, (4, 64), "bf16")
    for residual in (None, res):
        got = mx.moe_combine(y, w, pos=pos, residual=residual)
        assert_within(got, *reference(y, w, pos, residual, "bf16"), "skipped")
    assert not mx.moe_combine(y, w, pos=pos)[1].any()
    none = mx.moe_combine(y[:0], w, pos=pos, residual=res)
    assert torch.equal(none, res)
    assert mx.moe_combine(y, w[:0], pos=pos[:0]).shape == (0, 64)


@pytest.mark.parametrize("shift,N", [(0, 96), (1, 96), (8, 96), (3, 31)])
def test_strides_alignments_and_a_residual_in_place(shift, N):
    torch = torch_cuda()
    T, k = 21, 4
    y = randn(torch, 3, (T * k, N + 24), "bf16")[:, shift:shift + N]
    w = torch.rand((T, k), device="cuda")
    wide = randn(torch, 4, (T, N + 40), "bf16")
    before = wide.clone()
    out = wide[:, shift:shift + N]
    ref = reference(y, w, None, out, "bf16")
    assert mx.moe_combine(y, w, residual=out, out=out) is out
    assert_within(out, *ref, "in place")
    assert torch.equal(wide[:, :shift], before[:, :shift]) and torch.equal(wide[:, shift + N:], before[:, shift + N:])


def test_not_finite_stays_alone():
    torch = torch_cuda()
    y = randn(torch, 5, (12, 80), "f32")
    w = torch.rand((6, 2), device="cuda")
    clean = mx.moe_combine(y, w)
    y[5, 9], y[8, 1] = float("inf"), float("nan")
    got = mx.moe_combine(y, w)
    assert torch.isinf(got[2, 9]) and torch.isnan(got[4, 1])
    got[2, 9], got[4, 1] = clean[2, 9], clean[4, 1]
    assert torch.equal(got, clean)


def test_rows_beyond_32_bit_offsets():
    torch = torch_cuda()
    N = 4096
    rows = (1 << 31) // N + 3
    y = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
    y[rows - 1] = randn(torch, 6, (N,), "bf16")
    w = torch.full((2, 1), 0.5, device="cuda")
    pos = torch.tensor([[rows - 1], [0]], dtype=torch.int32, device="cuda")
    got = mx.moe_combine(y, w, pos=pos)
    assert torch.equal(got[0], y[rows - 1] / 2) and not got[1].any()


def test_more_tokens_than_a_grid_dimension_holds():
    torch = torch_cuda()
    T = 70001
    y = randn(torch, 7, (T, 8), "f32")
    got = mx.moe_combine(y, torch.ones((T, 1), device="cuda"), out_dtype=torch.float32)
    assert torch.equal(got, y)


def test_other_streams_and_graphs():
    torch = torch_cuda()
    y = randn(torch, 8, (64, 128), "bf16")
    w = torch.rand((16, 4), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = mx.moe_combine(y, w)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mx.moe_combine(y, w, out=out)
    for i in range(4):
        y.copy_(randn(torch, 40 + i, (64, 128), "bf16"))
        want = mx.moe_combine(y, w)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

"""mxfp4_moe_route against the definition in 64 bits: choices, weights and the
sort, for every lane layout of the kernels, with ties, excluded experts, rows
that leave none, odd counts, strides, streams and graphs."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import dtype_of
from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def reference(l, k, score, bias, renorm):
    """ids, weights, offsets, rows, pos of f64 logits [T, E]."""
    T, E = l.shape
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, 3.402823466385288598e38))
    dead = np.isneginf(l)
    with np.errstate(over="ignore"):
        if score == "softmax":
            top = l.max(1, keepdims=True)
            g = np.exp(l - np.where(np.isneginf(top), 0, top))
            total = g.sum(1, keepdims=True)
            g = g / np.where(total > 0, total, 1)
        else:
            g = 1 / (1 + np.exp(-l))
    by = l
    if bias is not None:
        dead = dead | np.isneginf(bias) | np.isnan(bias)
        by = g + bias
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), np.where(dead, 0, -by), dead), axis=1)[:, :k]
    gone = np.take_along_axis(dead, order, 1)
    w = np.where(gone, 0.0, np.take_along_axis(g, order, 1))
    if renorm:
        s = w.sum(1, keepdims=True)
        w = w / np.where(s > 0, s, 1)
    ids = np.where(gone, -1, order).astype(np.int32)
    flat = ids.reshape(-1)
    offsets, rows = [0], []
    for e in range(E):
        rows += np.flatnonzero(flat == e).tolist()
        offsets.append(len(rows))
    pos = np.full(flat.size, -1, np.int32)
    pos[rows] = np.arange(len(rows))
    rows += [-1] * (flat.size - len(rows))
    return ids, w, np.array(offsets), np.array(rows), pos.reshape(ids.shape)


def check(torch, logits, k, score="softmax", bias=None, renorm=True, what="", out=None):
    got = mx.moe_route(logits, k, score=score, bias=bias, renormalize=renorm, out=out)
    want = reference(logits.double().cpu().numpy(), k, score,
                     None if bias is None else bias.double().cpu().numpy(), renorm)
    names = ["ids", "weights", "offsets", "rows", "pos"]
    for name, g, w in zip(names, got, want):
        g = g.cpu().numpy()
        assert g.shape == w.shape, (what, name)
        if name == "weights":
            # computed in f64 (a few 2^-53 each, E of them in a sum) and rounded once to f32
            limit = w * (2.0**-24 + 4 * logits.shape[1] * 2.0**-53) + 2.0**-149
            assert (np.abs(g - w) <= limit).all(), (what, name)
        else:
            assert np.array_equal(g, w), (what, name, np.argwhere(g != w)[:4])
    return got


def logits_of(torch, seed, T, E, xt, scale=1.5):
    r = np.random.default_rng(seed)
    return torch.from_numpy((r.standard_normal((T, E)) * scale).astype(np.float32)).to(dtype_of(torch, xt)).cuda()


@pytest.mark.parametrize("score,use_bias,renorm", [("softmax", False, True), ("softmax", False, False),
                                                   ("softmax", True, True), ("sigmoid", False, True),
                                                   ("sigmoid", True, False)])
@pytest.mark.parametrize("T,E,k,xt", [(1, 1, 1, "f32"), (1, 64, 8, "bf16"), (3, 2, 2, "f16"), (17, 60, 6, "bf16"),
                                      (128, 65, 16, "f32"), (129, 100, 1, "f16"), (300, 128, 8, "f32"),
                                      (64, 256, 8, "bf16"), (257, 200, 17, "f32"), (1000, 256, 32, "bf16"),
                                      (40, 300, 5, "f32"), (150, 1000, 20, "f16"), (131, 1024, 32, "f32"),
                                      (5001, 64, 4, "f32")])
def test_matches_the_definition(T, E, k, xt, score, use_bias, renorm):
    torch = torch_cuda()
    logits = logits_of(torch, T * E + k, T, E, xt)
    bias = logits_of(torch, E, 1, E, "f32", 0.1).reshape(-1) if use_bias else None
    check(torch, logits, k, score, bias, renorm, "%d tokens of %d, k %d" % (T, E, k))


@pytest.mark.parametrize("T", [7, 400])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("use_bias", [False, True])
def test_excluded_experts_and_rows_that_leave_none(T, score, use_bias):
    torch = torch_cuda()
    E, k = 24, 6
    l = logits_of(torch, T, T, E, "f32")
    r = np.random.default_rng(T)
    l[torch.from_numpy(r.random((T, E)) < 0.5).cuda()] = -float("inf")
    l[0] = -float("inf")
    l[1] = float("nan")
    l[2, :] = -float("inf")
    l[2, 5] = 1.0  # one expert left
    l[3, ::2] = float("nan")
    l[4] = torch.finfo(torch.float32).min  # a mask of the lowest value excludes nothing
    l[5, 3] = float("inf")
    l[5, 9] = float("inf")
    l[T - 1] = -float("inf")
    bias = None
    if use_bias:
        bias = logits_of(torch, 3, 1, E, "f32", 0.1).reshape(-1)
        bias[4] = -float("inf")
        bias[7] = float("nan")
    got = check(torch, l, k, score, bias, True, "masked")
    assert bool((got[0][0] == -1).all()) and not got[1][0].any()


@pytest.mark.parametrize("T", [5, 700])
def test_every_row_empty(T):
    torch = torch_cuda()
    l = torch.full((T, 40), -float("inf"), device="cuda")
    got = check(torch, l, 4, what="all empty")
    assert not got[2].any() and bool((got[3] == -1).all())


@pytest.mark.parametrize("E,k", [(16, 8), (128, 16), (256, 20), (700, 12)])
def test_ties_go_to_the_lower_expert(E, k):
    torch = torch_cuda()
    r = np.random.default_rng(E)
    l = torch.from_numpy(r.integers(-2, 3, (200, E)).astype(np.float32)).cuda()
    l[0] = 0
    l[1, ::2] = -0.0  # equal to +0
    l[1, 1::2] = 0.0
    check(torch, l, k, what="ties")
    check(torch, l, k, "sigmoid", torch.zeros(E, device="cuda"), what="ties with a bias")


def test_bias_decides_beyond_f32():
    """Two sums that round to the same f32 are told apart."""
    torch = torch_cuda()
    l = torch.zeros((1, 8), device="cuda")
    l[0, 6] = 1e-7  # sigmoid 0.5 + 2.5e-8, below half a step of f32 at 0.5 + bias
    bias = torch.full((8,), 8.0, device="cuda")
    got = check(torch, l, 2, "sigmoid", bias, what="bias")
    assert got[0].tolist() == [[6, 0]]


@pytest.mark.parametrize("T", [9, 333])
def test_one_expert_takes_all(T):
    torch = torch_cuda()
    l = torch.zeros((T, 64), device="cuda")
    l[:, 63] = 50
    check(torch, l, 1, what="one expert")
    check(torch, l * 100, 3, renorm=False, what="far logits")


def test_no_tokens():
    torch = torch_cuda()
    offsets = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    out = mx.moe_route(torch.empty((0, 8), device="cuda"), 2,
                       out=(e(0, 2), torch.empty((0, 2), device="cuda"), offsets, e(0), e(0, 2)))
    assert not out[2].any()


@pytest.mark.parametrize("T", [30, 400])
def test_strided_rows_and_untouched_neighbours(T):
    torch = torch_cuda()
    wide = logits_of(torch, 4, T, 101, "bf16")
    i = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")
    pads = [i(T * 3 + 8), torch.full((T * 3 + 8,), 7.0, device="cuda"), i(61 + 8), i(T * 3 + 8), i(T * 3 + 8)]
    sizes = [T * 3, T * 3, 61, T * 3, T * 3]
    views = [p[4:4 + n] for p, n in zip(pads, sizes)]
    out = (views[0].view(T, 3), views[1].view(T, 3), views[2], views[3], views[4].view(T, 3))
    check(torch, wide[:, 7:67], 3, what="strided", out=out)
    for p, n in zip(pads, sizes):
        assert len(set(p[:4].tolist() + p[4 + n:].tolist())) == 1


def test_a_callers_workspace_gives_the_same():
    torch = torch_cuda()
    T, E, k = 1000, 96, 4
    l = logits_of(torch, 6, T, E, "f32")
    want = mx.moe_route(l, k)
    got = [torch.empty_like(t) for t in want]
    n = mx.mxfp4_moe_route_workspace_bytes(T, E)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    mx.mxfp4_moe_route(l, 2, E, None, T, E, k, 0, True, *got, workspace=ws, workspace_bytes=n)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bool((ws[n:] == 255).all())
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        mx.mxfp4_moe_route(l, 2, E, None, T, E, k, 0, True, *got, workspace=ws, workspace_bytes=n - 1)


def test_other_streams_and_graphs():
    torch = torch_cuda()
    T, E, k = 600, 64, 6
    l = logits_of(torch, 8, T, E, "bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.mxfp4_reserve_bytes(mx.mxfp4_moe_route_workspace_bytes(T, E))
        out = mx.moe_route(l, k)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mx.moe_route(l, k, out=out)
    for i in range(4):
        l.copy_(logits_of(torch, 20 + i, T, E, "bf16"))
        want = mx.moe_route(l, k)
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1e-7, 1.0, 1e6, 3e38])
def test_close_sums_and_far_biases(score, scale):
    """Biases so close that f32 estimates cannot tell the sums apart, or so far that they drown the scores."""
    torch = torch_cuda()
    T, E, k = 200, 72, 9
    l = logits_of(torch, 31, T, E, "bf16", 1e-3)
    bias = logits_of(torch, 32, 1, E, "f32", 1.0).reshape(-1).clamp(-1, 1) * scale
    bias[3] = float("inf")
    check(torch, l, k, score, bias, True, "scale %g" % scale)


@pytest.mark.parametrize("T", [20000, 70001])
def test_many_tokens(T):
    torch = torch_cuda()
    check(torch, logits_of(torch, T, T, 40, "bf16"), 3, "sigmoid", torch.linspace(0, 0.1, 40).cuda(), what="many")

"""mxfp4_gemm_grouped against the product in 64 bits on the oracle's quantized
rows: empty, odd and uneven groups, gathered rows, rows of no group, odd N and
K, strides, offsets that are none, streams and graphs."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
import oracle
from tests.expert_util import Weights, assert_within, dequant, product_limit
from tests.gpu_util import bf16_dev_to_bits, torch_cuda

pytestmark = pytest.mark.gpu


def activations(torch, seed, T, K, scale=1.0):
    r = np.random.default_rng(seed)
    return torch.from_numpy((r.standard_normal((T, K)) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def offsets_of(torch, sizes, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32), device="cuda")


def quantized(A):
    """f64 values that the rows of A stand for once quantized."""
    return dequant(*oracle.quantize(bf16_dev_to_bits(A.contiguous())))


def check(C, A, w, sizes, rows=None, repeat=1, gated=False, first=0, what=""):
    a = quantized(A)
    if rows is None:
        src = np.arange(C.shape[0])
    else:
        src = rows.cpu().numpy()
        src = np.where(src < 0, -1, src // repeat)
    ok = (src >= 0) & (src < a.shape[0])
    x = np.where(ok[:, None], a[np.where(ok, src, 0)], 0.0)
    ref = np.zeros(C.shape)
    limit = np.zeros(C.shape)
    at = first
    for e, n in enumerate(sizes):
        if n:
            ref[at:at + n], limit[at:at + n] = product_limit(x[at:at + n], w.values[e], "bf16", gated)
        at += n
    assert_within(C, ref, limit, what)


SIZES = [
    [1], [0, 1, 0], [5, 0, 3, 1], [16, 17, 15], [64, 1, 65], [130, 0, 0, 70, 2], [257, 3], [300, 129, 0, 40, 256, 7],
    [0, 0, 513], [20] * 12,
]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N,K", [(32, 32), (64, 128), (96, 160), (288, 704), (512, 1056), (1056, 288)])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_matches_the_product_in_64_bits(sizes, N, K, gated):
    torch = torch_cuda()
    w = Weights(torch, N + K, len(sizes), N, K)
    A = activations(torch, len(sizes), sum(sizes), K)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N, gated=gated)
    assert C.shape == (sum(sizes), N // 2 if gated else N)
    check(C, A, w, sizes, gated=gated, what=str(sizes))


@pytest.mark.parametrize("N", [16, 48, 272, 528])
def test_odd_groups_of_columns(N):
    torch = torch_cuda()
    sizes = [3, 40, 200]
    w = Weights(torch, N, 3, N, 352)
    A = activations(torch, 1, 243, 352)
    check(mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N), A, w, sizes, what="N %d" % N)


@pytest.mark.parametrize("T,E,k,N,K,gated", [(1, 8, 2, 96, 96, True), (7, 70, 4, 64, 256, False), (50, 5, 3, 160, 224, True),
                                             (400, 6, 2, 512, 512, True), (300, 3, 1, 320, 640, False)])
def test_gathered_by_the_router(T, E, k, N, K, gated):
    torch = torch_cuda()
    w = Weights(torch, T, E, N, K)
    A = activations(torch, 2, T, K)
    r = np.random.default_rng(T)
    logits = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).cuda()
    if T > 1:
        logits[1] = -float("inf")  # a padding token: its rows end up outside every group
    ids, _, offsets, rows, _ = mx.moe_route(logits, k)
    sizes = np.diff(offsets.cpu().numpy())
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets, N, rows=rows, repeat=k, gated=gated)
    check(C, A, w, sizes, rows, k, gated, what="routed")
    if T > 1:
        assert not C[int(offsets[-1]):].any()


def test_rows_of_no_group_and_rows_of_no_token():
    torch = torch_cuda()
    sizes, first, R = [4, 0, 90], 5, 120
    w = Weights(torch, 3, 3, 64, 192)
    A = activations(torch, 4, 30, 192)
    rows = torch.from_numpy(np.random.default_rng(0).integers(0, 60, R).astype(np.int32)).cuda()
    rows[6], rows[20], rows[50] = -1, 60, 1 << 30
    out = torch.full((R, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes, first), 64, rows=rows, repeat=2, out=out)
    assert C is out
    check(C, A, w, sizes, rows, 2, first=first, what="outside")
    assert not C[:5].any() and not C[99:].any() and not C[6].any() and not C[20].any()


def test_all_groups_empty():
    torch = torch_cuda()
    w = Weights(torch, 5, 2, 64, 64)
    A = activations(torch, 6, 40, 64)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full((40, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    assert not mx.gemm_grouped(A, w.Bw, w.Bs, zero, 64, out=out).any()
    assert mx.gemm_grouped(A[:0], w.Bw, w.Bs, zero, 64).shape == (0, 64)
    none = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    assert not mx.gemm_grouped(A[:0], w.Bw, w.Bs, offsets_of(torch, [4, 4]), 64, rows=none).any()


@pytest.mark.parametrize("sizes", [[2, 1], [200, 150]])
def test_one_group_equals_the_gemm_and_the_others_alone(sizes):
    torch = torch_cuda()
    w = Weights(torch, 7, 2, 256, 512)
    A = activations(torch, 8, sum(sizes), 512)
    both = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), 256)
    for e, (lo, hi) in enumerate([(0, sizes[0]), (sizes[0], sum(sizes))]):
        alone = mx.gemm_grouped(A[lo:hi], w.Bw[e], w.Bs[e], offsets_of(torch, [hi - lo]), 256)
        assert torch.equal(both[lo:hi], alone)
        plain = mx.gemm(A[lo:hi].contiguous(), w.Bw[e], w.Bs[e], 256)
        check(plain, A[lo:hi], type("W", (), {"values": [w.values[e]]}), [hi - lo], what="gemm")


@pytest.mark.parametrize("sizes", [[3, 0, 9], [150, 140]])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_strided_rows(sizes, shift):
    torch = torch_cuda()
    N, K, R = 96, 224, sum(sizes)
    w = Weights(torch, 9, len(sizes), N, K)
    A = activations(torch, 10, R, K + 40)[:, 16:16 + K]
    wide = torch.full((R, N + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, shift:shift + N]
    mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N, out=out)
    check(out, A, w, sizes, what="strided")
    assert bool((wide[:, :shift] == 3).all()) and bool((wide[:, shift + N:] == 3).all())


@pytest.mark.parametrize("power", [-60, 60])
def test_scales_far_from_one(power):
    torch = torch_cuda()
    sizes = [5, 130]
    w = Weights(torch, 11, 2, 64, 192, scale=2.0**-power)
    A = activations(torch, 12, 135, 192, scale=2.0**power)
    check(mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), 64), A, w, sizes, what="2^%d" % power)


def test_software_encoder_gives_the_same():
    torch = torch_cuda()
    sizes = [30, 0, 100]
    w = Weights(torch, 13, 3, 128, 320)
    A = activations(torch, 14, 130, 320)
    want = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), 128)
    mx.mxfp4_set_quant_mode(1)
    try:
        got = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), 128)
    finally:
        mx.mxfp4_set_quant_mode(0)
    assert torch.equal(want, got)


def test_matrices_beyond_32_bit_offsets():
    torch = torch_cuda()
    N = K = 8192
    E = (1 << 31) // (N * K // 2) + 2
    small = Weights(torch, 16, 1, N, 64)
    Bw = torch.zeros((E, N // 16, K * 8), dtype=torch.uint8, device="cuda")
    Bs = torch.full((E, N // 32, K), 127, dtype=torch.uint8, device="cuda")
    Bw[E - 1, :, :64 * 8] = small.Bw[0]  # the first 64 of K; the other codes stand for zero
    Bs[E - 1, :, :256] = small.Bs[0].reshape(N // 32, 256)
    for n in (2, 140):
        sizes = [1] + [0] * (E - 2) + [n]
        A = activations(torch, 17, n + 1, K)
        C = mx.gemm_grouped(A, Bw, Bs, offsets_of(torch, sizes), N)
        assert not C[0].any()
        ref, limit = product_limit(quantized(A)[1:, :64], small.values[0], "bf16", False)
        assert_within(C[1:], ref, limit, "last matrix")


def test_a_callers_workspace_gives_the_same():
    torch = torch_cuda()
    sizes = [10, 70, 1]
    N, K, R = 64, 160, 81
    w = Weights(torch, 18, 3, N, K)
    A = activations(torch, 19, R, K)
    off = offsets_of(torch, sizes)
    want = mx.gemm_grouped(A, w.Bw, w.Bs, off, N)
    n = mx.mxfp4_gemm_grouped_workspace_bytes(R, K, 3)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    got = torch.zeros_like(want)
    mx.mxfp4_gemm_grouped(A, K, R, w.Bw, w.Bs, 3, off, None, 1, got, N, R, N, K, False, ws, n)
    assert torch.equal(want, got) and bool((ws[n:] == 255).all())
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        mx.mxfp4_gemm_grouped(A, K, R, w.Bw, w.Bs, 3, off, None, 1, got, N, R, N, K, False, ws, n - 1)


def test_same_bits_every_time_and_on_other_streams():
    torch = torch_cuda()
    sizes = [33, 200, 5]
    w = Weights(torch, 20, 3, 320, 1024)
    A = activations(torch, 21, 238, 1024)
    off = offsets_of(torch, sizes)
    first = mx.gemm_grouped(A, w.Bw, w.Bs, off, 320, gated=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = [mx.gemm_grouped(A, w.Bw, w.Bs, off, 320, gated=True) for _ in range(6)]
    s.synchronize()
    assert all(torch.equal(first, y) for y in again)


@pytest.mark.parametrize("T", [6, 300])
def test_captured_into_a_graph(T):
    torch = torch_cuda()
    E, k, N, K = 4, 2, 128, 256
    w = Weights(torch, 22, E, N, K)
    A = activations(torch, 23, T, K)
    logits = torch.randn((T, E), device="cuda")
    need = max(mx.mxfp4_gemm_grouped_workspace_bytes(T * k, K, E), mx.mxfp4_moe_route_workspace_bytes(T, E))

    def block():
        _, weights, offsets, rows, pos = mx.moe_route(logits, k)
        return mx.moe_combine(mx.gemm_grouped(A, w.Bw, w.Bs, offsets, N, rows=rows, repeat=k), weights, pos=pos)

    block()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    mx.mxfp4_reserve_bytes(need, s)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        out = block()
    for i in range(4):
        A.copy_(activations(torch, 30 + i, T, K))
        logits.copy_(torch.randn((T, E), device="cuda"))
        want = block()
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)

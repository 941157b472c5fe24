"""mxfp4_gemm_grouped with groups of hundreds of rows, so that an expert has
several units: against the product in 64 bits with partial units, uneven and
empty groups, columns past the last tile, both store widths, offsets that are
none, and graphs."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights
from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import activations, check, offsets_of

pytestmark = pytest.mark.gpu

UNEVEN = [0, 1, 255, 256, 257, 64, 65, 128, 129, 191, 193, 900, 700, 1100, 33, 512]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [32, 96, 544, 768, 1568])
def test_k_tails(K, gated):
    torch = torch_cuda()
    E, N = 16, 4096
    w = Weights(torch, K, E, N, K)
    A = activations(torch, K + 1, sum(UNEVEN), K)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, UNEVEN), N, gated=gated)
    check(C, A, w, UNEVEN, gated=gated, what="K %d" % K)


@pytest.mark.parametrize("gated,N", [(False, 4128), (False, 4256), (False, 4320), (True, 4160), (True, 4288), (True, 4032)])
def test_columns_past_the_last_tile(gated, N):
    torch = torch_cuda()
    E, K = 16, 192
    w = Weights(torch, N, E, N, K)
    A = activations(torch, N, sum(UNEVEN), K)
    cols = N // 2 if gated else N
    for extra, shift in ((0, 0), (8, 0), (3, 1)):  # rows of 16 bytes, and rows that are not
        wide = torch.full((sum(UNEVEN), cols + extra), 5.0, dtype=torch.bfloat16, device="cuda")
        out = wide[:, shift:shift + cols]
        mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, UNEVEN), N, gated=gated, out=out)
        check(out, A, w, UNEVEN, gated=gated, what="N %d, stride + %d" % (N, extra))
        assert bool((wide[:, :shift] == 5).all()) and bool((wide[:, shift + cols:] == 5).all())


@pytest.mark.parametrize("gated", [False, True])
def test_gathered_rows_and_rows_of_no_token(gated):
    torch = torch_cuda()
    E, N, K, k, T = 8, 4096, 160, 4, 1500
    w = Weights(torch, 7, E, N, K)
    A = activations(torch, 8, T, K)
    logits = torch.from_numpy(np.random.default_rng(9).standard_normal((T, E)).astype(np.float32)).cuda()
    logits[::9] = -float("inf")
    _, _, offsets, rows, _ = mx.moe_route(logits, k)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets, N, rows=rows, repeat=k, gated=gated)
    check(C, A, w, np.diff(offsets.cpu().numpy()), rows, k, gated, what="routed")
    assert not C[int(offsets[-1]):].any()
    few = mx.gemm_grouped(A[:300], w.Bw, w.Bs, offsets, N, rows=rows, repeat=k, gated=gated)
    check(few, A[:300], w, np.diff(offsets.cpu().numpy()), rows, k, gated, what="rows of no token")


@pytest.mark.parametrize("gated", [False, True])
def test_more_tiles_than_workgroups_and_other_work_between(gated):
    torch = torch_cuda()
    E, N, K = 16, 8192, 1056
    sizes = (np.array(UNEVEN) * 2).tolist()
    w = Weights(torch, 12, E, N, K)
    A = activations(torch, 13, sum(sizes), K)
    off = offsets_of(torch, sizes)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated)
    at = np.concatenate([[0], np.cumsum(sizes)])
    for e in (1, 4, 11, 14):
        lo, hi = int(at[e]), int(at[e + 1])
        check(C[lo:hi], A[lo:hi], type("W", (), {"values": [w.values[e]]}), [hi - lo], gated=gated, what="group %d" % e)
    for n in (1, 40, 4000):
        mx.gemm_grouped(A[:n], w.Bw, w.Bs, off.clamp(max=n), N, gated=gated)
        assert torch.equal(C, mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated))


@pytest.mark.parametrize("R", [2048, 2055])
@pytest.mark.parametrize("kind", ["falling", "beyond", "below", "repeated"])
def test_offsets_that_are_none_touch_nothing_else(R, kind):
    """They give rows without meaning, inside C and the workspace."""
    torch = torch_cuda()
    E, N, K = 8, 4096, 96
    w = Weights(torch, 19, E, N, K)
    A = activations(torch, 20, R, K)
    off = torch.linspace(0, R, E + 1).to(torch.int32)
    if kind == "falling":
        off = off.flip(0)
    elif kind == "beyond":
        off = off * 3 + 1000
    elif kind == "below":
        off = off - R // 2
    else:
        off[::2] = 0
        off[1::2] = R  # every second group claims all rows
    n = mx.mxfp4_gemm_grouped_workspace_bytes(R, K, E)
    ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
    big = torch.full((R + 16, N), 3.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_gemm_grouped(A, K, R, w.Bw, w.Bs, E, off.cuda(), None, 1, big[8:8 + R], N, R, N, K, False, ws, n)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 255).all()) and bool((big[:8] == 3).all()) and bool((big[8 + R:] == 3).all())


@pytest.mark.parametrize("gated", [False, True])
def test_captured_into_a_graph(gated):
    torch = torch_cuda()
    E, N, K, R = 8, 4096, 352, 2100
    w = Weights(torch, 21, E, N, K)
    A = activations(torch, 22, R, K)
    off = offsets_of(torch, [300, 0, 500, 256, 44, 600, 0, 400])
    mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated)
    for seed in range(3):
        A.copy_(activations(torch, seed, R, K))
        off.copy_(offsets_of(torch, [100 * seed, 256, 3, 0, 700, 1, R - 960 - 100 * seed, 0]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated)), seed

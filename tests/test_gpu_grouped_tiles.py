"""The 128-row tiles of mxfp4_gemm_grouped (many groups, wide enough matrices)
against the product in 64 bits: every K tail, partial units, uneven and empty
groups, columns past the last tile, both store widths, more tiles than
workgroups, and offsets that are none."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights
from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import activations, check, offsets_of

pytestmark = pytest.mark.gpu


def uneven(seed, E, mean):
    """E group sizes around the mean, among them empty ones, one row and the tile borders."""
    r = np.random.default_rng(seed)
    n = np.maximum(0, (r.exponential(mean, E))).astype(int)
    n[:8] = [0, 1, 127, 128, 129, 64, 33, 0]
    n[8] += mean * 4
    r.shuffle(n)
    return n.tolist()


# every shape below meets the tiles' rule: 32 rows a group and 256 tiles
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 256, 288, 384, 416, 512, 544, 640, 1056])
def test_every_k_tail(K, gated):
    torch = torch_cuda()
    E, N = 64, 1024
    sizes = uneven(K, E, 40)
    w = Weights(torch, K, E, N, K)
    A = activations(torch, K + 1, sum(sizes), K)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N, gated=gated)
    check(C, A, w, sizes, gated=gated, what="K %d" % K)


@pytest.mark.parametrize("gated,N", [(False, 1056), (False, 1312), (False, 1248), (True, 1088), (True, 1216), (True, 1984)])
def test_columns_past_the_last_tile(gated, N):
    torch = torch_cuda()
    E, K = 64, 192
    sizes = uneven(N, E, 45)
    w = Weights(torch, N, E, N, K)
    A = activations(torch, N, sum(sizes), K)
    cols = N // 2 if gated else N
    for extra, shift in ((0, 0), (8, 0), (3, 1)):  # rows of 16 bytes, and rows that are not
        wide = torch.full((sum(sizes), cols + extra), 5.0, dtype=torch.bfloat16, device="cuda")
        out = wide[:, shift:shift + cols]
        mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N, gated=gated, out=out)
        check(out, A, w, sizes, gated=gated, what="N %d, stride + %d" % (N, extra))
        assert bool((wide[:, :shift] == 5).all()) and bool((wide[:, shift + cols:] == 5).all())


@pytest.mark.parametrize("gated", [False, True])
def test_gathered_rows_and_rows_of_no_token(gated):
    torch = torch_cuda()
    E, N, K, k, T = 64, 2048, 160, 4, 700
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
def test_more_tiles_than_workgroups(gated):
    torch = torch_cuda()
    E, N, K = 96, 4096, 64
    sizes = uneven(11, E, 60)
    w = Weights(torch, 12, E, N, K)
    A = activations(torch, 13, sum(sizes), K)
    off = offsets_of(torch, sizes)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated)
    check(C, A, w, sizes, gated=gated, what="many tiles")
    for _ in range(3):
        assert torch.equal(C, mx.gemm_grouped(A, w.Bw, w.Bs, off, N, gated=gated))


def test_one_group_takes_all():
    torch = torch_cuda()
    E, N, K = 2, 4096, 256
    for sizes in ([5000, 0], [0, 4999], [1, 5000]):
        w = Weights(torch, 14, E, N, K)
        A = activations(torch, 15, sum(sizes), K)
        check(mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N), A, w, sizes, what=str(sizes))


def test_the_same_as_units_of_16_rows():
    """A group's rows do not depend on the other groups, nor on which form ran."""
    torch = torch_cuda()
    E, N, K = 64, 1024, 384
    sizes = uneven(16, E, 40)
    w = Weights(torch, 17, E, N, K)
    A = activations(torch, 18, sum(sizes), K)
    C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, sizes), N)
    at = np.concatenate([[0], np.cumsum(sizes)])
    for e in (int(np.argmax(sizes)), 3, 50):
        if sizes[e]:
            lo, hi = int(at[e]), int(at[e + 1])
            alone = mx.gemm_grouped(A[lo:hi], w.Bw[e], w.Bs[e], offsets_of(torch, [hi - lo]), N)
            one = type("W", (), {"values": [w.values[e]]})
            check(alone, A[lo:hi], one, [hi - lo], what="alone")
            check(C[lo:hi], A[lo:hi], one, [hi - lo], what="among others")


@pytest.mark.parametrize("E,R,N", [(3, 40, 64), (64, 2560, 1024)])
@pytest.mark.parametrize("kind", ["falling", "beyond", "below", "repeated"])
def test_offsets_that_are_none_touch_nothing_else(E, R, N, kind):
    """They give rows without meaning, inside C and the workspace."""
    torch = torch_cuda()
    K = 96
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

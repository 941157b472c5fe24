"""A workspace of the caller's: the same results as with the library's, no
bytes touched outside it, one too small is refused, and graphs captured on one
stream with a workspace each replay on two streams at once."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights
from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import activations, offsets_of

pytestmark = pytest.mark.gpu


def job(torch, seed, sizes, N=96, K=160, T=400, E=12):
    w = Weights(torch, seed, len(sizes), N, K)
    A = activations(torch, seed + 1, sum(sizes), K)
    off = offsets_of(torch, sizes)
    logits = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32)).cuda()
    need = mx.mxfp4_gemm_grouped_workspace_bytes(sum(sizes), K, len(sizes)), mx.mxfp4_moe_route_workspace_bytes(T, E)

    def call(ws=(None, None)):
        return (mx.gemm_grouped(A, w.Bw, w.Bs, off, N, workspace=ws[0]), *mx.moe_route(logits, 3, workspace=ws[1]))

    return call, need


def test_same_results_and_nothing_outside():
    torch = torch_cuda()
    call, need = job(torch, 1, [3, 0, 200, 41])
    whole = [torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda") for n in need]
    got = call([w[256:256 + n] for w, n in zip(whole, need)])
    for a, b in zip(call(), got):
        assert torch.equal(a, b)
    for w, n in zip(whole, need):
        assert bool((w[:256] == 0xA5).all()) and bool((w[256 + n:] == 0xA5).all())
        assert not bool((w[256:256 + n] == 0xA5).all())


def test_too_small_is_refused():
    torch = torch_cuda()
    call, need = job(torch, 2, [30, 34])
    for i in range(2):
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
        ws[i] = ws[i][:-1]
        with pytest.raises(RuntimeError, match="WORKSPACE"):
            call(ws)


def test_graphs_of_one_stream_replay_at_once():
    torch = torch_cuda()
    stream = torch.cuda.Stream()
    graphs, outs, eager, kept = [], [], [], []
    for seed, sizes in ((3, [300, 20, 7]), (4, [9] * 24)):
        call, need = job(torch, seed, sizes)
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
        kept.append((call, ws))  # a graph reads its inputs and its workspace where they were
        eager.append(call(ws))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append([call(ws) for _ in range(8)])
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        torch.cuda.synchronize()
        for o in outs:
            for r in o:
                for t in r:
                    t.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for e, o in zip(eager, outs):
            for r in o:
                for a, b in zip(e, r):
                    assert torch.equal(a, b)

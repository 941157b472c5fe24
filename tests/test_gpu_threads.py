"""Several host threads on one stream, and each on its per-thread stream: every
call's result is the one it has alone, though the two launches of the grouped
product and of the router hand their data on through a workspace."""
import threading

import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.expert_util import Weights
from tests.gpu_util import torch_cuda
from tests.test_gpu_grouped import activations, offsets_of

pytestmark = pytest.mark.gpu


PER_THREAD = 2  # hipStreamPerThread


@pytest.mark.parametrize("stream", [None, PER_THREAD])
def test_threads_call_at_once(stream):
    torch = torch_cuda()
    N, K, calls = 96, 160, 60
    jobs = []
    for i, sizes in enumerate(([3, 0, 40, 7], [300, 1], [20] * 16, [0, 0, 90])):
        w = Weights(torch, i, len(sizes), N, K)
        A = activations(torch, 10 + i, sum(sizes), K)
        off = offsets_of(torch, sizes)
        logits = torch.from_numpy(np.random.default_rng(20 + i).standard_normal((150 + 90 * i, 8 + i)).astype(np.float32)).cuda()

        def job(outs=None, A=A, w=w, off=off, logits=logits):
            outs = outs or (None, None)
            return (mx.gemm_grouped(A, w.Bw, w.Bs, off, N, out=outs[0], stream=stream),
                    *mx.moe_route(logits, 3, out=outs[1], stream=stream))

        jobs.append(job)
    torch.cuda.synchronize()
    alone = [job() for job in jobs]
    # of each call, made before: another stream writes them
    outs = [[(torch.empty_like(a[0]), tuple(map(torch.empty_like, a[1:]))) for _ in range(calls)] for a in alone]
    torch.cuda.synchronize()
    results = [[] for _ in jobs]
    start = threading.Barrier(len(jobs))

    def work(i):
        start.wait()
        for n in range(calls):
            results[i].append(jobs[i](outs[i][n]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, got in enumerate(results):
        assert len(got) == calls
        for n, r in enumerate(got):
            for a, b in zip(alone[i], r):
                assert torch.equal(a, b), "thread %d, call %d" % (i, n)

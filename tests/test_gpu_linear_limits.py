"""The dense layer and its gradients at the ends of their ranges, and called by several threads at once."""
import threading

import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.linear_util import Matrix, assert_within, grad_pre_limit, linear_limit, product_limit, quantized, rows

pytestmark = pytest.mark.gpu


def test_most_rows():
    M, N, K = 1 << 20, 64, 32
    w = Matrix(1, N, K)
    x, dz = rows(2, M, K), rows(3, M, N, "bf16", 0.1)
    want_y, want_z = linear_limit(x, w.values, "bf16", None, "silu", True)
    y, z = mx.linear(x, w.Bw, w.Bs, N, activation="silu", gated=True, pre=True)
    assert_within(y, want_y, "y")
    assert_within(z, want_z, "pre")
    assert_within(mx.linear_grad_input(dz, w.Bw, w.Bs, K), product_limit(dz, w.values, "bf16"), "dx")
    assert_within(mx.linear_grad_weight(dz, x), product_limit(dz.t().contiguous(), quantized(x), "f32"), "dw")
    dy = rows(4, M, N // 2, "bf16", 0.1)
    want_dz, want_db = grad_pre_limit(dy, z, "silu", True)
    got, db = mx.linear_grad_pre(dy, z, activation="silu", gated=True, bias=True, out=z)
    assert_within(got, want_dz, "dz")
    assert_within(db, want_db, "dbias")
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        mx.linear(torch.empty((M + 1, K), dtype=torch.bfloat16, device="cuda"), w.Bw, w.Bs, N)


@pytest.mark.parametrize("M", [1, 3, 40, 200])
def test_most_columns(M):
    N, K = 1 << 20, 32
    w = Matrix(5, N, K)
    x, dz = rows(6, M, K), rows(7, M, N, "bf16", 0.1)
    want, _ = linear_limit(x, w.values, "bf16")
    assert_within(mx.linear(x, w.Bw, w.Bs, N), want, "y")
    assert_within(mx.linear_grad_input(dz, w.Bw, w.Bs, K), product_limit(dz, w.values, "bf16"), "dx")
    assert_within(mx.linear_grad_weight(dz, x, out_dtype=torch.bfloat16),
                  product_limit(dz.t().contiguous(), quantized(x), "bf16"), "dw")


@pytest.mark.parametrize("M", [1, 20, 300])
def test_largest_k(M):
    N, K = 48, 1 << 17
    w = Matrix(8, N, K)
    x, dz = rows(9, M, K), rows(10, M, N, "bf16", 0.1)
    want, _ = linear_limit(x, w.values, "f32")
    assert_within(mx.linear(x, w.Bw, w.Bs, N, out_dtype=torch.float32), want, "y")
    assert_within(mx.linear_grad_input(dz, w.Bw, w.Bs, K), product_limit(dz, w.values, "bf16"), "dx")
    assert_within(mx.linear_grad_weight(dz, x), product_limit(dz.t().contiguous(), quantized(x), "f32"), "dw")


def test_rows_far_apart():
    """Row strides of 2^20 elements, the largest: rows of x, dz, residual and outputs within one buffer each."""
    M, N, K, far = 260, 64, 96, 1 << 20
    w = Matrix(11, N, K)

    def spread(t):
        whole = torch.empty(((t.shape[0] - 1) * far + t.shape[1],), dtype=t.dtype, device="cuda")
        view = whole.as_strided(t.shape, (far, 1))
        view.copy_(t)
        return view

    x, dz, r = spread(rows(12, M, K)), spread(rows(13, M, N, "bf16", 0.1)), spread(rows(14, M, N, "f32"))
    y, z = spread(torch.zeros((M, N), device="cuda")), spread(torch.zeros((M, N), dtype=torch.bfloat16, device="cuda"))
    want_y, want_z = linear_limit(x, w.values, "f32", None, "gelu", False, r)
    mx.linear(x, w.Bw, w.Bs, N, activation="gelu", residual=r, pre=z, out=y)
    assert_within(y, want_y, "y")
    assert_within(z, want_z, "pre")
    dx = spread(torch.zeros((M, K), device="cuda"))
    assert_within(mx.linear_grad_input(dz, w.Bw, w.Bs, K, out=dx), product_limit(dz, w.values, "f32"), "dx")
    dw = spread(torch.zeros((N, K), device="cuda"))
    assert_within(mx.linear_grad_weight(dz, x, out=dw), product_limit(dz.t().contiguous(), quantized(x), "f32"), "dw")
    want_dz, want_db = grad_pre_limit(r, z, "gelu")
    got, db = mx.linear_grad_pre(r, z, activation="gelu", bias=True, out=dz)
    assert_within(got, want_dz, "dz")
    assert_within(db, want_db, "dbias")


def test_threads_on_one_stream():
    """Calls of two and three launches that hand data on through the stream's workspace, by four threads at once."""
    N, K = 512, 512
    w = Matrix(21, N, K)
    inputs = [(rows(30 + i, 100 + 60 * i, K), rows(40 + i, 100 + 60 * i, N, "bf16", 0.1)) for i in range(4)]

    def step(x, dz):
        return (mx.linear(x, w.Bw, w.Bs, N, activation="silu"), mx.linear_grad_input(dz, w.Bw, w.Bs, K),
                mx.linear_grad_weight(dz, x), mx.linear_grad_pre(dz, None, bias=True)[1])

    want = [step(*i) for i in inputs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)
    stream = torch.cuda.current_stream()

    def work(i):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(30):
                got = step(*inputs[i])
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_two_graphs_with_workspaces_of_their_own():
    """Graphs captured on one stream and replayed on two at the same time."""
    N, K, M = 1024, 512, 200
    w = Matrix(22, N, K)
    need = max(mx.mxfp4_linear_workspace_bytes(M, N, K), mx.mxfp4_linear_grad_weight_workspace_bytes(M, N, K))
    stream, graphs = torch.cuda.Stream(), []
    for i in range(2):
        x, dz = rows(50 + i, M, K), rows(60 + i, M, N, "bf16", 0.1)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        want = mx.linear(x, w.Bw, w.Bs, N), mx.linear_grad_weight(dz, x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(20):
                out = mx.linear(x, w.Bw, w.Bs, N, workspace=ws), mx.linear_grad_weight(dz, x, workspace=ws)
        graphs.append((graph, out, want, torch.cuda.Stream(), x, dz, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, out, _, side, *_ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, want, *_ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
            for t in out:
                t.zero_()
        torch.cuda.synchronize()

"""The dense layer and its input's gradient on a prepared matrix of nearly 2^31 bytes, whose last column tile has groups past the end."""
import pytest

torch = pytest.importorskip("torch")

import block_scaled_mxfp4_bf16_amd as mx
from tests.linear_util import assert_within, quantized, rounded, rows

pytestmark = pytest.mark.gpu

N, K = 1040432, 4128  # 65027 groups of 33024 bytes: 2^31 - 32000; 16 rows more would be beyond
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


class Largest:
    """Random codes and scale bytes, laid out on the device; values(first, last) are those of some rows in f64."""

    def __init__(self):
        g = torch.Generator(device="cuda")
        g.manual_seed(3)
        G, gp = K // 32, (K // 32 + 7) // 8 * 8
        padded = (N + 255) // 256 * 256
        self.Bw = torch.randint(0, 256, (N // 16, K * 8), generator=g, device="cuda", dtype=torch.uint8)
        self.scales = torch.randint(118, 124, (N, G), generator=g, device="cuda", dtype=torch.uint8)
        pad = torch.full((padded, gp), 127, dtype=torch.uint8, device="cuda")
        pad[:N, :G] = self.scales
        self.Bs = pad.view(padded // 32, 2, 16, gp // 8, 2, 4).permute(0, 3, 5, 2, 4, 1).reshape(padded // 32, gp * 32).contiguous()

    def values(self, first, last):
        b = self.Bw[first // 16:last // 16].view(-1, K // 32, 16, 16)  # group, K chunk of 32, row, byte
        b = b.permute(0, 2, 1, 3).reshape(last - first, K // 2)
        table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device="cuda")
        code = torch.stack([b & 15, b >> 4], -1).reshape(last - first, K)
        return table[code.int()] * torch.exp2(self.scales[first:last].double() - 127).repeat_interleave(32, 1)


@pytest.fixture(scope="module")
def largest():
    m = Largest()
    assert m.Bw.nbytes < 2**31 < m.Bw.nbytes + K * 8
    yield m
    del m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [1, 20, 80])
def test_layer(largest, M):
    """One row quantized on the way, 20 before; 80 in the large tiles, the last of which ends within 256 columns."""
    x = rows(5, M, K)
    y = mx.linear(x, largest.Bw, largest.Bs, N)
    q = quantized(x)
    for first in range(0, N, 65536):
        last = min(N, first + 65536)
        w = largest.values(first, last)
        z = q @ w.t()
        assert_within(y[:, first:last], (z, rounded(z, K * 2.0**-23 * (q.abs() @ w.abs().t()), "bf16")), "y from %d" % first)


@pytest.mark.parametrize("M", [3, 140])
def test_input_gradient(largest, M):
    """Rows that are zero but for 64 columns, the first and the last among them: 64 terms a sum, the others add nothing."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    at = torch.randint(0, N, (64,), generator=g, device="cuda")
    at[:4] = torch.tensor([0, N - 1, N - 16, N - 17], device="cuda")
    at = at.unique()
    dz = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dz[:, at] = torch.randn((M, at.numel()), generator=g, device="cuda").to(torch.bfloat16)
    dx = mx.linear_grad_input(dz, largest.Bw, largest.Bs, K, out_dtype=torch.float32)
    w = torch.cat([largest.values(n // 16 * 16, n // 16 * 16 + 16)[n % 16:n % 16 + 1] for n in at.tolist()])
    p = dz[:, at].double()
    assert_within(dx, (p @ w, rounded(p @ w, at.numel() * 2.0**-23 * (p.abs() @ w.abs()), "f32")), "dx")

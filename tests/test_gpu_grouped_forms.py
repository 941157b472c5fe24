"""Which bits of a grouped product depend on what: a group's rows have the
same ones whatever the other groups hold, as long as the number of rows and of
groups is the same; the two forms of the product (16-row units with K split
over four waves, 128-row tiles with one sum along K), chosen by those numbers, add
in different orders and agree within both sums' error."""
import numpy as np
import pytest

import block_scaled_mxfp4_bf16_amd as mx
import oracle
from tests.expert_util import HALF_STEP, SMALLEST, Weights, assert_within, dequant, gated as gate
from tests.gpu_util import bf16_dev_to_bits, torch_cuda
from tests.test_gpu_grouped import activations, offsets_of

pytestmark = pytest.mark.gpu


def both_sums_limit(x, w, is_gated):
    """How far two f32 sums of the same products, in any orders and rounded
    once to bf16 each, can be apart: twice K * 2^-23 * sum |x w| (through the gate
    as its slope of at most 1.1 and its own (|g| + 8) * 2^-22 pass it on), and half a
    step of bf16 each."""
    ref = x @ w.T
    err = w.shape[1] * 2.0**-23 * (np.abs(x) @ np.abs(w).T)
    if is_gated:
        n = ref.shape[1] // 2
        g, u, eg, eu = ref[:, :n], ref[:, n:], err[:, :n], err[:, n:]
        ref = gate(ref)
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(g / (1 + np.exp(-g))) * eu + (np.abs(g) + 8) * 2.0**-22 * np.abs(ref)
    return 2 * (err + HALF_STEP["bf16"] * (np.abs(ref) + err) + SMALLEST["bf16"])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [96, 384, 1056])
def test_the_two_forms_agree_within_their_error(K, gated):
    torch = torch_cuda()
    E, N, n = 64, 1024, 40
    w = Weights(torch, K, E, N, K)
    A = activations(torch, K + 1, E * n, K)
    tiles = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, [n] * E), N, gated=gated)
    x = dequant(*oracle.quantize(bf16_dev_to_bits(A)))
    for e in (0, 31, 63):  # one group at a time is far from a tile for every CU
        lo = e * n
        alone = mx.gemm_grouped(A[lo:lo + n], w.Bw[e], w.Bs[e], offsets_of(torch, [n]), N, gated=gated)
        assert_within(alone, tiles[lo:lo + n].double().cpu().numpy(), both_sums_limit(x[lo:lo + n], w.values[e], gated),
                      "group %d" % e)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("E,N,sizes,others", [
    (64, 1024, [40] * 64, [1, 79] * 16 + [40] + [122, 0, 0] * 10 + [20]),  # tiles
    (6, 96, [5, 0, 37, 21, 1, 8], [0, 21, 37, 5, 8, 1]),                   # 16-row units
])
def test_a_groups_bits_do_not_depend_on_the_other_groups(E, N, sizes, others, gated):
    torch = torch_cuda()
    K, group = 416, 32 if E == 64 else 2
    assert len(others) == E and sum(others) == sum(sizes) and others[group] == sizes[group]
    w = Weights(torch, E, E, N, K)
    rows = activations(torch, 5, sizes[group], K)
    got = []
    for seed, s in ((6, sizes), (7, others)):
        A = activations(torch, seed, sum(s), K)
        lo = sum(s[:group])
        A[lo:lo + s[group]] = rows
        C = mx.gemm_grouped(A, w.Bw, w.Bs, offsets_of(torch, s), N, gated=gated)
        got.append(C[lo:lo + s[group]])
    assert torch.equal(*got)

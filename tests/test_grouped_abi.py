"""The grouped product rejects bad arguments on the host, before any HIP call
(no GPU is needed for these checks)."""
import pytest

import block_scaled_mxfp4_bf16_amd as mx

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 1 << 20  # an aligned non-null address; never dereferenced (checks fail first)

GROUPED = dict(A=FAKE, lda=64, a_rows=10, Bq=FAKE, Bs=FAKE, experts=4, offsets=FAKE, rows=None, repeat=1, C=FAKE, ldc=96,
               R=10, N=96, K=64, gated=0, ws=None, ws_bytes=0)


def call(**change):
    args = dict(GROUPED)
    assert set(change) <= set(args)
    args.update(change)
    return mx.lib().mxfp4_gemm_grouped(*args.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(A=None), INVALID), (dict(Bq=None), INVALID), (dict(Bs=None), INVALID), (dict(offsets=None), INVALID),
    (dict(C=None), INVALID), (dict(R=-1), INVALID), (dict(a_rows=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(experts=0), INVALID), (dict(repeat=0), INVALID), (dict(lda=63), INVALID),
    (dict(lda=68), INVALID), (dict(ldc=95), INVALID), (dict(gated=1, ldc=47), INVALID), (dict(A=FAKE + 8), INVALID),
    (dict(Bq=FAKE + 8), INVALID), (dict(Bs=FAKE + 8), INVALID), (dict(offsets=FAKE + 2), INVALID),
    (dict(rows=FAKE + 2), INVALID), (dict(C=FAKE + 1), INVALID),
    (dict(K=48), UNSUPPORTED), (dict(N=90), UNSUPPORTED), (dict(N=80, gated=1), UNSUPPORTED),
    (dict(R=(1 << 20) + 1), UNSUPPORTED), (dict(a_rows=(1 << 20) + 1), UNSUPPORTED), (dict(experts=4097), UNSUPPORTED),
    (dict(repeat=1 << 31), UNSUPPORTED), (dict(lda=1 << 31), UNSUPPORTED), (dict(ldc=1 << 31), UNSUPPORTED),
    (dict(N=1 << 40, ldc=1 << 40), UNSUPPORTED), (dict(K=1 << 40, lda=1 << 40), UNSUPPORTED),
    (dict(ws=FAKE, ws_bytes=100), WORKSPACE), (dict(ws=FAKE + 16, ws_bytes=1 << 30), WORKSPACE),
])
def test_grouped_refuses(change, code):
    assert call(**change) == code


def test_no_rows_is_no_work():
    assert call(R=0, C=None, a_rows=0, A=None) == 0


def test_workspace_size():
    assert mx.mxfp4_gemm_grouped_workspace_bytes(0, 64, 4) == 0
    assert mx.mxfp4_gemm_grouped_workspace_bytes(1, 1 << 40, 4) == 0
    # one quad of 64 rows and one K step: 4096 bytes of codes, 256 of scales
    assert mx.mxfp4_gemm_grouped_workspace_bytes(1, 64, 4) >= 4096 + 256
    assert mx.mxfp4_gemm_grouped_workspace_bytes(256, 2048, 64) >= 64 * 16 * (4096 + 256)


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    A = torch.zeros((6, 64), dtype=torch.bfloat16)
    Bw = torch.zeros((2, 64 * 16), dtype=torch.uint8)
    Bs = torch.zeros((2, 256 * 8), dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        mx.gemm_grouped(A.half(), Bw, Bs, off, 32)
    with pytest.raises(TypeError):
        mx.gemm_grouped(A, Bw, Bs, off, 32, out=torch.zeros((6, 32)))
    for kw in (dict(offsets=off[:2]), dict(offsets=off.long()), dict(Bw=Bw[:1]), dict(A=A.t()), dict(A=A[0]),
               dict(rows=torch.zeros(6, dtype=torch.int64)), dict(out=torch.zeros((5, 32), dtype=torch.bfloat16))):
        args = dict(A=A, Bw=Bw, Bs=Bs, offsets=off, N=32)
        args.update(kw)
        with pytest.raises(ValueError):
            mx.gemm_grouped(**args)
    with pytest.raises(ValueError, match="cuda"):
        mx.gemm_grouped(A, Bw, Bs, off, 32)

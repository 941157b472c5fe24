"""The expert operators reject bad arguments on the host, before any HIP call
(no GPU is needed for these checks)."""
import pytest

import block_scaled_mxfp4_bf16_amd as mx

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 1 << 20  # an aligned non-null address; never dereferenced (checks fail first)

GEMV = dict(x=FAKE, x_type=0, ldx=512, Bq=FAKE, Bs=FAKE, ids=None, experts=1, y=FAKE, y_type=0, ldy=256, M=1, N=256,
            K=512, repeat=1, gated=0)


def call(name, base, **change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(mx.lib(), name)(*args.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), INVALID), (dict(Bq=None), INVALID), (dict(Bs=None), INVALID), (dict(y=None), INVALID),
    (dict(x_type=3), INVALID), (dict(x_type=-1), INVALID), (dict(y_type=7), INVALID),
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(M=-4), INVALID),
    (dict(experts=0), INVALID), (dict(repeat=0), INVALID), (dict(repeat=2), INVALID),
    (dict(ldx=511), INVALID), (dict(ldx=520 + 4), INVALID), (dict(ldy=255), INVALID), (dict(gated=1, ldy=127), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(Bq=FAKE + 8), INVALID), (dict(Bs=FAKE + 4), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(y_type=2, y=FAKE + 2), INVALID), (dict(ids=FAKE + 2), INVALID),
    (dict(K=496), UNSUPPORTED), (dict(N=250, ldy=250), UNSUPPORTED), (dict(N=240, gated=1), UNSUPPORTED),
    (dict(M=(1 << 20) + 1), UNSUPPORTED), (dict(ids=FAKE, repeat=1 << 33), UNSUPPORTED),
    (dict(ids=FAKE, experts=1 << 40), UNSUPPORTED),
    (dict(K=1 << 20, ldx=1 << 20, N=1 << 13, ldy=1 << 13), UNSUPPORTED),
    (dict(K=1 << 62, ldx=1 << 62), UNSUPPORTED), (dict(N=1 << 62, ldy=1 << 62), UNSUPPORTED),
    (dict(ldx=1 << 26), UNSUPPORTED),
])
def test_gemv_refuses(change, code):
    assert call("mxfp4_gemv", GEMV, **change) == code


def test_gemv_binding_refuses():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    Bw = torch.zeros((2, 64 * 8), dtype=torch.uint8)
    Bs = torch.zeros((8, 256), dtype=torch.uint8)
    with pytest.raises(TypeError):
        mx.gemv(x.double(), Bw, Bs, 32)
    with pytest.raises(ValueError):
        mx.gemv(x, Bw[:1], Bs, 32)
    with pytest.raises(ValueError):
        mx.gemv(x, Bw, Bs[:1], 32)
    with pytest.raises(ValueError):
        mx.gemv(x.t(), Bw, Bs, 32)
    with pytest.raises(ValueError):
        mx.gemv(x, torch.cat([Bw, Bw]), torch.cat([Bs, Bs]), 32)  # two matrices, no ids
    with pytest.raises(ValueError):
        mx.gemv(x, Bw, Bs, 32, ids=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        mx.gemv(x, Bw, Bs, 32, ids=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        mx.gemv(x, Bw, Bs, 32, out=torch.zeros((2, 31), dtype=torch.bfloat16))

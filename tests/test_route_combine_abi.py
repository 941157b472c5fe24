"""The router and the combination reject bad arguments on the host, before any
HIP call (no GPU is needed for these checks)."""
import pytest

import block_scaled_mxfp4_bf16_amd as mx

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
FAKE = 1 << 20  # an aligned non-null address; never dereferenced (checks fail first)

ROUTE = dict(logits=FAKE, x_type=0, ld=64, bias=None, T=500, E=64, k=8, score=0, renorm=1, ids=FAKE, weights=FAKE,
             offsets=FAKE, rows=FAKE, pos=FAKE, ws=None, ws_bytes=0)
COMBINE = dict(y=FAKE, y_type=0, ld_y=64, rows=8, weights=FAKE, pos=None, residual=None, ld_res=64, out=FAKE, out_type=0,
               ld_out=64, T=4, k=2, N=64)


def call(name, base, **change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(mx.lib(), name)(*args.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(offsets=None), INVALID), (dict(rows=None), INVALID), (dict(pos=None), INVALID),
    (dict(x_type=3), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(T=-1), INVALID),
    (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(ld=63), INVALID),
    (dict(logits=FAKE + 1), INVALID), (dict(x_type=2, logits=FAKE + 2), INVALID), (dict(bias=FAKE + 2), INVALID),
    (dict(ids=FAKE + 1), INVALID), (dict(weights=FAKE + 2), INVALID), (dict(offsets=FAKE + 2), INVALID),
    (dict(rows=FAKE + 1), INVALID), (dict(pos=FAKE + 3), INVALID),
    (dict(E=1025, ld=1025), UNSUPPORTED), (dict(k=33), UNSUPPORTED), (dict(T=(1 << 20) + 1), UNSUPPORTED),
    (dict(ld=1 << 62), UNSUPPORTED),
    (dict(ws=FAKE, ws_bytes=0), WORKSPACE), (dict(ws=FAKE + 64, ws_bytes=1 << 20), WORKSPACE),
])
def test_route_refuses(change, code):
    assert call("mxfp4_moe_route", ROUTE, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(y=None), INVALID), (dict(weights=None), INVALID), (dict(out=None), INVALID), (dict(y_type=3), INVALID),
    (dict(out_type=-1), INVALID), (dict(T=-1), INVALID), (dict(rows=-1), INVALID), (dict(N=0), INVALID),
    (dict(k=0), INVALID), (dict(ld_y=63), INVALID), (dict(ld_out=63), INVALID), (dict(residual=FAKE, ld_res=63), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(out=FAKE + 1), INVALID), (dict(out_type=2, out=FAKE + 2), INVALID),
    (dict(residual=FAKE + 1), INVALID), (dict(weights=FAKE + 2), INVALID), (dict(pos=FAKE + 2), INVALID),
    (dict(N=1 << 31, ld_y=1 << 31, ld_out=1 << 31), UNSUPPORTED), (dict(k=(1 << 20) + 1), UNSUPPORTED),
    (dict(T=1 << 40), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED), (dict(ld_y=1 << 62), UNSUPPORTED),
])
def test_combine_refuses(change, code):
    assert call("mxfp4_moe_combine", COMBINE, **change) == code


def test_combine_of_no_tokens_needs_no_buffers():
    assert call("mxfp4_moe_combine", COMBINE, T=0, y=None, weights=None, out=None) == 0


def test_workspace_size():
    assert mx.mxfp4_moe_route_workspace_bytes(1, 64) == 0
    assert 0 < mx.mxfp4_moe_route_workspace_bytes(8192, 128) <= 1 << 20
    assert mx.mxfp4_moe_route_workspace_bytes(8192, 2000) == 0
    assert mx.mxfp4_moe_route_workspace_bytes(-1, 64) == 0
    assert mx.lib().mxfp4_reserve_bytes(1 << 60, None) == UNSUPPORTED


def test_route_binding_refuses():
    torch = pytest.importorskip("torch")
    l = torch.zeros((4, 8))
    for bad in (dict(score="relu"), dict(bias=torch.zeros(7)), dict(bias=torch.zeros(8, dtype=torch.float64))):
        with pytest.raises(ValueError):
            mx.moe_route(l, 2, **bad)
    with pytest.raises(TypeError):
        mx.moe_route(l.double(), 2)
    with pytest.raises(ValueError):
        mx.moe_route(l.reshape(-1), 2)
    with pytest.raises(ValueError):
        mx.moe_route(torch.zeros((8, 4)).t(), 2)
    with pytest.raises(ValueError, match="cuda"):
        mx.moe_route(l, 2)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = [i(4, 2), torch.zeros(4, 2), i(9), i(8), i(4, 2)]
    for n in range(5):
        out = list(good)
        out[n] = out[n].double()
        with pytest.raises(ValueError, match="must be"):
            mx.moe_route(l, 2, out=out)


def test_combine_binding_refuses():
    torch = pytest.importorskip("torch")
    y, w = torch.zeros((8, 16), dtype=torch.bfloat16), torch.zeros((4, 2))
    with pytest.raises(TypeError):
        mx.moe_combine(y.double(), w)
    with pytest.raises(TypeError):
        mx.moe_combine(y, w, residual=torch.zeros((4, 16)), out=torch.zeros((4, 16), dtype=torch.bfloat16))
    for bad in (dict(pos=torch.zeros((4, 2), dtype=torch.int64)), dict(pos=torch.zeros((4, 3), dtype=torch.int32)),
                dict(residual=torch.zeros((4, 15), dtype=torch.bfloat16)),
                dict(out=torch.zeros((3, 16), dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            mx.moe_combine(y, w, **bad)
    with pytest.raises(ValueError):
        mx.moe_combine(y, w.double())
    with pytest.raises(ValueError):
        mx.moe_combine(y[:7], w)
    with pytest.raises(ValueError, match="cuda"):
        mx.moe_combine(y, w)

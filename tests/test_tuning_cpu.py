"""Argument checks of the adapter and router-training calls: refused on the
host with the documented status, before anything is enqueued (no GPU)."""
import pytest

from routed_expert_layer_route_b200 import build as pkg_build
from routed_expert_layer_route_b200 import moe

FAKE = 1 << 40  # aligned non-null pointer value; never dereferenced
INVALID, SHAPE, SMALL = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED_SHAPE,
                         moe.MOE_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def L():
    pkg_build.build()
    return moe.lib()


BAD_SHAPES = [dict(T=-1), dict(T=(1 << 20) + 1), dict(din=4), dict(din=100), dict(dout=12),
              dict(dout=16392), dict(din=0), dict(r=0), dict(r=129), dict(n=0), dict(n=1025)]


def linear(L, x=FAKE, w=FAKE, bias=None, ad=FAKE, a=FAKE, b=FAKE, s=None, T=4, din=64, dout=64, r=8,
           n=2, y=FAKE, y_dtype=0, u=None, ws=FAKE, ws_bytes=1 << 40):
    return L.moe_adapter_linear(x, w, bias, ad, a, b, s, T, din, dout, r, n, y, y_dtype, u, ws,
                                ws_bytes, None)


def backward(L, dy=FAKE, x=FAKE, w=FAKE, ad=FAKE, a=FAKE, b=FAKE, s=None, u=FAKE, T=4, din=64,
             dout=64, r=8, n=2, dx=FAKE, dx_dtype=0, da=FAKE, db=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L.moe_adapter_backward(dy, x, w, ad, a, b, s, u, T, din, dout, r, n, dx, dx_dtype, da, db,
                                  ws, ws_bytes, None)


@pytest.mark.parametrize("bad", BAD_SHAPES, ids=str)
def test_adapter_shapes(L, bad):
    assert linear(L, **bad) == SHAPE
    assert backward(L, **bad) == SHAPE
    size = dict(T=4, din=64, dout=64, r=8, n=2)
    assert moe.moe_adapter_workspace_size(**size) > 0
    assert moe.moe_adapter_workspace_size(**{**size, **bad}) == 0


def test_adapter_workspace_grows_with_the_sizes(L):
    base = dict(T=64, din=256, dout=256, r=8, n=4)
    size = moe.moe_adapter_workspace_size(**base)
    assert size % 256 == 0
    for k in base:  # a workspace of larger sizes serves smaller ones
        assert moe.moe_adapter_workspace_size(**{**base, k: 2 * base[k]}) >= size


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(ad=None), dict(a=None), dict(b=None), dict(y=None), dict(ws=None),
    dict(ws=FAKE + 16), dict(x=FAKE + 8), dict(w=FAKE + 2), dict(a=FAKE + 8), dict(b=FAKE + 4),
    dict(y=FAKE + 4), dict(u=FAKE + 4), dict(ad=FAKE + 2), dict(s=FAKE + 1), dict(bias=FAKE + 2),
    dict(y_dtype=2), dict(y_dtype=-1)], ids=str)
def test_linear_arguments(L, bad):
    assert linear(L, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(dy=None), dict(ad=None), dict(b=None), dict(a=None), dict(x=None), dict(u=None), dict(ws=None),
    dict(dx=None, da=None, db=None), dict(dx=FAKE + 8), dict(da=FAKE + 4), dict(db=FAKE + 8),
    dict(dy=FAKE + 2), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(u=FAKE + 4), dict(dx_dtype=5)], ids=str)
def test_backward_arguments(L, bad):
    assert backward(L, **bad) == INVALID


def test_adapter_workspace_too_small(L):
    need = moe.moe_adapter_workspace_size(4, 64, 64, 8, 2)
    assert linear(L, ws_bytes=need - 1) == SMALL
    assert backward(L, ws_bytes=need - 1) == SMALL


def test_adapter_no_rows(L):
    assert linear(L, T=0, x=None, y=None, ws=None, ws_bytes=0) == moe.MOE_OK


def balance(L, z=FAKE, idx=FAKE, mask=None, T=4, E=64, k1=4, cb=0.1, cz=0.1, n=FAKE, loss=FAKE,
            prob=None, ws=FAKE, ws_bytes=1 << 40):
    return L.moe_balance_loss(z, idx, mask, T, E, k1, cb, cz, n, loss, prob, ws, ws_bytes, None)


def route(L, z=FAKE, idx=FAKE, dw=FAKE, n=None, mask=None, T=4, E=64, k1=4, k2=8, cb=0.1, cz=0.1,
          dl=None, dz=FAKE, dtype=0, ws=None, ws_bytes=0):
    return L.moe_route_backward(z, idx, dw, n, mask, T, E, k1, k2, cb, cz, dl, dz, dtype, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(k1=0), INVALID), (dict(k1=33), INVALID), (dict(E=3), INVALID), (dict(z=None), INVALID),
    (dict(z=FAKE + 4), INVALID), (dict(idx=FAKE + 4), INVALID), (dict(cb=float("nan")), INVALID),
    (dict(cz=float("nan")), INVALID)], ids=str)
def test_router_training_arguments(L, bad, status):
    assert balance(L, **bad) == status
    assert route(L, **bad) == status


def test_balance_arguments(L):
    for bad in (dict(idx=None), dict(n=None), dict(loss=None), dict(n=FAKE + 2), dict(loss=FAKE + 1),
                dict(prob=FAKE + 2), dict(ws=None), dict(ws=FAKE + 128)):
        assert balance(L, **bad) == INVALID, bad
    need = moe.moe_balance_workspace_size(4, 64)
    assert need % 256 == 0 and balance(L, ws_bytes=need - 1) == SMALL
    assert moe.moe_balance_workspace_size(4, 0) == 0
    assert moe.moe_balance_workspace_size(-1, 64) == 0


def test_route_backward_arguments(L):
    for bad in (dict(k2=3), dict(dw=None), dict(idx=None), dict(dz=None), dict(dz=FAKE + 8),
                dict(dtype=3), dict(dw=FAKE + 2), dict(n=FAKE + 2), dict(dl=FAKE + 1),
                dict(ws=FAKE + 16, ws_bytes=1 << 20)):
        assert route(L, **bad) == INVALID, bad
    assert route(L, ws=FAKE, ws_bytes=100) == SMALL
    assert route(L, T=0) == moe.MOE_OK

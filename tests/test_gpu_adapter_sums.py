"""How near the adapter calls' float32 outputs are to 64 bits.

A sum on the tensor cores rounds towards zero at each step of 16 products: it
loses half of the last of 24 bits at a step on average, 2^-24 / m of the running
sum with m its mantissa (the mean of 1 / m over a logarithmic scale: 0.72).  A
running sum of n steps of random sign grows as a random walk, so what it lost
is, in the 2-norm over many outputs, 0.72 n 2^-24 / sqrt(3) of the result.  All
else (u's parts of 24 bits together, rounded joins and stores) stays below 2^-22."""
import math

import pytest
import torch

import tune_ref as ref
from routed_expert_layer_route_b200 import moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
SEGMENT = 48  # most steps of one sum of a float32 output
INNER = 16    # of one sum of an inner product, and of the projection of few rows
PARTS = 12    # of an adapter's part: three parts of u for each 16 of 64 ranks


def norm_bound(steps):
    return 0.72 * steps * 2.0 ** -24 / math.sqrt(3) + 2.0 ** -22


def far(got, want):
    return float((got.double() - want).norm() / want.norm())


def by_rows(u, b, adapter, n):
    """The adapters' part of y from given u, in 64 bits."""
    y = torch.zeros(u.shape[0], b.shape[2], dtype=torch.float64, device=DEV)
    for i in range(n):
        t = (adapter == i).nonzero()[:, 0]
        y[t] = u[t].double() @ b[i].double()
    return y


@pytest.mark.parametrize("T,din,dout,r,n,rows", [
    (1100, 8192, 1032, 16, 4, "runs"), (2600, 4096, 2056, 24, 3, "runs"), (100, 8192, 264, 40, 6, "mixed"),
    (300, 4104, 136, 16, 3, "mixed"), (40, 4096, 136, 16, 4, "mixed")], ids=str)
def test_projection_of_a_long_k(T, din, dout, r, n, rows):
    c = ref.Case(T, din, dout, r, n, rows, seed=31)
    y, u = torch.empty(T, dout, device=DEV), torch.empty(T, r, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, y, ws, u_out=u)
    want = c.x.double() @ c.w.double().t() + c.bias.double() + by_rows(u, c.b, c.adapter, n)
    assert far(y, want) <= norm_bound(SEGMENT)
    assert far(u, ref.inner(c.x, c.a, c.adapter, c.scale)[0]) <= norm_bound(INNER)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("K", [2056, 4096, 16384])
@pytest.mark.parametrize("T,r", [(1, 32), (20, 16), (60, 40), (300, 32), (1500, 64), (2500, 10), (2500, 32),
                                 (2500, 128), (4500, 33)], ids=str)
def test_inner_products_of_a_long_k(T, r, K):
    c = ref.Case(T, K, 64, r, 1, "one", seed=37)
    y, u = torch.empty(T, 64, device=DEV), torch.empty(T, r, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_linear(c.x, c.w, None, c.adapter, c.a, c.b, None, y, ws, u_out=u)
    assert far(u, c.x.double() @ c.a[0].double().t()) <= norm_bound(INNER)
    want = c.x.double() @ c.w.double().t() + u.double() @ c.b[0].double()
    assert far(y, want) <= norm_bound(INNER if T <= 32 else SEGMENT)
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T,dout,r,n", [(2600, 2056, 64, 3), (500, 264, 33, 4), (50, 264, 64, 3)], ids=str)
def test_the_adapters_part_alone(T, dout, r, n):
    # u with 24 bits
    c = ref.Case(T, 128, dout, r, n, "runs", seed=32)
    y, u = torch.zeros(T, dout, device=DEV), torch.empty(T, r, device=DEV)
    moe.moe_adapter_linear(c.x, None, None, c.adapter, c.a, c.b, c.scale, y, c.workspace(), u_out=u)
    assert far(y, by_rows(u, c.b, c.adapter, n)) <= norm_bound(PARTS)


def d_lora_b(c, u, dy):
    db = torch.full((c.n, c.r, c.dout), 7.0, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_backward(dy, None, None, c.adapter, c.a, c.b, None, u, None, db, ws)
    assert moe.moe_read_device_status(ws) == 0
    return db


@pytest.mark.parametrize("T,din,dout,r", [
    (768, 8, 264, 16), (768, 2048, 2048, 64), (20000, 4096, 4096, 64), (131072, 16384, 8, 128)], ids=str)
def test_gradient_of_many_rows(T, din, dout, r):
    # one adapter's sum over all rows, however many a piece has
    c = ref.Case(T, 8, 8, r, 1, "one", seed=33)
    g = torch.Generator(device=DEV).manual_seed(T)
    c.din, c.dout = din, dout
    c.a = torch.zeros(1, r, din, device=DEV, dtype=torch.bfloat16)
    c.b = torch.zeros(1, r, dout, device=DEV, dtype=torch.bfloat16)
    dy = torch.randn(T, dout, generator=g, device=DEV).bfloat16()
    db = d_lora_b(c, c.u, dy)
    assert far(db, (c.u.double().t() @ dy.double())[None]) <= norm_bound(SEGMENT)


def test_both_gradients_of_many_rows():
    c = ref.Case(20000, 4096, 4096, 64, 2, "one", seed=34)
    da, db = torch.empty(2, 64, 4096, device=DEV), torch.empty(2, 64, 4096, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, c.scale, c.u, da, db, ws)
    v = ref.inner(c.dy, c.b, c.adapter, c.scale)[0]
    assert far(da[1], v.t() @ c.x.double()) <= norm_bound(SEGMENT) + norm_bound(INNER)
    assert far(db[1], c.u.double().t() @ c.dy.double()) <= norm_bound(SEGMENT)
    assert (da[0] == 0).all() and (db[0] == 0).all()
    for got, k in ((da, dict(d_lora_a=torch.empty_like(da), d_lora_b=None)),
                   (db, dict(d_lora_a=None, d_lora_b=torch.empty_like(db)))):
        moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, c.scale, c.u, ws=ws, **k)
        assert torch.equal(got, k["d_lora_a"] if k["d_lora_b"] is None else k["d_lora_b"])
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("row", [0, 1000, 1999, 3999])
def test_infinities_in_long_sums(row):
    # pieces of 2000 rows, three sums each: what an inf or a NaN in any of them makes
    c = ref.Case(4000, 8, 8, 128, 1, "one", seed=36)
    c.din = 16384
    c.a = torch.zeros(1, 128, 16384, device=DEV, dtype=torch.bfloat16)
    dy = c.dy.clone()
    dy[row, 3] = float("inf")
    dy[2500, 5] = dy[2501, 5] = float("inf")
    u = c.u.clone()
    u[row, 7] = float("nan")
    u[3000, 9] = 0.0
    dy[3000, 6] = float("-inf")
    want = torch.einsum("tr,td->trd", u.double(), dy.double()).sum(0)
    got = d_lora_b(c, u, dy)[0]
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)].double(), want[torch.isinf(want)])
    assert far(got[fine], want[fine]) <= norm_bound(SEGMENT)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2600, 1032, 2056, 24, 3, "runs"), (2600, 1032, 2056, 16, 9, "mixed"),
                                   (5000, 520, 1032, 40, 4, "mixed")], ids=str)
def test_more_tiles_than_pairs_with_a_long_k(shape, dtype):
    # the K ring turns within a tile, segments and units of adapters follow each other over tiles
    c = ref.Case(*shape, seed=35)
    y, u = torch.empty(c.T, c.dout, device=DEV, dtype=dtype), torch.empty(c.T, c.r, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, y, ws, u_out=u)
    want, e, wu, eu = ref.linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale)
    ref.check(y, want, e, "y")
    ref.check(u, wu, eu, "u")
    for _ in range(3):
        again = torch.empty_like(y)
        moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, again, ws)
        assert torch.equal(again, y)
    assert moe.moe_read_device_status(ws) == 0

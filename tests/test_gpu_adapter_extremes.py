"""Numbers at the ends of their types in the adapters' weight gradients."""
import pytest
import torch

import tune_ref as ref
from routed_expert_layer_route_b200 import moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def d_lora_b(c, u, dy):
    db = torch.full((c.n, c.r, c.dout), 7.0, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_backward(dy, None, None, c.adapter, c.a, c.b, None, u, None, db, ws)
    assert moe.moe_read_device_status(ws) == 0
    return db


def outer_by_rows(u, z, adapter, n):
    """sum of u_t z_t^T over each adapter's own rows: infinities by the formula."""
    return torch.stack([torch.einsum("tr,td->trd", u[adapter == i].double(), z[adapter == i].double()).sum(0)
                        for i in range(n)])


def check_with_infinities(got, want, finite_bound, what):
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[torch.isinf(want)].double(), want[torch.isinf(want)]), what
    off = (got.double() - want).abs()[fine] - finite_bound[fine] - 2.0 ** -24 * want.abs()[fine]
    assert float(off.max()) <= 0.0, what


@pytest.mark.parametrize("T,din,dout,r,n", [(9, 64, 72, 3, 2), (300, 264, 136, 10, 3), (700, 40, 520, 70, 1),
                                            (3000, 72, 40, 17, 2)], ids=str)
def test_infinities_in_gradients(T, din, dout, r, n):
    # an inf in a row makes its adapter's sums of that column infinite, not NaN
    c = ref.Case(T, din, dout, r, n, "runs", seed=36)
    c.adapter = (torch.arange(T, device=DEV) // 3 % (n + 1)).int()
    c.adapter[c.adapter == n] = ref.EMPTY
    rows = (c.adapter != ref.EMPTY).nonzero()[:, 0]
    x, dy = c.x.clone(), c.dy.clone()
    x[rows[0], 5] = float("inf")
    x[rows[-1], din - 1] = float("-inf")
    x[rows[1], 9] = x[rows[2], 9] = float("inf")  # NaN where their factors differ in sign
    ws = c.workspace()
    da = torch.full((n, r, din), 7.0, device=DEV)
    moe.moe_adapter_backward(dy, x, None, c.adapter, c.a, c.b, c.scale, None, da, None, ws)
    v, ev = ref.inner(dy, c.b, c.adapter, c.scale)
    want = outer_by_rows(v, x, c.adapter, n)
    _, e = ref.outer(v, torch.where(torch.isfinite(x), x, torch.zeros_like(x)), c.adapter, n, eu=ev)
    assert torch.isinf(want).any()
    check_with_infinities(da, want, e, "d_lora_a")
    dy[rows[0], 0] = float("-inf")
    dy[rows[-1], dout - 1] = float("inf")
    u = c.u.clone()
    u[rows[1], r - 1] = float("inf")
    u[rows[2], 0] = float("nan")
    want = outer_by_rows(u, dy, c.adapter, n)
    calm = [torch.where(torch.isfinite(t), t, torch.zeros_like(t)) for t in (u, dy)]
    check_with_infinities(d_lora_b(c, u, dy), want, ref.outer(*calm, c.adapter, n)[1], "d_lora_b")
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T", [5, 600, 2500, 4500])
def test_the_largest_numbers_of_u(T):
    # above the largest bf16: the first part may not become an infinity
    c = ref.Case(T, 64, 72, 6, 2, "one", seed=37)
    u = torch.zeros(T, 6, device=DEV)
    top = torch.finfo(torch.float32).max
    u[1, 0], u[2, 1], u[3, 5] = top, -top, 3.3953e38
    dy = torch.zeros(T, 72, device=DEV, dtype=torch.bfloat16)
    dy[1, 3], dy[2, 7], dy[3, 71], dy[1, 64] = 0.5, 0.25, -0.5, 0.0
    db = d_lora_b(c, u, dy)
    want = (u.double().t() @ dy.double())[None]
    assert torch.isfinite(db).all()
    assert float((db[1].double() - want[0]).abs().max()) <= 2.0 ** -22 * top
    assert (db[1][want[0] == 0] == 0).all() and (db[0] == 0).all()


@pytest.mark.parametrize("T", [20, 100, 2500, 5000])
def test_the_largest_numbers_of_the_projection(T):
    # u itself above the largest bf16: one product of the inner sum, the rest zeros
    n, r, d = 2, 5, 72
    c = ref.Case(T, d, d, r, n, "one", seed=38)
    for t in (c.x, c.a, c.b):
        t.zero_()
    big = 2.0 ** 64 * (1 - 2.0 ** -8)
    c.x[3, 8], c.a[1, 2, 8] = big, big          # u = 2^128 (1 - 2^-8)^2 = 2^128 (1 - 2^-7 + 2^-16)
    c.x[7, 9], c.a[1, 4, 9] = -(2.0 ** 64 - 2.0 ** 56), 2.0 ** 63
    c.b[1, 2, 3], c.b[1, 4, 5] = 0.5, 1.0
    scale = torch.tensor([1.0, 1.0 + 2.0 ** -7 - 2.0 ** -12], device=DEV)
    wu = scale[1].double() * (c.x.double() @ c.a[1].double().t())
    y, u = torch.zeros(T, d, device=DEV), torch.empty(T, r, device=DEV)
    moe.moe_adapter_linear(c.x, None, None, c.adapter, c.a, c.b, scale, y, c.workspace(), u_out=u)
    assert float(wu.abs().max()) > 3.397e38 and torch.isfinite(u).all()
    assert torch.allclose(u.double(), wu, rtol=2.0 ** -22, atol=0.0)
    assert torch.allclose(y.double(), wu @ c.b[1].double(), rtol=2.0 ** -22, atol=0.0)

"""moe_adapter_linear and moe_adapter_backward against their 64-bit forms, at
the sizes, row orders and ranks where a kernel's tiles end, and the calls
around them: captured and replayed, on a side stream, beside moe_layer."""
import pytest
import torch

import tune_ref as ref
from routed_expert_layer_route_b200 import moe, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

# T, din, dout, r, n, rows
SHAPES = [
    (1, 64, 8, 1, 1, "one"), (1, 2048, 128, 16, 8, "one"), (1, 512, 512, 16, 4, "none"),
    (3, 8, 8, 3, 2, "mixed"), (7, 200, 72, 10, 3, "mixed"), (8, 768, 2048, 64, 5, "mixed"),
    (9, 2048, 768, 16, 64, "mixed"), (17, 1032, 136, 128, 7, "mixed"), (32, 4096, 256, 8, 32, "mixed"),
    (33, 264, 1000, 33, 3, "runs"), (64, 1024, 1024, 16, 16, "mixed"), (65, 136, 264, 64, 5, "mixed"),
    (127, 512, 128, 16, 3, "runs"), (128, 128, 256, 17, 2, "one"), (129, 72, 40, 5, 9, "mixed"),
    (255, 1000, 1544, 10, 3, "runs"), (257, 512, 520, 128, 40, "mixed"), (300, 64, 4096, 2, 300, "mixed"),
    (513, 2048, 128, 16, 4, "runs"), (1030, 1024, 776, 48, 6, "runs"), (700, 256, 128, 16, 2, "none"),
    (2561, 136, 2056, 24, 3, "runs"), (1200, 200, 4104, 16, 12, "mixed"),
    (64, 4096, 2056, 16, 5, "mixed"), (40, 2056, 4096, 20, 6, "runs"), (4200, 64, 64, 4, 300, "mixed"),
    (17000, 64, 72, 3, 5, "runs"), (2100, 136, 264, 100, 4, "mixed"), (2048, 1032, 128, 16, 1, "one"),
    (2047, 72, 136, 9, 200, "mixed"), (4096, 264, 64, 12, 256, "mixed"), (4097, 64, 200, 33, 2, "runs"),
    (200, 8, 8, 3, 2, "mixed"), (2100, 8, 16, 20, 3, "mixed"), (66, 16384, 8, 1, 1, "one"), (12, 8, 16384, 16, 2, "mixed"),
]


def run_linear(c, dtype, bias=True, scale=True, keep=True, product=None, ws=None, stream=None):
    y = torch.full((c.T, c.dout), 7.0, device=DEV, dtype=dtype) if product is None else product.clone()
    u = torch.full((c.T, c.r), 7.0, device=DEV) if keep else None
    ws = c.workspace() if ws is None else ws
    moe.moe_adapter_linear(c.x, c.w if product is None else None, c.bias if bias else None,
                           c.adapter, c.a, c.b, c.scale if scale else None, y, ws, u_out=u,
                           stream=stream)
    return y, u, ws


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_linear(shape, dtype):
    c = ref.Case(*shape)
    full = dtype == torch.float32
    y, u, ws = run_linear(c, dtype, bias=full, scale=full, keep=full)
    want, e, wu, eu = ref.linear(c.x, c.w, c.bias if full else None, c.adapter, c.a, c.b,
                                 c.scale if full else None)
    ref.check(y, want, e, "y")
    if full:
        ref.check(u, wu, eu, "u")
        assert (u[c.adapter == ref.EMPTY] == 0).all()
    y2, _, _ = run_linear(c, dtype, bias=full, scale=full, keep=full, ws=ws)
    assert torch.equal(y, y2)  # deterministic, and the workspace serves again
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_linear_beside_a_product(shape, dtype):
    c = ref.Case(*shape, seed=1)
    product = torch.randn(c.T, c.dout, device=DEV).to(dtype)
    y, u, ws = run_linear(c, dtype, bias=False, product=product)
    want, e, wu, eu = ref.linear(c.x, None, None, c.adapter, c.a, c.b, c.scale, product=product)
    ref.check(y, want, e, "y")
    ref.check(u, wu, eu, "u")
    none = c.adapter == ref.EMPTY
    assert torch.equal(y[none], product[none])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_backward(shape, dtype):
    c = ref.Case(*shape, seed=2)
    w_t = c.w.t().contiguous()
    scale = c.scale if dtype == torch.float32 else None
    da = torch.full((c.n, c.r, c.din), 7.0, device=DEV)
    db = torch.full((c.n, c.r, c.dout), 7.0, device=DEV)
    dx = torch.full((c.T, c.din), 7.0, device=DEV, dtype=dtype)
    ws = c.workspace()
    moe.moe_adapter_backward(c.dy, c.x, w_t, c.adapter, c.a, c.b, scale, c.u, da, db, ws, dx=dx)
    want_dx, e_dx, v, ev = ref.linear(c.dy, w_t, None, c.adapter, c.b, c.a, scale)
    ref.check(dx, want_dx, e_dx, "dx")
    want, e = ref.outer(v, c.x, c.adapter, c.n, eu=ev)
    ref.check(da, want, e, "d_lora_a")
    want, e = ref.outer(c.u, c.dy, c.adapter, c.n)
    ref.check(db, want, e, "d_lora_b")
    for i in range(c.n):
        if not (c.adapter == i).any():
            assert (da[i] == 0).all() and (db[i] == 0).all()
    # each output alone, and dx added to what is there
    only = torch.full_like(da, 7.0)
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, scale, None, only, None, ws)
    assert torch.equal(only, da)
    only = torch.full_like(db, 7.0)
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, scale, c.u, None, only, ws)
    assert torch.equal(only, db)
    base = torch.randn(c.T, c.din, device=DEV).to(dtype)
    add = base.clone()
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, scale, None, None, None, ws, dx=add)
    want, e, _, _ = ref.linear(c.dy, None, None, c.adapter, c.b, c.a, scale, product=base)
    ref.check(add, want, e, "dx added")
    assert moe.moe_read_device_status(ws) == 0


def test_gradients_against_differences():
    # the directional derivative of sum(dy * y) in 64 bits, by central differences
    c = ref.Case(50, 128, 96, 6, 3, seed=3)
    y, u, ws = run_linear(c, torch.float32)
    da, db = torch.empty(c.n, c.r, c.din, device=DEV), torch.empty(c.n, c.r, c.dout, device=DEV)
    dx = torch.empty(c.T, c.din, device=DEV)
    moe.moe_adapter_backward(c.dy, c.x, c.w.t().contiguous(), c.adapter, c.a, c.b, c.scale, u, da,
                             db, ws, dx=dx)

    def f(x, a, b):
        return float((c.dy.double() * ref.linear(x, c.w, c.bias, c.adapter, a, b, c.scale)[0]).sum())
    x, a, b = c.x.double(), c.a.double(), c.b.double()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    h = 1e-4  # f is quadratic along a and b together, linear along each: no cut-off error
    for grad, at in ((dx, 0), (da, 1), (db, 2)):
        v = torch.randn(grad.shape, generator=gen, device=DEV, dtype=torch.float64)
        up, dn = [x, a, b], [x, a, b]
        up[at] = up[at] + h * v
        dn[at] = dn[at] - h * v
        num = (f(*up) - f(*dn)) / (2 * h)
        got = float((grad.double() * v).sum())
        # float32 gradients of relative error 2^-15 against a sum of random signs
        assert abs(got - num) <= 2.0 ** -15 * float(grad.double().norm() * v.norm()) + 1e-7 * abs(f(x, a, b)) / h


@pytest.mark.parametrize("T,dout", [(5, 72), (40, 136), (300, 264)])
def test_bad_numbers_stay_in_their_rows(T, dout):
    # NaN and inf in one adapter, in one row of x, or in a row without an adapter reach only their own rows
    c = ref.Case(T, 256, dout, 12, 4, seed=4)
    c.adapter = (torch.arange(T, device=DEV) % 5).int()
    c.adapter[c.adapter == 4] = ref.EMPTY
    ws = c.workspace()
    want, e, _, _ = ref.linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale)
    c.a[2, 3, 7] = float("nan")
    c.b[1, 5, 3] = float("inf")
    c.b[3, 2, :] = float("nan")
    c.x[4, 9] = float("nan")
    y, u, _ = run_linear(c, torch.float32, ws=ws)
    row = torch.arange(T, device=DEV)
    fine = (row % 5 == 0) | ((row % 5 == 4) & (row != 4))
    ref.check(y[fine], want[fine], e[fine])
    ones = (row % 5 == 1)
    cols = torch.arange(dout, device=DEV) != 3
    ref.check(y[ones][:, cols], want[ones][:, cols], e[ones][:, cols])
    assert torch.isinf(y[ones][:, 3]).all()
    assert torch.isnan(y[row % 5 == 2]).all() and torch.isnan(y[row % 5 == 3]).all()
    assert torch.isnan(y[4]).all() and (u[4] == 0).all()
    # gradients: adapter 0 sees none of it
    da, db = torch.empty(c.n, c.r, c.din, device=DEV), torch.empty(c.n, c.r, c.dout, device=DEV)
    c.u[2, 0] = float("nan")
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, c.scale, c.u, da, db, ws)
    assert torch.isfinite(da[0]).all() and torch.isfinite(db[0]).all() and torch.isfinite(db[3]).all()
    assert torch.isnan(da[3, 2]).all() and torch.isfinite(da[3, 3:]).all() and torch.isnan(db[2, 0]).all() and torch.isfinite(db[2, 1:]).all()


@pytest.mark.parametrize("T,din,dout", [(600, 1000, 520), (3000, 264, 2056), (70, 2056, 136)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("base", [True, False], ids=["product", "beside"])
def test_a_broken_adapter_in_every_tile(T, din, dout, dtype, base):
    # the rows of the others, whose products with it are 0 x inf, keep their values
    c = ref.Case(T, din, dout, 20, 3, seed=5)
    c.adapter = (torch.arange(T, device=DEV) % 4).int()
    c.adapter[c.adapter == 3] = ref.EMPTY
    product = None if base else torch.randn(T, dout, device=DEV).to(dtype)
    want, e, _, _ = ref.linear(c.x, c.w if base else None, c.bias if base else None, c.adapter, c.a,
                               c.b, c.scale, product=product)
    c.b[1, 7] = float("inf")
    c.b[1, 8] = float("-inf")
    c.x[5::60] = float("nan")
    y, _, ws = run_linear(c, dtype, bias=base, product=product)
    row = torch.arange(T, device=DEV)
    broken, own = row % 4 == 1, row % 60 == 5
    assert not torch.isfinite(y[broken]).any()
    fine = ~broken & ~own
    ref.check(y[fine], want[fine], e[fine])
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T", [1, 20, 70, 400])
def test_ids_out_of_range_count_as_none(T):
    c = ref.Case(T, 128, 64, 8, 3, seed=5)
    want, _, ws = run_linear(c, torch.float32)
    c.adapter[T // 2] = ref.EMPTY
    want, _, _ = run_linear(c, torch.float32, ws=ws)
    da = torch.empty(c.n, c.r, c.din, device=DEV)
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, None, None, da, None, ws)
    assert moe.moe_read_device_status(ws) == 0
    for bad in (3, -1, 1 << 20):
        c.adapter[T // 2] = bad
        y, u, _ = run_linear(c, torch.float32, ws=ws)
        assert torch.equal(y, want) and (u[T // 2] == 0).all()
        assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
        got = torch.empty_like(da)
        moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, None, None, got, None, ws)
        assert torch.equal(got, da)
        assert moe.moe_read_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK


@pytest.mark.parametrize("T", [1, 31, 200])
def test_rows_and_buffers_behind_the_batch_stay(T):
    c = ref.Case(T, 192, 104, 9, 2, seed=6)
    big_y = torch.full((T + 300, c.dout), 3.25, device=DEV)
    big_u = torch.full((T + 300, c.r), 3.25, device=DEV)
    ws = c.workspace()
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, big_y[:T], ws, u_out=big_u[:T])
    big_dx = torch.full((T + 300, c.din), 3.25, device=DEV, dtype=torch.bfloat16)
    big_da = torch.full((c.n + 1, c.r, c.din), 3.25, device=DEV)
    big_db = torch.full((c.n + 1, c.r, c.dout), 3.25, device=DEV)
    moe.moe_adapter_backward(c.dy, c.x, c.w.t().contiguous(), c.adapter, c.a, c.b, c.scale,
                             big_u[:T], big_da[:c.n], big_db[:c.n], ws, dx=big_dx[:T])
    assert (big_y[T:] == 3.25).all() and (big_u[T:] == 3.25).all() and (big_dx[T:] == 3.25).all()
    assert (big_da[c.n:] == 3.25).all() and (big_db[c.n:] == 3.25).all()


@pytest.mark.parametrize("T", [4, 300])
def test_captured_and_replayed_on_new_values(T):
    c = ref.Case(T, 256, 192, 16, 5, seed=7)
    other = ref.Case(T, 256, 192, 16, 5, seed=8)
    w_t = c.w.t().contiguous()
    ws = c.workspace()
    y, u = torch.empty(T, c.dout, device=DEV), torch.empty(T, c.r, device=DEV)
    da, db = torch.empty(c.n, c.r, c.din, device=DEV), torch.empty(c.n, c.r, c.dout, device=DEV)
    dx = torch.empty(T, c.din, device=DEV)

    def step():
        moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, y, ws, u_out=u)
        moe.moe_adapter_backward(c.dy, c.x, w_t, c.adapter, c.a, c.b, c.scale, u, da, db, ws, dx=dx)
    step()  # lazy set-up outside the capture
    torch.cuda.synchronize()
    graph, twin = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    with torch.cuda.graph(twin):  # a second graph on the same workspace
        step()
    for name in ("x", "a", "b", "scale", "adapter", "dy"):
        getattr(c, name).copy_(getattr(other, name))
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, u, da, db, dx)]
    for t in (y, u, da, db, dx):
        t.fill_(7.0)
    graph.replay()
    twin.replay()
    graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((y, u, da, db, dx), want):
        assert torch.equal(got, w)
    assert moe.moe_read_device_status(ws) == 0


def test_side_stream_and_two_calls_at_once():
    c, d = ref.Case(300, 512, 256, 16, 4, seed=9), ref.Case(20, 512, 256, 16, 4, seed=10)
    want_c, _, _ = run_linear(c, torch.float32)
    want_d, _, _ = run_linear(d, torch.float32)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        ws1 = c.workspace()
        y1 = torch.empty(c.T, c.dout, device=DEV)
    with torch.cuda.stream(s2):
        ws2 = d.workspace()
        y2 = torch.empty(d.T, d.dout, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, y1, ws1, stream=s1)
        moe.moe_adapter_linear(d.x, d.w, d.bias, d.adapter, d.a, d.b, d.scale, y2, ws2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(y1, want_c) and torch.equal(y2, want_d)


def test_one_workspace_for_smaller_batches():
    big = ref.Case(600, 512, 256, 32, 6, seed=11)
    ws = big.workspace()
    for T in (600, 1, 64, 65, 333, 7):
        c = ref.Case(T, 512, 256, 32, 6, seed=T)
        y, _, _ = run_linear(c, torch.float32, ws=ws)
        want, e, _, _ = ref.linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale)
        ref.check(y, want, e, "T = %d" % T)
    assert moe.moe_read_device_status(ws) == 0


def test_no_rows():
    c = ref.Case(0, 64, 64, 4, 3)
    ws = c.workspace()
    y = torch.empty(0, 64, device=DEV)
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, y, ws)
    da, db = torch.full((3, 4, 64), 7.0, device=DEV), torch.full((3, 4, 64), 7.0, device=DEV)
    moe.moe_adapter_backward(c.dy, c.x, c.w, c.adapter, c.a, c.b, c.scale, c.u, da, db, ws)
    assert (da == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T", [3, 48, 512])
def test_beside_the_routed_layer(T):
    # each request's adapter added to the layer's own output
    d, E, I, k1 = 256, 16, 128, 2
    L = synth.make_layer(T, d, E, I, seed=3, device=DEV)
    c = ref.Case(T, d, d, 8, 6, seed=12)
    y = torch.empty(T, d, device=DEV)
    moe.moe_layer(L.x, L.w_router, L.bias, L.w_gate, L.w_up, L.w_down, k1, k1, y,
                  moe.workspace(T, d, E, I, k1))
    product = y.clone()
    moe.moe_adapter_linear(L.x, None, None, c.adapter, c.a, c.b, c.scale, y, c.workspace())
    want, e, _, _ = ref.linear(L.x, None, None, c.adapter, c.a, c.b, c.scale, product=product)
    ref.check(y, want, e)


def test_pack_w_down_lays_an_adapter_out_by_rank():
    c = ref.Case(20, 64, 128, 16, 3, seed=13)
    torch_layout = c.b.transpose(1, 2).contiguous()  # [n x dout x r]
    assert torch.equal(moe.moe_pack_w_down(torch_layout), c.b)


def test_python_checks():
    c = ref.Case(4, 64, 64, 4, 2)
    ws, y = c.workspace(), torch.empty(4, 64, device=DEV)
    good = dict(x=c.x, w=c.w, bias=c.bias, adapter=c.adapter, lora_a=c.a, lora_b=c.b, scale=c.scale,
                y=y, ws=ws)
    moe.moe_adapter_linear(**good)
    for name, bad in (("x", c.x.float()), ("x", c.x.cpu()), ("w", c.w[:32]), ("w", c.w.t()),
                      ("adapter", c.adapter.long()), ("lora_a", c.a[:1]), ("scale", c.scale.double()),
                      ("y", y.half()), ("y", torch.empty(4, 128, device=DEV)[:, ::2]),
                      ("bias", c.bias[:8]), ("ws", ws[:4096]), ("ws", ws[16:])):
        with pytest.raises(moe.MoeError):
            moe.moe_adapter_linear(**{**good, name: bad})

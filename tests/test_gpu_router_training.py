"""moe_balance_loss and moe_route_backward against their 64-bit forms, on the
routes that moe_route, moe_route_cascade and moe_route_skip write, and a
router's adapters trained through both.

Error bounds, in float32 roundings of 2^-24 relative: a probability takes the
difference to the largest logit (its rounding moves the exponential by
|z - max| 2^-24), the exponential itself (2^-21 with the hardware's power of
two), a sum over E values in a warp tree and a division.  With logits within
+-20 that is below 2^-18 for every probability, and the sums of positive
terms keep it."""
import math

import pytest
import torch

import tune_ref as ref
from routed_expert_layer_route_b200 import moe

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
P_ERR = 2.0 ** -18  # relative error of a probability, and of sums of them

# T, E, k1, k2
SHAPES = [(1, 1, 1, 1), (1, 128, 8, 16), (2, 2, 1, 2), (3, 31, 4, 8), (5, 33, 5, 33), (8, 64, 8, 8),
          (64, 128, 8, 16), (65, 127, 4, 16), (77, 300, 6, 1000), (100, 512, 10, 20), (33, 1000, 32, 40),
          (16, 1024, 32, 1023), (257, 256, 2, 100), (4099, 128, 4, 16), (1000, 511, 5, 20)]


def make(T, E, k1, seed=0, variable=False, mask=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000 + T * 7 + E + k1)
    z = torch.randn(T, E, generator=g, device=DEV) * 2.0
    idx = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k1].int()
    if variable:  # any slot after the first may be empty, as skipping leaves them
        drop = torch.rand(T, k1, generator=g, device=DEV) < 0.4
        drop[:, 0] = False
        idx = torch.where(drop, torch.full_like(idx, ref.EMPTY), idx)
    m = (torch.rand(T, generator=g, device=DEV) < 0.7) if mask else None
    d_w = torch.randn(T, k1, generator=g, device=DEV)
    return z.contiguous(), idx.contiguous(), m, d_w


def balance(z, idx, mask=None, c_bal=0.01, c_z=0.001, ws=None, stream=None):
    T, E = z.shape
    counts = torch.full((E + 1,), 77, dtype=torch.int32, device=DEV)
    loss, prob = torch.full((3,), 77.0, device=DEV), torch.full((E,), 77.0, device=DEV)
    ws = moe.balance_workspace(T, E) if ws is None else ws
    moe.moe_balance_loss(z, idx, c_bal, c_z, counts, loss, ws, token_mask=mask, prob_mean=prob,
                         stream=stream)
    return counts, loss, prob, ws


def check_balance(z, idx, mask, got):
    counts, loss, prob, ws = got
    want_n, P, bal, zl = ref.balance(z, idx, mask)
    assert torch.equal(counts.cpu().long(), want_n.long())
    assert torch.allclose(prob.double().to(P.device), P, rtol=P_ERR, atol=2.0 ** -40)
    # L_z: lse is off by 2^-23 of the largest term in it, which squares to twice that
    top = float(z[torch.isfinite(z)].abs().max()) if torch.isfinite(z).any() else 0.0
    for g, w, tol in ((loss[1], bal, P_ERR * abs(bal)),
                      (loss[2], zl, 2.0 ** -20 * (top + 7.0) ** 2),
                      (loss[0], 0.01 * bal + 0.001 * zl,
                       0.01 * P_ERR * abs(bal) + 0.001 * 2.0 ** -20 * (top + 7.0) ** 2)):
        assert abs(float(g) - w) <= tol + 2.0 ** -24 * abs(w)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("variable,mask", [(False, False), (True, True)], ids=["plain", "ragged"])
def test_balance(shape, variable, mask):
    T, E, k1, _ = shape
    z, idx, m, _ = make(T, E, k1, variable=variable, mask=mask)
    got = balance(z, idx, m)
    check_balance(z, idx, m, got)
    again = balance(z, idx, m, ws=got[3])  # deterministic, and the workspace serves again
    for a, b in zip(got[:3], again[:3]):
        assert torch.equal(a, b)
    assert moe.moe_read_device_status(got[3]) == 0
    if m is not None:
        as_bytes = balance(z, idx, m.to(torch.uint8) * 200, ws=got[3])
        assert torch.equal(as_bytes[1], got[1])


def route_backward(z, idx, k2, d_w, dtype=torch.float32, **kw):
    dz = torch.full(z.shape, 7.0, device=DEV, dtype=dtype)
    moe.moe_route_backward(z, idx, k2, d_w, dz, **kw)
    return dz


def check_dz(dz, want, mag, what=""):
    h = ref.HALF_STEP[dz.dtype]
    # every term carries two probabilities and one sum of them: 4 P_ERR of the terms' magnitudes
    bound = 4 * P_ERR * mag + 2.0 ** -126
    far = (dz.double() - want).abs() - (bound + h * (want.abs() + bound))
    assert float(far.max()) <= 0.0, (what, float(far.max()))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("variable,mask", [(False, False), (True, True)], ids=["plain", "ragged"])
def test_route_backward(shape, dtype, variable, mask):
    T, E, k1, k2 = shape
    z, idx, m, d_w = make(T, E, k1, seed=1, variable=variable, mask=mask)
    counts = balance(z, idx, m)[0]
    if variable:
        d_w[idx == ref.EMPTY] = float("nan")  # not used
    d_loss = torch.tensor([1.5], device=DEV)
    losses = dict(counts=counts, balance_coef=0.3, z_coef=0.05, d_loss=d_loss)
    plain = dict(counts=counts, c_bal=0.3, c_z=0.05, d_loss=1.5)
    for name, dw, kw, pkw in (("weights", d_w, {}, {}), ("losses", None, losses, plain),
                              ("both", d_w, losses, plain)):
        dz = route_backward(z, idx, k2, dw, dtype, token_mask=m, **kw)
        want, mag = ref.route_backward(z, idx, k2, dw, mask=m, **pkw)
        check_dz(dz, want, mag, name)
        assert torch.equal(dz, route_backward(z, idx, k2, dw, dtype, token_mask=m, **kw))
        if m is not None:
            assert (dz[~m] == 0).all()
    no_scale = route_backward(z, idx, k2, None, dtype, token_mask=m, counts=counts, balance_coef=0.3,
                              z_coef=0.05)
    want, mag = ref.route_backward(z, idx, k2, None, mask=m, counts=counts, c_bal=0.3, c_z=0.05)
    check_dz(no_scale, want, mag)


@pytest.mark.parametrize("E,k1,k2", [(128, 8, 8), (128, 4, 16), (40, 6, 64), (512, 5, 20)])
def test_routes_of_the_layer(E, k1, k2):
    # the weights that moe_route writes are the softmax whose gradient is taken
    T = 200
    z = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV) * 2
    idx = torch.empty(T, k1, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k1, device=DEV)
    tab = torch.rand(E, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV)
    routes = {
        "fixed": lambda: moe.moe_route(None, None, None, z, k1, k2, idx, w),
        "cascade": lambda: moe.moe_route_cascade(None, None, None, z, k1, k2, 0.5, idx, w),
        "skip": lambda: moe.moe_route_skip(None, None, None, z, k1, k2, tab, 0.6, 0.2, idx, w)}
    for name, call in routes.items():
        call()
        in_k2 = ref.k2_set(z, idx, k2)
        full = ref.weights(z.double(), in_k2)
        there = idx != ref.EMPTY
        at = idx.long().masked_fill(~there, 0)
        assert torch.allclose(full.gather(1, at)[there], w.double()[there], rtol=1e-5, atol=1e-30)
        d_w = torch.randn(T, k1, device=DEV)
        dz = route_backward(z, idx, k2, d_w)
        check_dz(dz, *ref.route_backward(z, idx, k2, d_w), what=name)
        # against differences of sum(d_w w) in 64 bits over the fixed set
        v = torch.randn(T, E, device=DEV, dtype=torch.float64)

        def f(zz):
            return (ref.weights(zz, in_k2).gather(1, at) * d_w.double()).masked_fill(~there, 0).sum(1)
        h = 1e-5
        num = (f(z.double() + h * v) - f(z.double() - h * v)) / (2 * h)
        got = (dz.double() * v).sum(1)
        # cut-off h^2 |f'''| and the difference's rounding, both below 1e-8 here
        assert float((got - num).abs().max()) <= 1e-4 * float(dz.double().norm(dim=1).max() * v.norm(dim=1).max())


def test_balance_gradient_against_differences():
    z, idx, m, _ = make(40, 48, 4, seed=6, mask=True)
    counts = balance(z, idx, m)[0]
    dz = route_backward(z, idx, 8, None, counts=counts, balance_coef=0.5, z_coef=0.2, token_mask=m)
    share = counts[:48].double() / float(counts[:48].sum())

    def f(zz):
        p, lse = torch.softmax(zz, 1)[m], torch.logsumexp(zz, 1)[m]
        N = float(m.sum())
        return float(0.5 * 48 * (share * p.sum(0) / N).sum() + 0.2 * lse.square().sum() / N)
    gen = torch.Generator(device=DEV).manual_seed(8)
    for _ in range(4):
        v = torch.randn(z.shape, generator=gen, device=DEV, dtype=torch.float64)
        h = 1e-5
        num = (f(z.double() + h * v) - f(z.double() - h * v)) / (2 * h)
        got = float((dz.double() * v).sum())
        assert abs(got - num) <= 1e-5 * float(dz.double().norm() * v.norm())


@pytest.mark.parametrize("E,k1", [(8, 1), (300, 1), (64, 3)])
def test_one_expert_in_k2_leaves_the_losses_alone(E, k1):
    # a weight of 1 has no gradient, however small the losses' is beside it; nor
    # have empty slots or a K2 of one given expert
    T = 500
    z, idx, _, d_w = make(T, E, k1, seed=16)
    if k1 > 1:
        idx[:, 1:] = ref.EMPTY
    counts = balance(z, idx)[0]
    kw = dict(counts=counts, balance_coef=1e-3, z_coef=1e-5)
    both = route_backward(z, idx[:, :1].contiguous(), 1, d_w[:, :1].contiguous(), **kw)
    assert torch.equal(both, route_backward(z, idx[:, :1].contiguous(), 1, None, **kw))


def test_ties_take_the_lower_index():
    T, E, k1, k2 = 6, 96, 2, 7
    z = torch.zeros(T, E, device=DEV)
    z[1, 50:] = 1.0
    z[2, ::3] = -0.0
    z[3, 5:9] = 2.0
    z[4] = -math.inf
    z[4, 90:] = 0.5
    z[5, :90] = -math.inf
    idx = torch.tensor([[95, 0], [95, 94], [1, 2], [6, 8], [95, 90], [91, 90]], dtype=torch.int32, device=DEV)
    d_w = torch.randn(T, k1, device=DEV)
    dz = route_backward(z, idx, k2, d_w)
    want, mag = ref.route_backward(z, idx, k2, d_w)
    check_dz(dz, want, mag)
    assert torch.equal(dz != 0, want != 0)


def test_empty_and_odd_rows():
    T, E, k1 = 9, 40, 3
    z, idx, _, d_w = make(T, E, k1, seed=9)
    z[0] = -math.inf                      # no distribution: as padding
    z[1, :] = -math.inf
    z[1, 7] = 3.0                         # one expert is all
    z[2, idx[2].long()] = -math.inf       # the given experts have probability 0
    idx[3] = ref.EMPTY                    # no slot at all
    idx[4] = idx[4, 0]                    # one expert three times
    z[5] += 5000.0                        # far from 0
    z[6, ::2] = -30000.0
    got = balance(z, idx)
    check_balance(z, idx, None, got)
    assert int(got[0][E]) == T - 1
    for k2 in (3, 6, 40):
        dz = route_backward(z, idx, k2, d_w, counts=got[0], balance_coef=0.3, z_coef=0.01)
        want, mag = ref.route_backward(z, idx, k2, d_w, counts=got[0], c_bal=0.3, c_z=0.01)
        # a difference to 5000 is rounded to 2^-12 first: row 5 by itself
        rows = torch.arange(T, device=DEV) != 5
        check_dz(dz[rows], want[rows], mag[rows])
        assert torch.allclose(dz[5].double(), want[5], rtol=2.0 ** -9, atol=1e-6)
        assert (dz[0] == 0).all()


def test_padding_rows_are_not_read():
    T, E, k1 = 50, 64, 4
    z, idx, m, d_w = make(T, E, k1, seed=10, mask=True)
    clean = balance(z, idx, m)
    dz = route_backward(z, idx, 8, d_w, counts=clean[0], balance_coef=0.3, z_coef=0.1, token_mask=m)
    z[~m] = float("nan")
    idx[~m] = 1 << 20
    d_w[~m] = float("inf")
    again = balance(z, idx, m, ws=clean[3])
    for a, b in zip(clean[:3], again[:3]):
        assert torch.equal(a, b)
    assert moe.moe_read_device_status(clean[3]) == 0
    assert torch.equal(dz, route_backward(z, idx, 8, d_w, counts=clean[0], balance_coef=0.3, z_coef=0.1,
                                          token_mask=m, ws=clean[3]))
    assert moe.moe_read_device_status(clean[3]) == 0
    none = torch.zeros(T, dtype=torch.bool, device=DEV)
    counts, loss, prob, _ = balance(z, idx, none, ws=clean[3])
    assert (counts == 0).all() and (loss == 0).all() and (prob == 0).all()
    dz = route_backward(z, idx, 8, d_w, counts=counts, balance_coef=0.3, z_coef=0.1, token_mask=none)
    assert (dz == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_logits_show(bad):
    z, idx, _, d_w = make(20, 64, 4, seed=11)
    counts = balance(z, idx)[0]
    clean = route_backward(z, idx, 64, d_w, counts=counts, balance_coef=0.3)
    z[7, 3] = bad
    got = balance(z, idx)
    assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
    fine = balance(torch.zeros_like(z), idx, ws=got[3])  # the next call is not touched by it
    assert torch.isfinite(fine[1]).all() and torch.isfinite(fine[2]).all()
    dz = route_backward(z, idx, 64, d_w, counts=counts, balance_coef=0.3)
    assert torch.isnan(dz[7]).all()
    rows = torch.arange(20, device=DEV) != 7
    assert torch.equal(dz[rows], clean[rows])


@pytest.mark.parametrize("E", [40, 300])
def test_all_experts_with_a_nan_at_a_given_one(E):
    # k2 beyond E is all experts, also where the k2 set is searched for; the
    # other rows are as without the NaN
    z, idx, _, d_w = make(9, E, 4)
    want, got = torch.empty(9, E, device=DEV), torch.empty(9, E, device=DEV)
    moe.moe_route_backward(z, idx, E, d_w, want)
    bad = z.clone()
    bad[3, int(idx[3, 1])] = float("nan")
    moe.moe_route_backward(bad, idx, 2 ** 31 - 1, d_w, got)
    torch.cuda.synchronize()
    assert torch.isnan(got[3]).any()
    keep = [t for t in range(9) if t != 3]
    assert torch.equal(got[keep], want[keep])


def test_counts_of_many_batches():
    # the counts' sum needs more than 32 bits
    T, E, k1, k2 = 6, 16, 2, 4
    z, idx, _, d_w = make(T, E, k1)
    counts = torch.full((E + 1,), 2 ** 30, dtype=torch.int32, device=DEV)
    counts[::2] = 2 ** 31 - 1
    counts[E] = T
    dz = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(z, idx, k2, d_w, dz, counts=counts, balance_coef=0.5, z_coef=0.01)
    want, mag = ref.route_backward(z, idx, k2, d_w, counts, 0.5, 0.01)
    check_dz(dz, want, mag)


def test_a_repeated_expert_counts_each_time():
    T, E, k1, k2 = 7, 48, 4, 8
    z, idx, _, d_w = make(T, E, k1)
    idx[:, 2] = idx[:, 0]
    idx[4] = idx[4, 1]
    counts, loss, prob, _ = balance(z, idx)
    assert torch.equal(counts.cpu().long(), ref.balance(z, idx, None)[0].long())
    dz = torch.empty(T, E, device=DEV)
    moe.moe_route_backward(z, idx, k2, d_w, dz)
    want, mag = ref.route_backward(z, idx, k2, d_w)
    check_dz(dz, want, mag)


def test_ids_out_of_range():
    z, idx, _, d_w = make(30, 64, 4, seed=12)
    hole = idx.clone()
    hole[3, 1] = ref.EMPTY
    hole[8, 0] = ref.EMPTY
    want = balance(z, hole)
    dz = route_backward(z, hole, 8, d_w, ws=want[3])
    assert moe.moe_read_device_status(want[3]) == 0
    idx[3, 1], idx[8, 0] = 64, -5
    got = balance(z, idx, ws=want[3])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert moe.moe_read_device_status(want[3]) == moe.MOE_ERR_DEVICE_CHECK
    assert torch.equal(route_backward(z, idx, 8, d_w, ws=want[3]), dz)
    assert moe.moe_read_device_status(want[3]) == moe.MOE_ERR_DEVICE_CHECK
    assert torch.equal(route_backward(z, idx, 8, d_w), dz)  # without a workspace too


def test_captured_replayed_and_on_a_side_stream():
    z, idx, m, d_w = make(500, 128, 8, seed=13, mask=True)
    z2, idx2, m2, d_w2 = make(500, 128, 8, seed=14, mask=True)
    counts, loss, prob, ws = balance(z, idx, m)
    dz = torch.empty(500, 128, device=DEV)
    s = torch.cuda.Stream()

    def step(stream=None):
        moe.moe_balance_loss(z, idx, 0.01, 0.001, counts, loss, ws, token_mask=m, prob_mean=prob, stream=stream)
        moe.moe_route_backward(z, idx, 16, d_w, dz, counts=counts, balance_coef=0.01, z_coef=0.001,
                               token_mask=m, stream=stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in ((z, z2), (idx, idx2), (m, m2), (d_w, d_w2)):
        a.copy_(b)
    torch.cuda.synchronize()
    step(stream=s)
    torch.cuda.synchronize()
    want = [t.clone() for t in (counts, loss, prob, dz)]
    for t in (counts, loss, prob, dz):
        t.fill_(7)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((counts, loss, prob, dz), want):
        assert torch.equal(got, w)


def test_outputs_of_no_tokens():
    z, idx = torch.empty(0, 16, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    counts, loss, prob, _ = balance(z, idx)
    assert (counts == 0).all() and (loss == 0).all() and (prob == 0).all()
    moe.moe_route_backward(z, idx, 4, torch.empty(0, 2, device=DEV), torch.empty(0, 16, device=DEV))


@pytest.mark.parametrize("T,E", [(24, 16), (300, 128)])
def test_training_a_routers_adapters(T, E):
    # adapters beside the router, its logits routed, losses and weights back to the adapters:
    # the gradients are those of the 64-bit chain over the same route
    k1, k2, d = 4, 8, 256
    c = ref.Case(T, d, E, 8, 3, "runs", seed=15)
    ws, bws = c.workspace(), moe.balance_workspace(T, E)
    z, u = torch.empty(T, E, device=DEV), torch.empty(T, 8, device=DEV)
    idx = torch.empty(T, k1, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k1, device=DEV)
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, z, ws, u_out=u)
    moe.moe_route(None, None, None, z, k1, k2, idx, w)
    counts, loss, _, _ = balance(z, idx, c_bal=0.1, c_z=0.01, ws=bws)
    d_w = torch.randn(T, k1, device=DEV)
    dz = torch.empty(T, E, device=DEV, dtype=torch.bfloat16)
    moe.moe_route_backward(z, idx, k2, d_w, dz, counts=counts, balance_coef=0.1, z_coef=0.01)
    da, db = torch.empty(c.n, 8, d, device=DEV), torch.empty(c.n, 8, E, device=DEV)
    dx = torch.empty(T, d, device=DEV)
    moe.moe_adapter_backward(dz, c.x, c.w.t().contiguous(), c.adapter, c.a, c.b, c.scale, u, da, db, ws, dx=dx)
    assert moe.moe_read_device_status(ws) == 0 and moe.moe_read_device_status(bws) == 0

    x, a, b = (t.double().requires_grad_() for t in (c.x, c.a, c.b))
    per = torch.cat([a, torch.zeros(1, 8, d, device=DEV, dtype=torch.float64)])
    row = torch.where(c.adapter == ref.EMPTY, torch.full_like(c.adapter, c.n), c.adapter).long()
    s = torch.cat([c.scale.double(), torch.zeros(1, device=DEV, dtype=torch.float64)])[row]
    perb = torch.cat([b, torch.zeros(1, 8, E, device=DEV, dtype=torch.float64)])
    uu = torch.einsum("td,trd->tr", x, per[row]) * s[:, None]
    zz = x @ c.w.double().t() + c.bias.double() + torch.einsum("tr,tro->to", uu, perb[row])
    in_k2 = ref.k2_set(z, idx, k2)
    ww = torch.softmax(zz.masked_fill(~in_k2, -math.inf), 1).gather(1, idx.long())
    share = counts[:E].double() / (T * k1)
    total = (ww * d_w.double()).sum() + 0.1 * E * (share * torch.softmax(zz, 1).mean(0)).sum() \
        + 0.01 * torch.logsumexp(zz, 1).square().mean()
    total.backward()
    # dlogits were rounded to bf16 (2^-8 each): every gradient is linear in them
    for got, want in ((da, a.grad), (db, b.grad), (dx, x.grad)):
        assert float((got.double() - want).norm()) <= (2.0 ** -8 + 2.0 ** -14) * float(want.norm())

"""Plain 64-bit forms of the adapter calls, the balance loss and the route's
gradient, and the error bounds the kernels are held to.

Bounds are elementwise and count roundings: a float32 sum of K products, in
any order and with truncating adders, is off by at most (K + 2) 2^-23 times
the sum of the products' magnitudes; u may be carried as bf16 parts, two or
more (2^-16 relative); an output is rounded once (float32 2^-24, bf16 2^-8).
"""
import math

import torch

from routed_expert_layer_route_b200 import moe

EMPTY = moe.MOE_EMPTY_SLOT
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def adapter_rows(T, n, kind, gen, device):
    """kind: "mixed" every row its own adapter or none, "runs" runs of rows,
    "one" all rows one adapter, "none" no adapter at all."""
    ids = torch.randint(0, n + 1, (T,), generator=gen, device=device)
    if kind == "runs":
        ids = ids[torch.arange(T, device=device) // 37 * 37 % max(T, 1)]
    elif kind == "one":
        ids = torch.full_like(ids, n - 1)
    elif kind == "none":
        ids = torch.full_like(ids, n)
    return torch.where(ids < n, ids, torch.full_like(ids, EMPTY)).int()


class Case:
    """Seeded inputs of one adapter projection on the GPU."""

    def __init__(self, T, din, dout, r, n, kind="mixed", seed=0, device="cuda:0"):
        g = torch.Generator(device=device)
        g.manual_seed(seed * 7919 + T + din + dout + r + n)

        def normal(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)

        self.T, self.din, self.dout, self.r, self.n = T, din, dout, r, n
        self.x = normal(T, din, std=1.0)
        self.w = normal(dout, din, std=din ** -0.5)
        self.bias = normal(dout, std=0.5, dtype=torch.float32)
        self.a = normal(n, r, din, std=din ** -0.5)
        self.b = normal(n, r, dout, std=r ** -0.5)
        self.scale = torch.rand(n, generator=g, device=device) + 0.5
        self.adapter = adapter_rows(T, n, kind, g, device)
        self.dy = normal(T, dout, std=1.0)
        self.u = normal(T, r, std=1.0, dtype=torch.float32)

    def workspace(self):
        return moe.adapter_workspace(self.T, self.din, self.dout, self.r, self.n)


def _by_adapter(adapter, n):
    return [(adapter == i).nonzero()[:, 0] for i in range(n)]


def inner(x, a, adapter, scale):
    """u [T x r] in 64 bits and its error bound."""
    n, r, din = a.shape
    u = torch.zeros(x.shape[0], r, dtype=torch.float64, device=x.device)
    e = torch.zeros_like(u)
    for i, t in enumerate(_by_adapter(adapter, n)):
        s = 1.0 if scale is None else float(scale[i])
        u[t] = s * (x[t].double() @ a[i].double().t())
        # the sum, the factor and the store: din + 2 + 2 roundings
        e[t] = s * (din + 4) * 2.0 ** -23 * (x[t].double().abs() @ a[i].double().abs().t())
    return u, e


def linear(x, w, bias, adapter, a, b, scale, product=None):
    """(y, error bound without the output's rounding, u, u's error bound)."""
    n, r, din = a.shape
    u, eu = inner(x, a, adapter, scale)
    if product is None:
        y = x.double() @ w.double().t()
        mag = x.double().abs() @ w.double().abs().t()
    else:
        y = product.double().clone()
        mag = y.abs()
    e = torch.zeros_like(y)
    for i, t in enumerate(_by_adapter(adapter, n)):
        y[t] += u[t] @ b[i].double()
        mag[t] += u[t].abs() @ b[i].double().abs()
        e[t] += (eu[t] + 2.0 ** -16 * u[t].abs()) @ b[i].double().abs()
    if bias is not None:
        y += bias.double()
        mag += bias.double().abs()
    # one sum of din + 2 r (two parts) + bias and product
    e += (din + 2 * r + 4) * 2.0 ** -23 * mag
    return y, e, u, eu


def outer(u, z, adapter, n, eu=None):
    """g [n x r x D] = sum of u_t z_t^T over each adapter's rows, and its error bound."""
    g = torch.zeros(n, u.shape[1], z.shape[1], dtype=torch.float64, device=z.device)
    e = torch.zeros_like(g)
    for i, t in enumerate(_by_adapter(adapter, n)):
        ui, zi = u[t].double(), z[t].double()
        g[i] = ui.t() @ zi
        per = 2.0 ** -16 + (2 * len(t) + 4) * 2.0 ** -23
        e[i] = per * (ui.abs().t() @ zi.abs())
        if eu is not None:
            e[i] += eu[t].t() @ zi.abs()
    return g, e


def check(got, want, bound, what=""):
    """Every element within its bound and one rounding to got's type, and the
    whole within 2^-15 (the parts of u) and that rounding in the 2-norm."""
    h = HALF_STEP[got.dtype]
    g = got.double()
    assert torch.isfinite(g).all(), what
    far = (g - want).abs() - (bound + h * (want.abs() + bound))
    assert float(far.max()) <= 0.0 if far.numel() else True, \
        "%s: %d elements beyond their bound, worst by %.3g" % (what, int((far > 0).sum()), float(far.max()))
    norm = float(want.norm())
    if norm > 0:
        rel = float((g - want).norm()) / norm
        assert rel <= 2.0 ** -15 + h, "%s: relative error %.3g" % (what, rel)


# ---------------------------------------------------------------- router training
def live_rows(logits, mask):
    live = torch.ones(logits.shape[0], dtype=torch.bool, device=logits.device)
    if mask is not None:
        live &= mask.bool()
    return live & ~(logits == -math.inf).all(1)


def balance(logits, idx, mask):
    """(counts [E + 1], P [E], L_bal, L_z) in 64 bits."""
    E = logits.shape[1]
    live = live_rows(logits, mask)
    z = logits[live].double()
    slots = idx[live].flatten()
    ok = (slots >= 0) & (slots < E)
    counts = torch.bincount(slots[ok].long(), minlength=E)
    N, R = int(live.sum()), int(counts.sum())
    if N == 0:
        return torch.zeros(E + 1, dtype=torch.int64), torch.zeros(E, dtype=torch.float64), 0.0, 0.0
    P = torch.softmax(z, 1).sum(0) / N
    bal = E * float((counts.double() / max(R, 1)) @ P)
    zl = float(torch.logsumexp(z, 1).square().sum() / N)
    return torch.cat([counts, torch.tensor([N], device=counts.device)]).cpu(), P, bal, zl


def k2_set(logits, idx, k2):
    """[T x E] bool: the given experts and, of the others, those of the largest
    logits (equal ones by the lower index), min(k2, E) in all."""
    T, E = logits.shape
    given = torch.zeros(T, E + 1, dtype=torch.bool, device=logits.device)
    ok = (idx >= 0) & (idx < E)
    given.scatter_(1, torch.where(ok, idx.long(), torch.full_like(idx.long(), E)), True)
    given = given[:, :E]
    key = torch.where(given, torch.full_like(logits, math.inf), logits + 0.0)
    order = torch.sort(key.double() + torch.where(given, 1.0, 0.0), dim=1, descending=True,
                       stable=True)[1]
    place = torch.empty_like(order).scatter_(1, order, torch.arange(E, device=logits.device)
                                             .expand(T, E))
    return given | (place < min(k2, E))


def weights(z, in_k2):
    """Eq. 2 over a fixed set, 64 bits: w = softmax over the set."""
    w = torch.softmax(z.masked_fill(~in_k2, -math.inf), 1)
    return torch.nan_to_num(w, nan=0.0)


def route_backward(logits, idx, k2, d_w, counts=None, c_bal=0.0, c_z=0.0, d_loss=1.0, mask=None):
    """(dlogits, its magnitude: the sum of the magnitudes of the terms) in 64 bits."""
    T, E = logits.shape
    z = logits.double()
    live = live_rows(logits, mask)
    dz, mag = torch.zeros_like(z), torch.zeros_like(z)
    if d_w is not None:
        ok = (idx >= 0) & (idx < E)
        at = torch.where(ok, idx.long(), torch.full_like(idx.long(), E))
        g = torch.zeros(T, E + 1, dtype=torch.float64, device=z.device)
        g.scatter_add_(1, at, torch.where(ok, d_w, torch.zeros_like(d_w)).double())
        g = g[:, :E]
        w = weights(z, k2_set(logits, idx, k2))
        dz += w * (g - (w * g).sum(1, keepdim=True))
        mag += w * (g.abs() + (w * g.abs()).sum(1, keepdim=True))
    if counts is not None:
        p = torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
        lse = torch.nan_to_num(torch.logsumexp(z, 1, keepdim=True), neginf=0.0)
        n = counts.to(z.device).double()
        f = n[:E] / max(float(n[:E].sum()), 1.0)
        per = d_loss / max(float(n[E]), 1.0)
        pf = (p @ f)[:, None]
        dz += per * p * (c_bal * E * (f - pf) + 2.0 * c_z * lse)
        mag += abs(per) * p * (abs(c_bal) * E * (f + pf) + 2.0 * abs(c_z) * lse.abs())
    dz[~live] = 0.0
    mag[~live] = 0.0
    return dz, mag

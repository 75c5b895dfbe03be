"""Cases of the adapter and router-training operators, with their plain forms.

Four calls of the package, for a routed layer that serves and tunes many low-rank
adapters on one set of frozen weights:

  moe_adapter_linear    y[t] = x[t] W^T + b + s_a (x[t] A_a^T) B_a, a the adapter of row t
  moe_adapter_backward  the gradients of x and of every adapter's A and B
  moe_balance_loss      per-expert counts, the load-balance loss and the z loss of a route
  moe_route_backward    the router logits' gradient: through the routing weights
                        (Eq. 2: a softmax over the k2 best experts) and both losses

An adapter's matrices are stored by rank: A [n x r x din], B [n x r x dout].
"""
import math

import torch

own = False

EMPTY = 0x7FFFFFFF  # a row without an adapter, a slot without an expert


# ------------------------------------------------------------------ the cases
def linear(name, T, din, dout, r, n, out, rows, bias, keep_u, base=True):
    """rows: how rows get their adapters, "request" (each row its own request's) or
    "runs" (prompts: runs of rows); base False: the product is there, the adapters' part is added."""
    return {"name": name, "op": "linear", "T": T, "din": din, "dout": dout, "r": r, "n": n,
            "out": out, "rows": rows, "bias": bias, "keep_u": keep_u, "base": base}


def backward(name, T, din, dout, r, n, out, rows, need_dx):
    return {"name": name, "op": "backward", "T": T, "din": din, "dout": dout, "r": r, "n": n,
            "out": out, "rows": rows, "need_dx": need_dx}


def balance(name, T, E, k1, mask, variable):
    """variable: routes with fewer than k1 experts (empty slots); mask: padding rows."""
    return {"name": name, "op": "balance", "T": T, "E": E, "k1": k1, "mask": mask,
            "variable": variable}


def route(name, T, E, k1, k2, out, mask, variable, losses):
    """losses: the balance and z losses' gradients are added."""
    return {"name": name, "op": "route", "T": T, "E": E, "k1": k1, "k2": k2, "out": out,
            "mask": mask, "variable": variable, "losses": losses}


def listed():
    return [
        # one token's router logits, the request's adapter beside the shared router
        linear("decode_1_router", 1, 2048, 128, 16, 8, "float32", "request", True, False),
        # a decode batch, every row another request, hidden to hidden
        linear("decode_32_hidden", 32, 2048, 2048, 16, 32, "bfloat16", "request", False, False),
        # prompts of several requests through the router
        linear("prompt_4096_router", 4096, 2048, 128, 16, 8, "float32", "runs", True, False),
        # odd sizes and an odd rank, the inner products kept for the backward pass
        linear("prompt_777_odd", 777, 1000, 1544, 10, 3, "float32", "runs", True, True),
        # the largest: long prompts, hidden to hidden at the larger width
        linear("prompt_8192_wide", 8192, 4096, 4096, 32, 16, "bfloat16", "runs", False, False),
        # tuning the router's adapters on a prompt batch
        backward("tune_4096_router", 4096, 2048, 128, 16, 4, "float32", "runs", True),
        # odd sizes, an odd rank, few rows for each adapter
        backward("tune_333_odd", 333, 1024, 520, 12, 5, "float32", "request", True),
        # tuning a wide projection's adapters
        backward("tune_8192_wide", 8192, 2048, 2048, 64, 8, "bfloat16", "runs", True),
        # a small batch's counts and losses, with padding rows
        balance("balance_64", 64, 128, 8, True, False),
        # a training step's worth of tokens over many experts
        balance("balance_65536", 65536, 512, 10, False, False),
        # odd sizes, variable routes, weights over all experts
        route("route_777_odd", 777, 300, 6, 300, "float32", True, True, True),
        # a training step's worth of tokens, gradient rounded for the next product
        route("route_65536", 65536, 512, 5, 20, "bfloat16", False, False, True),
    ]


def _size(rng, lo, hi, step):
    """A multiple of step between lo and hi, even over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "balance", "route"])
    if op in ("linear", "backward"):
        T = _size(rng, 1, 8192, 1)
        din, dout = _size(rng, 64, 4096, 8), _size(rng, 64, 4096, 8)
        r = _size(rng, 1, 64, 1)
        n = min(_size(rng, 1, 32, 1), 512 // r)
        out = rng.choice(["float32", "bfloat16"])
        rows = rng.choice(["request", "runs"])
        if op == "backward":
            din, dout = min(din, 2048), min(dout, 2048)
            c = backward("", T, din, dout, r, n, out, rows, rng.random() < 0.8)
        else:
            c = linear("", T, din, dout, r, n, out, rows, rng.random() < 0.5,
                       rng.random() < 0.3, rng.random() < 0.8)
            c["bias"] = c["bias"] and c["base"]
    else:
        T, E = _size(rng, 1, 65536, 1), _size(rng, 8, 512, 1)
        k1 = min(E, _size(rng, 1, 10, 1))
        mask, variable = rng.random() < 0.5, rng.random() < 0.3
        if op == "balance":
            c = balance("", T, E, k1, mask, variable)
        else:
            k2 = E if rng.random() < 0.2 else min(E, k1 + _size(rng, 1, 24, 1) - 1)
            c = route("", T, E, k1, k2, rng.choice(["float32", "bfloat16"]), mask, variable,
                      rng.random() < 0.7)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _adapter_rows(T, n, rows, gen):
    """The adapter of each row: adapters of uneven popularity, one request in ten without."""
    pop = 1.0 / torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
    starts = torch.ones(T, device="cuda")
    if rows == "runs":  # about one request for 300 rows
        starts = (torch.rand(T, generator=gen, device="cuda") < 1.0 / 300).float()
    request = torch.cumsum(starts, 0).long()
    ids = torch.multinomial(pop, T + 1, replacement=True, generator=gen).int()
    none = torch.rand(T + 1, generator=gen, device="cuda") < 0.1
    return torch.where(none, torch.full_like(ids, EMPTY), ids)[request].contiguous()


def _tokens(T, d, gen):
    """Rows as a norm in front of the projection leaves them."""
    x = torch.randn(T, d, generator=gen, device="cuda")
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dev = {"device": "cuda"}

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    c, s = case, {"case": case}
    T = c["T"]
    if c["op"] in ("linear", "backward"):
        din, dout, r, n = c["din"], c["dout"], c["r"], c["n"]
        dtype = getattr(torch, c["out"])
        s["x"] = _tokens(T, din, gen)
        s["w"] = normal(dout, din, std=0.02)
        s["adapter"] = _adapter_rows(T, n, c["rows"], gen)
        s["a"] = normal(n, r, din, std=din ** -0.5)
        s["b"] = normal(n, r, dout, std=0.05)
        s["scale"] = torch.rand(n, generator=gen, device="cuda") + 0.5
        if c["op"] == "linear":
            s["bias"] = normal(dout, std=0.5, dtype=torch.float32) if c["bias"] else None
            s["product"] = None if c["base"] else normal(T, dout, dtype=dtype)
            s["y"] = torch.empty(T, dout, dtype=dtype, **dev)
            s["u"] = torch.empty(T, r, **dev) if c["keep_u"] else None
        else:
            s["dy"] = normal(T, dout, std=0.1)
            s["w_t"] = s["w"].t().contiguous()  # laid out once, the weights are frozen
            s["u"] = _inner(s["x"].float(), s["a"].float(), s["adapter"], s["scale"])[0]
            s["dx"] = torch.empty(T, din, dtype=dtype, **dev) if c["need_dx"] else None
            s["da"] = torch.empty(n, r, din, **dev)
            s["db"] = torch.empty(n, r, dout, **dev)
    else:
        E, k1 = c["E"], c["k1"]
        pop = torch.log(1.0 / torch.arange(1, E + 1, device="cuda"))
        pop = 0.3 * pop[torch.randperm(E, generator=gen, device="cuda")]
        s["logits"] = torch.randn(T, E, generator=gen, device="cuda") + pop
        idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)[1][:, :k1].int()
        if c["variable"]:  # each token keeps its first 1 to k1 experts
            kept = torch.randint(1, k1 + 1, (T, 1), generator=gen, device="cuda")
            idx = torch.where(torch.arange(k1, device="cuda") < kept, idx,
                              torch.full_like(idx, EMPTY))
        s["idx"] = idx.contiguous()
        s["mask"] = None
        if c["mask"]:  # one row in five is padding
            s["mask"] = torch.rand(T, generator=gen, device="cuda") < 0.8
        if c["op"] == "balance":
            s["counts"] = torch.empty(E + 1, dtype=torch.int32, **dev)
            s["loss"] = torch.empty(3, **dev)
            s["prob"] = torch.empty(E, **dev)
        else:
            s["d_w"] = normal(T, k1, std=0.1, dtype=torch.float32)
            s["d_loss"] = torch.full((1,), 1.5, **dev)
            s["counts"] = _counts(s["idx"], s["mask"], E)
            s["dz"] = torch.empty(T, E, dtype=getattr(torch, c["out"]), **dev)
    return s


BALANCE, ZETA = 0.01, 0.001  # the losses' coefficients


# ------------------------------------------------------------------ plain forms
def _inner(x, a, adapter, scale):
    """u = s_a x A_a^T of every row [T x r], and the same spread over all adapters' ranks [T x n r]."""
    n, r, _ = a.shape
    mine = (adapter.long()[:, None] == torch.arange(n, device=x.device)).float() * scale
    spread = (x @ a.reshape(n * r, -1).t()).view(-1, n, r) * mine[:, :, None]
    return spread.sum(1), spread.view(-1, n * r)


def _spread(u, adapter, n):
    mine = (adapter.long()[:, None] == torch.arange(n, device=u.device)).float()
    return (mine[:, :, None] * u[:, None, :]).reshape(u.shape[0], -1)


def _plain_linear(s):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    u, spread = _inner(x, a, s["adapter"], s["scale"])
    y = spread @ b.reshape(-1, b.shape[2])
    y = y + (x @ s["w"].float().t() if s["product"] is None else s["product"].float())
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["y"].dtype), "u": u if s["u"] is not None else None}


def _plain_backward(s):
    x, dy, a, b = s["x"].float(), s["dy"].float(), s["a"].float(), s["b"].float()
    n, r, din = a.shape
    _, v = _inner(dy, b, s["adapter"], s["scale"])
    out = {"da": (v.t() @ x).view(n, r, din),
           "db": (_spread(s["u"], s["adapter"], n).t() @ dy).view(n, r, -1), "dx": None}
    if s["dx"] is not None:
        out["dx"] = (dy @ s["w"].float() + v @ a.reshape(n * r, din)).to(s["dx"].dtype)
    return out


def _counts(idx, mask, E):
    """Routed slots of every expert, and the tokens, over the rows that count."""
    live = torch.ones(idx.shape[0], dtype=torch.bool, device=idx.device) if mask is None else mask
    at = torch.where(live[:, None] & (idx != EMPTY), idx.long(), torch.full_like(idx.long(), E))
    n = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    n.scatter_add_(0, at.flatten(), torch.ones_like(at.flatten(), dtype=torch.int32))
    n[E] = live.sum()
    return n


def _softmax(z):
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    return e / total, top + torch.log(total)


def _plain_balance(s):
    E = s["case"]["E"]
    counts = _counts(s["idx"], s["mask"], E)
    p, lse = _softmax(s["logits"])
    sq = lse.square()
    if s["mask"] is not None:
        p, sq = p * s["mask"][:, None], sq * s["mask"][:, None]
    tokens = counts[E].clamp(min=1)
    share = counts[:E].double() / counts[:E].sum().clamp(min=1)
    prob = p.sum(0, dtype=torch.float64) / tokens
    bal, zl = E * (share * prob).sum(), sq.sum(dtype=torch.float64) / tokens
    return {"counts": counts, "prob": prob.float(),
            "loss": torch.stack([BALANCE * bal + ZETA * zl, bal, zl]).float()}


def _plain_route(s):
    c, z, idx = s["case"], s["logits"], s["idx"]
    E = c["E"]
    # the given experts, and after them those of the largest logits, k2 in all
    there = idx != EMPTY
    at = torch.where(there, idx.long(), torch.full_like(idx.long(), E))
    g = torch.zeros(z.shape[0], E + 1, device=z.device)
    given = g.scatter(1, at, 1.0)[:, :E] > 0
    g = g.scatter_add(1, at, torch.where(there, s["d_w"], torch.zeros_like(s["d_w"])))[:, :E]
    rank = torch.sort(torch.where(given, torch.full_like(z, math.inf), z), dim=1,
                      descending=True, stable=True)[1][:, :c["k2"]]
    among = torch.zeros_like(z).scatter(1, rank, 1.0) > 0
    w, _ = _softmax(torch.where(among, z, torch.full_like(z, -math.inf)))
    dz = w * (g - (g * w).sum(1, keepdim=True))
    if c["losses"]:
        p, lse = _softmax(z)
        n = s["counts"]
        share = n[:E].float() / n[:E].sum().clamp(min=1)
        per = s["d_loss"] / n[E].clamp(min=1)
        dz = dz + per * p * (BALANCE * E * (share - (p * share).sum(1, keepdim=True))
                             + 2 * ZETA * lse)
    if s["mask"] is not None:
        dz = dz * s["mask"][:, None]
    return {"dz": dz.to(s["dz"].dtype)}


PLAIN = {"linear": _plain_linear, "backward": _plain_backward, "balance": _plain_balance,
         "route": _plain_route}


# ------------------------------------------------------------------ the package's calls
_workspaces = {}  # one for each set of sizes, as a program keeps them


def _workspace(make, *sizes):
    key = (make.__name__,) + sizes
    if key not in _workspaces:
        _workspaces[key] = make(*sizes)
    return _workspaces[key]


def _own_linear(moe, s):
    (T, din), (n, r, dout) = s["x"].shape, s["b"].shape
    ws = _workspace(moe.adapter_workspace, T, din, dout, r, n)
    w = s["w"]
    if s["product"] is not None:
        w = None
        s["y"].copy_(s["product"])
    moe.moe_adapter_linear(s["x"], w, s["bias"], s["adapter"], s["a"], s["b"], s["scale"],
                           s["y"], ws, u_out=s["u"])
    return {"y": s["y"], "u": s["u"]}


def _own_backward(moe, s):
    (T, din), (n, r, dout) = s["x"].shape, s["b"].shape
    ws = _workspace(moe.adapter_workspace, T, din, dout, r, n)
    moe.moe_adapter_backward(s["dy"], s["x"], s["w_t"], s["adapter"], s["a"], s["b"], s["scale"],
                             s["u"], s["da"], s["db"], ws, dx=s["dx"])
    return {"da": s["da"], "db": s["db"], "dx": s["dx"]}


def _own_balance(moe, s):
    T, E = s["logits"].shape
    ws = _workspace(moe.balance_workspace, T, E)
    moe.moe_balance_loss(s["logits"], s["idx"], BALANCE, ZETA, s["counts"], s["loss"], ws,
                         token_mask=s["mask"], prob_mean=s["prob"])
    return {"counts": s["counts"], "prob": s["prob"], "loss": s["loss"]}


def _own_route(moe, s):
    c = s["case"]
    more = {}
    if c["losses"]:
        more = dict(counts=s["counts"], balance_coef=BALANCE, z_coef=ZETA, d_loss=s["d_loss"])
    moe.moe_route_backward(s["logits"], s["idx"], c["k2"], s["d_w"], s["dz"],
                           token_mask=s["mask"], **more)
    return {"dz": s["dz"]}


OWN = {"linear": _own_linear, "backward": _own_backward, "balance": _own_balance,
       "route": _own_route}


def run(state):
    if own:
        from routed_expert_layer_route_b200 import moe
        return OWN[state["case"]["op"]](moe, state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, T = case, case["T"]
    if c["op"] in ("linear", "backward"):
        din, dout, r, n = c["din"], c["dout"], c["r"], c["n"]
        size = 4 if c["out"] == "float32" else 2
        used = min(n, T)  # adapters that rows can have
        ab = 2 * used * r * (din + dout)
        if c["op"] == "linear":
            base = 2 * din * dout if c["base"] else size * T * dout
            return {"bytes": 2 * T * din + base + ab + 4 * T + size * T * dout
                    + (4 * T * r if c["keep_u"] else 0) + (4 * dout if c["bias"] else 0),
                    "flops": 2 * T * din * dout * bool(c["base"]) + 2 * T * r * (din + dout)}
        dx = (2 * din * dout + size * T * din) if c["need_dx"] else 0
        return {"bytes": 2 * T * (din + dout) + ab + 4 * T * (r + 1) + 4 * n * r * (din + dout) + dx,
                "flops": 2 * T * r * (din + 2 * dout)
                + (2 * T * din * (dout + r) if c["need_dx"] else 0)}
    E, k1 = c["E"], c["k1"]
    read = 4 * T * E + 4 * T * k1 + (T if c["mask"] else 0)
    if c["op"] == "balance":
        return {"bytes": read + 4 * (2 * E + 4), "flops": 5 * T * E}
    size = 4 if c["out"] == "float32" else 2
    return {"bytes": read + 4 * T * k1 + size * T * E + (4 * (E + 2) if c["losses"] else 0),
            "flops": (5 + 6 * c["losses"]) * T * E}


# ------------------------------------------------------------------ in 64 bits, apart from the above
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] in ("linear", "backward"):
        x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
        rows = [(s["adapter"] == i).nonzero()[:, 0] for i in range(c["n"])]
        scale = s["scale"].double()
        if c["op"] == "linear":
            y = s["product"].double() if not c["base"] else x @ s["w"].double().t()
            u = torch.zeros(c["T"], c["r"], dtype=torch.float64, device="cuda")
            for i, t in enumerate(rows):
                u[t] = scale[i] * (x[t] @ a[i].t())
                y[t] += u[t] @ b[i]
            if s["bias"] is not None:
                y += s["bias"].double()
            return {"y": y, "u": u if c["keep_u"] else None}
        dy, u = s["dy"].double(), s["u"].double()
        dx = dy @ s["w"].double()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for i, t in enumerate(rows):
            v = scale[i] * (dy[t] @ b[i].t())
            dx[t] += v @ a[i]
            da[i] = v.t() @ x[t]
            db[i] = u[t].t() @ dy[t]
        return {"da": da, "db": db, "dx": dx if c["need_dx"] else None}
    z, E, T = s["logits"].double(), c["E"], c["T"]
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    logp = torch.log_softmax(z, 1)
    lse = torch.logsumexp(z, 1)
    slots = s["idx"][live]
    count = torch.bincount(slots[slots != EMPTY].long(), minlength=E).double()
    tokens = max(1, int(live.sum()))
    share = count / max(1.0, float(count.sum()))
    if c["op"] == "balance":
        prob = logp[live].exp().sum(0) / tokens
        bal, zl = E * (share @ prob), lse[live].square().sum() / tokens
        return {"counts": None, "prob": prob,
                "loss": torch.stack([BALANCE * bal + ZETA * zl, bal, zl])}
    # the routing weights' part by the chain rule over their logarithms
    order = torch.argsort(s["logits"], dim=1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(1, order, torch.arange(E, device="cuda").expand(T, E))
    in_k2 = place < c["k2"]
    logw = z - torch.logsumexp(z.masked_fill(~in_k2, -math.inf), 1, keepdim=True)
    w = logw.exp().masked_fill(~in_k2, 0.0)
    there = s["idx"] != EMPTY
    at = s["idx"].long().masked_fill(~there, 0)
    wg = w.gather(1, at) * s["d_w"].double().masked_fill(~there, 0.0)
    dz = -w * wg.sum(1, keepdim=True)
    dz.scatter_add_(1, at, wg)
    if c["losses"]:
        p = logp.exp()
        d = float(s["d_loss"]) / tokens
        dz += d * BALANCE * E * (p * share - p * (p @ share)[:, None])
        dz += d * ZETA * 2 * lse[:, None] * p
    dz[~live] = 0.0
    return {"dz": dz}

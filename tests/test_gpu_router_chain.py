"""The routing weights' gradient from the layer's own output: y[t] = sum_s w[t, s]
out[pos[t, s]], so dL/dw[t, s] = <dy[t], out[pos[t, s]]> with out as
moe_expert_ffn writes it; then back through Eq. 2 to the logits and to a
router's adapters."""
import pytest
import torch

import tune_ref as ref
from routed_expert_layer_route_b200 import moe, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("T,k1,k2", [(1, 2, 4), (40, 4, 8), (300, 4, 64)])
def test_from_the_layers_output_to_the_routers_adapters(T, k1, k2):
    d, E, I, r, n = 256, 64, 128, 8, 3
    L = synth.make_layer(T, d, E, I, seed=11, device=DEV)
    c = ref.Case(T, d, E, r, n, seed=41)
    ws = moe.workspace(T, d, E, I, k1)
    aws = moe.adapter_workspace(T, d, E, r, n)
    z, u = torch.empty(T, E, device=DEV), torch.empty(T, r, device=DEV)
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, z, aws, u_out=u)
    idx, w = torch.empty(T, k1, dtype=torch.int32, device=DEV), torch.empty(T, k1, device=DEV)
    moe.moe_route(None, None, None, z, k1, k2, idx, w)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    slot, pos = (torch.empty(T * k1, dtype=torch.int32, device=DEV) for _ in range(2))
    moe.moe_permute(idx, E, offsets, slot, pos)
    out = torch.empty(T * k1, d, device=DEV)
    moe.moe_expert_ffn(c.x, offsets, slot, L.w_gate, L.w_up, L.w_down, k1, out, ws)
    dy = torch.randn(T, d, device=DEV)
    own = out[pos.long()].view(T, k1, d)
    d_w = (own * dy[:, None]).sum(2)
    dz = torch.empty(T, E, device=DEV, dtype=torch.bfloat16)
    moe.moe_route_backward(z, idx, k2, d_w, dz)
    da, db = torch.empty(n, r, d, device=DEV), torch.empty(n, r, E, device=DEV)
    moe.moe_adapter_backward(dz, c.x, None, c.adapter, c.a, c.b, c.scale, u, da, db, aws)
    # the same in 64 bits from the outputs of the routed experts on
    zz = z.double().requires_grad_()
    ww = torch.softmax(zz.masked_fill(~ref.k2_set(z, idx, k2), -float("inf")), 1).gather(1, idx.long())
    ((ww[:, :, None] * own.double()).sum(1) * dy.double()).sum().backward()
    # dz is rounded to bf16; its terms are off by 2^-16 of their magnitudes, and by what the
    # float32 sums over d values of d_w are: w_m (e_m + sum_i w_i e_i) for m in K2
    mag = (own.double().abs() * dy.double().abs()[:, None]).sum(2)
    terms = ref.route_backward(z, idx, k2, d_w)[1]
    bound = (2.0 ** -8 * float(zz.grad.norm()) + 2.0 ** -16 * float(terms.norm())
             + (1 + k1 ** 0.5) * d * 2.0 ** -24 * float((ww * mag).detach().norm()))
    assert float((dz.double() - zz.grad).norm()) <= bound
    v, ev = ref.inner(dz, c.b, c.adapter, c.scale)
    want, e = ref.outer(v, c.x, c.adapter, n, eu=ev)
    ref.check(da, want, e, "d_lora_a")
    want, e = ref.outer(u, dz, c.adapter, n)
    ref.check(db, want, e, "d_lora_b")
    assert moe.moe_read_device_status(ws) == 0 and moe.moe_read_device_status(aws) == 0

"""One workspace for calls of several kinds and sizes: "initialised once ...
calls leave it initialised" holds whichever calls come in between, as each
call that needs zeros at its start finds them."""
import pytest
import torch

import tune_ref as ref
from parity import assert_close_layer, run_layer
from routed_expert_layer_route_b200 import moe, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
CM = moe.MOE_WDOWN_CHANNEL_MAJOR


def initialised(size):
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    moe.moe_workspace_init(ws)
    return ws


def balance(T, E, ws, k1=4):
    g = torch.Generator(device=DEV).manual_seed(T * 31 + E)
    z = torch.randn(T, E, generator=g, device=DEV) * 2.0
    idx = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :min(k1, E)].int().contiguous()
    counts = torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)
    loss, prob = torch.full((3,), -7.0, device=DEV), torch.full((E,), -7.0, device=DEV)
    moe.moe_balance_loss(z, idx, 0.01, 0.001, counts, loss, ws, prob_mean=prob)
    return z, idx, counts, loss, prob


def check_balance(T, E, ws, what):
    z, idx, counts, loss, prob = balance(T, E, ws)
    assert torch.equal(counts.cpu().long(), ref.balance(z, idx, None)[0].long()), what
    for got, fresh in zip((counts, loss, prob), balance(T, E, moe.balance_workspace(T, E))[2:]):
        assert torch.equal(got, fresh), what


def adapters(T, ws, din=256, dout=192):
    c = ref.Case(T, din, dout, 16, 5, seed=21)
    y = torch.empty(T, dout, device=DEV)
    moe.moe_adapter_linear(c.x, c.w, c.bias, c.adapter, c.a, c.b, c.scale, y, ws)
    da, db = torch.empty(c.n, c.r, din, device=DEV), torch.empty(c.n, c.r, dout, device=DEV)
    moe.moe_adapter_backward(c.dy, c.x, None, c.adapter, c.a, c.b, c.scale, c.u, da, db, ws)
    return y, da, db


@pytest.mark.parametrize("order", [
    [(64, 64), (64, 128)], [(64, 512), (1, 8), (64, 512)], [(4096, 64), (64, 128), (64, 512)],
    [(64, 512), (64, 64), (64, 128), (64, 1024), (4096, 512), (4096, 64), (4096, 128), (4096, 1024),
     (64, 300), (5000, 128), (64, 512), (64, 256), (4096, 300)]], ids=len)
def test_balance_losses_of_several_expert_counts(order):
    ws = moe.balance_workspace(5000, 1024)
    for T, E in order * 2:
        check_balance(T, E, ws, (T, E))
    assert moe.moe_read_device_status(ws) == 0


def test_balance_losses_after_adapters_and_layers():
    d, E, I, k1 = 512, 64, 128, 4
    L = synth.make_layer(40, d, E, I, seed=5, device=DEV)
    size = max(moe.moe_workspace_size(40, d, E, I, k1), moe.moe_adapter_workspace_size(700, 256, 192, 16, 5),
               moe.moe_balance_workspace_size(700, 512))
    ws = initialised(size)
    for _ in range(2):
        check_balance(700, 512, ws, "first")
        adapters(700, ws)
        check_balance(64, 512, ws, "after adapters")
        adapters(20, ws)
        check_balance(700, 128, ws, "after few rows")
        run_layer(L, k1, 8, ws=ws)
        check_balance(64, 300, ws, "after a layer")
    assert moe.moe_read_device_status(ws) == 0


@pytest.mark.parametrize("T", [1, 5])
def test_decode_layers_after_adapters_and_balance_losses(T):
    d, E, I, k1 = 2048, 64, 128, 4
    L = synth.make_layer(T, d, E, I, seed=6, device=DEV)
    w_down = moe.moe_pack_w_down(L.w_down)
    want = run_layer(L, k1, 8, flags=CM, w_down=w_down)[0].cpu().numpy()
    size = max(moe.moe_workspace_size(T, d, E, I, k1), moe.moe_adapter_workspace_size(700, 256, 192, 16, 5),
               moe.moe_balance_workspace_size(700, 512))
    ws = initialised(size)
    fresh = adapters(700, moe.adapter_workspace(700, 256, 192, 16, 5))
    for _ in range(2):
        for got, w in zip(adapters(700, ws), fresh):
            assert torch.equal(got, w)
        assert_close_layer(run_layer(L, k1, 8, ws=ws, flags=CM, w_down=w_down)[0].cpu().numpy(), want, "adapters")
        balance(700, 512, ws)
        assert_close_layer(run_layer(L, k1, 8, ws=ws, flags=CM, w_down=w_down)[0].cpu().numpy(), want, "balance")

"""The decode layer's accumulator on a workspace that other calls use in
between: layers of another width, moe_route's and moe_permute's scratch."""
import pytest
import torch

from parity import assert_close_layer, run_layer
from routed_expert_layer_route_b200 import moe, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
CM = moe.MOE_WDOWN_CHANNEL_MAJOR


def between_width(ws):
    run_layer(synth.make_layer(40, 256, 64, 128, seed=8, device=DEV), 4, 8, ws=ws)


def between_route(ws):
    L = synth.make_layer(300, 512, 64, 64, seed=9, device=DEV)
    idx = torch.empty(300, 4, dtype=torch.int32, device=DEV)
    w = torch.empty(300, 4, device=DEV)
    moe.moe_route(L.x, L.w_router, None, None, 4, 8, idx, w, ws=ws)


def between_permute(ws):
    T, E, k1 = 3000, 1024, 4
    idx = torch.rand(T, E, device=DEV).argsort(1)[:, :k1].int().contiguous()
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    slots, pos = (torch.empty(T * k1, dtype=torch.int32, device=DEV) for _ in range(2))
    moe.moe_permute(idx, E, offsets, slots, pos, ws=ws)
    assert torch.equal(offsets[1:] - offsets[:-1],
                       torch.bincount(idx.flatten().long(), minlength=E).int())


@pytest.mark.parametrize("between", [between_width, between_route, between_permute])
@pytest.mark.parametrize("T", [1, 4])
def test_decode_layer(T, between):
    d, E, I, k1 = 2048, 64, 128, 4
    L = synth.make_layer(T, d, E, I, seed=7, device=DEV)
    w_down = moe.moe_pack_w_down(L.w_down)
    want = run_layer(L, k1, 8, flags=CM, w_down=w_down)[0].cpu().numpy()
    ws = moe.workspace(3000, d, 1024, I, k1)  # room for every call here
    for _ in range(2):
        between(ws)
        got = run_layer(L, k1, 8, ws=ws, flags=CM, w_down=w_down)[0].cpu().numpy()
        assert_close_layer(got, want)
    assert moe.moe_read_device_status(ws) == 0

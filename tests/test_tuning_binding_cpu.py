"""What the binding of the adapter and router-training calls refuses before the
library is called: a kernel is never given host memory or a strided buffer."""
import pytest
import torch

from routed_expert_layer_route_b200 import moe

HOST = -1  # get_device() of a tensor in host memory


@pytest.fixture
def no_library(monkeypatch):
    """A library that records calls."""
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(name) or moe.MOE_OK

        def moe_status_string(self, status):
            return b"refused"
    monkeypatch.setattr(moe, "lib", Library)
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    return calls


def arguments(T=4, d=64, E=32, r=4, n=2, k1=2):
    bf16, f32, i32 = (dict(dtype=t) for t in (torch.bfloat16, torch.float32, torch.int32))
    x, w = torch.zeros(T, d, **bf16), torch.zeros(E, d, **bf16)
    a, b, ad = torch.zeros(n, r, d, **bf16), torch.zeros(n, r, E, **bf16), torch.zeros(T, **i32)
    z, idx = torch.zeros(T, E), torch.zeros(T, k1, **i32)
    return {
        "moe_adapter_linear": dict(x=x, w=w, bias=None, adapter=ad, lora_a=a, lora_b=b, scale=None,
                                   y=torch.zeros(T, E)),
        "moe_adapter_backward": dict(dy=torch.zeros(T, E, **bf16), x=x, w_t=None, adapter=ad, lora_a=a,
                                     lora_b=b, scale=None, u=torch.zeros(T, r),
                                     d_lora_a=torch.zeros(n, r, d), d_lora_b=torch.zeros(n, r, E)),
        "moe_balance_loss": dict(logits=z, topk_idx=idx, balance_coef=0.1, z_coef=0.1,
                                 counts=torch.zeros(E + 1, **i32), loss=torch.zeros(3)),
        "moe_route_backward": dict(logits=z, topk_idx=idx, k2=4, d_topk_w=torch.zeros(T, k1),
                                   dlogits=torch.zeros(T, E))}


@pytest.mark.parametrize("name", sorted(arguments()))
def test_workspaces(name, no_library, monkeypatch):
    call, given = getattr(moe, name), arguments()[name]
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    where = {"ws": 0, "others": 0}
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device",
                        lambda t: where["ws" if t.numel() >= ws.numel() else "others"])
    call(**given, ws=ws)
    assert no_library == [name]  # all where the current device is
    for at, bad in ((HOST, ws), (1, ws), (0, torch.zeros(1 << 21, dtype=torch.uint8)[::2])):
        where["ws"] = at
        with pytest.raises(moe.MoeError) as refused:
            call(**given, ws=bad)
        assert refused.value.status == moe.MOE_ERR_INVALID_ARG
    where.update(ws=0, others=HOST)
    with pytest.raises(moe.MoeError):
        call(**given, ws=ws)
    assert no_library == [name]

"""A stream of another device than the object's (Router, BlockNorm) or the current one (MXFP4 layers) is
refused before anything is launched.  Streams and tensors are stand-ins: no device needed."""
import types

import pytest

from mixture_experts_routed_dispatch_amd import moe


class Stop(Exception):
    """Raised in place of a launch."""


def stop(*a, **k):
    raise Stop


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stop)


def stream(index):
    import torch
    return types.SimpleNamespace(device=torch.device("cuda", index), cuda_stream=0x1000)


@pytest.mark.parametrize("cls", [moe.Router, moe.BlockNorm])
def test_router_and_norm(cls):
    import torch
    o = cls.__new__(cls)
    o.device, o._index = torch.device("cuda", 0), 0
    with pytest.raises(ValueError, match="cuda:1"):
        o._call(stop, stream(1))
    with pytest.raises(Stop):
        o._call(stop, stream(0))


def test_layer_with_4bit_weights(monkeypatch):
    layer = moe.Layer.__new__(moe.Layer)
    layer.plan, layer.precision = 0, moe.MOE_MXFP4
    layer.T, layer.E, layer.I, layer.d, layer.k = 2, 4, 128, 256, 2
    layer._rows = moe._dense(2, 256)
    layer._weights = moe._dense(4, 256, 256), moe._dense(4, 256, 128)
    layer._mxfp4 = ((moe._dense(1), moe._dense(1)), (moe._dense(1), moe._dense(1)))
    layer._mxfp4_sizes = (1, 1, 1, 1)
    for name in ("moe_forward", "moe_forward_routed", "moe_prepare_weights", "moe_expand_weights"):
        monkeypatch.setattr(moe, name, stop)
    monkeypatch.setattr(moe, "_check", lambda *a: None)
    t = types.SimpleNamespace(numel=lambda: 1, is_contiguous=lambda: True, get_device=lambda: 0, device="cuda:0",
                              data_ptr=lambda: 0x1000)
    monkeypatch.setattr(moe, "_new", lambda *a: t)
    calls = [lambda s: layer.forward(t, t, t, t, t, t, t, y=t, stream=s),
             lambda s: layer.forward(t, t, t, t, t, t, t, stream=s),
             lambda s: layer.forward_routed(t, t, t, t, t, t, out=t, stream=s),
             lambda s: layer.forward_routed(t, t, t, t, t, t, stream=s),
             lambda s: layer.prepare_weights(t, t, stream=s),
             lambda s: layer.expand_weights(t, t, t, t, stream=s)]
    for f in calls:
        with pytest.raises(ValueError, match="cuda:1"):
            f(stream(1))
        with pytest.raises(Stop):
            f(stream(0))

"""Calls on tensors of another device than the current one are refused by the
binding, with or without a stream (no GPU needed: the tensors and the devices are
stand-ins, and what is looked for comes before any launch)."""
import pytest
import torch

from communication_efficient_gradient_amd import gq


class On:
    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.fixture
def two_devices(monkeypatch):
    now = {"device": 0}
    monkeypatch.setattr(gq, "_current_device", lambda: now["device"])
    monkeypatch.setattr(gq, "_raw_stream", lambda d: 0)
    return now


@pytest.mark.parametrize("stream", [None, 0, 1 << 20])
def test_only_the_current_device(two_devices, stream):
    for current in (0, 1):
        two_devices["device"] = current
        assert gq._queue(stream, On(current)) == (stream or 0)
        with pytest.raises(ValueError, match=f"current device is cuda:{current}"):
            gq._queue(stream, On(1 - current))


def test_calls_ask(two_devices, monkeypatch):
    """Every operator of a step asks before it launches: with a current device of 1
    each of these is refused, and the library is never reached."""
    two_devices["device"] = 1

    class Unreached:
        def __getattr__(self, name):
            def f(*args):
                if name.endswith("_workspace") or name == "gq_act_size":
                    return 0
                raise AssertionError(name + " was called")
            return f

    for f in ("_matrix", "_buffer", "_vec", "_space", "_form", "_block_form", "_block_weight",
              "_state"):
        monkeypatch.setattr(gq, f, lambda *a, **k: (0, 0))
    monkeypatch.setattr(gq, "_table", lambda *a: (0, 1))
    monkeypatch.setattr(gq, "_lib", Unreached())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    a = gq.gq_act(4, 6, gq.GQ_BF16, 128)
    t, d = torch.zeros(4, 6), gq.adamw(1e-3)
    calls = [lambda: gq.gq_act_pack(a, t, t, t), lambda: gq.gq_act_unpack(a, t, t, t),
             lambda: gq.gq_act_linear(a, t, t, t, t, None, t),
             lambda: gq.gq_act_wgrad(a, t, t, t, t),
             lambda: gq.gq_block_pack(a, t, t, t), lambda: gq.gq_block_unpack(a, t, t, t),
             lambda: gq.gq_block_pack_weight(a, t, (t, t)),
             lambda: gq.gq_block_linear(a, t, t, t, t, None, t),
             lambda: gq.gq_block_wgrad(a, t, t, t, t), lambda: gq.gq_adamw(d, t, t, t, t, 1),
             lambda: gq.gq_grad_norm(t, 1.0, t)]
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()

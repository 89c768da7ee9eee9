"""Tensors and streams of another device than the current one are refused by
the 4-bit and router-gradient calls (stand-ins for them: no GPU is needed)."""
import pytest

torch = pytest.importorskip("torch")


class On:
    def __init__(self, index):
        self.device, self.device_index = f"cuda:{index}", index

    def get_device(self):
        return self.device_index


def test_everything_has_to_be_on_the_current_device(monkeypatch):
    from mixture_experts_ffn_moe_amd import _lib
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    _lib._on_current(On(0), None, On(0))
    _lib._on_current(On(0), stream=On(0))
    with pytest.raises(ValueError, match="tensor is on cuda:1"):
        _lib._on_current(On(0), On(1))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        _lib._on_current(On(0), stream=On(1))

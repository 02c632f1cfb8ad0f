"""The binding of the experts' packing: where it launches and what it checks (no GPU needed: a
stand-in tensor says that it lives on a second GPU, and the packing itself is a recorder)."""

import pytest
import torch

import weight_only_bit_02_amd as awq
from weight_only_bit_02_amd import grouped

DEV = torch.device("cuda", 1)


class OnGpu1(torch.Tensor):
    """A host tensor that says cuda:1."""
    is_cuda = True
    device = DEV

    def get_device(self):
        return DEV.index


class Guard:
    """torch.cuda.device without a GPU: which device is current."""
    current = 0

    def __init__(self, device):
        self.device = torch.device(device)

    def __enter__(self):
        self.before, Guard.current = Guard.current, self.device.index

    def __exit__(self, *_):
        Guard.current = self.before


def _tensor(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu1)


@pytest.fixture
def launched(monkeypatch):
    """The device that is current at each packing."""
    devices = []

    def pack(W, s=None, flags=None, out=None, **_):
        devices.append(Guard.current)
        N, K = W.shape
        return out or grouped.PackedLinear(torch.zeros(N, K // 8), torch.zeros(N, 1), torch.zeros(N, 1), N, K)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(grouped, "quantize_pack", pack)
    monkeypatch.setattr(grouped, "alloc_packed", lambda N, K, *_: grouped.PackedLinear(
        torch.zeros(N, K // 8), torch.zeros(N, 1), torch.zeros(N, 1), N, K))
    return devices


def test_packs_on_the_device_of_the_weights(launched):
    W = _tensor(3, 4, 128)
    for s, calls in ((None, 1), (_tensor(128), 1), (_tensor(3, 128), 3)):
        launched.clear()
        w = awq.quantize_pack_experts(W, s, flags=_tensor(1, dtype=torch.int32))
        assert launched == [1] * calls and Guard.current == 0
        assert tuple(w.qweight.shape) == (3, 4, 16)


def test_refuses_scales_and_flags_of_another_kind(launched):
    W = _tensor(3, 4, 128)
    for s in (torch.zeros(128).half(), torch.zeros(3, 128).half(), _tensor(127), _tensor(2, 128), _tensor(3, 1, 128)):
        with pytest.raises(ValueError):
            awq.quantize_pack_experts(W, s)
    for s in ([1.0], _tensor(128, dtype=torch.float32), 3.0):
        with pytest.raises(TypeError):
            awq.quantize_pack_experts(W, s)
    with pytest.raises(ValueError):
        awq.quantize_pack_experts(W, flags=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        awq.quantize_pack_experts(W, flags=_tensor(1, dtype=torch.int64))
    assert not launched

"""gate / layer / project refuse a stream of another device than their
tensors': the library launches on the current device, and memory that the
binding allocates would lie on the stream's."""

import pytest
import torch

import block_scaled_fp4_topk_amd as m


class OnDevice:
    """A stream's attributes, none of which reach the GPU."""

    def __init__(self, index):
        self.device_index, self.device, self.cuda_stream = index, torch.device("cuda", index), 0


class Tensor:
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def test_stream_and_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert m._current(Tensor(), None) == torch.device("cuda", 0)
    assert m._current(Tensor(), OnDevice(0)) == torch.device("cuda", 0)
    with pytest.raises(ValueError, match="stream"):
        m._current(Tensor(), OnDevice(1))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        m._current(Tensor(), OnDevice(1))


@pytest.mark.gpu
def test_operators_refuse_it():
    from helpers import require_gpu
    require_gpu()
    from test_gpu_operators import adapted, experts, rnd
    x, w, ex = rnd(0, 4, 512), rnd(1, 8, 512), experts(8, 512, 256, 16)
    a = adapted(5, 64, 512, 16)
    for call in (lambda s: m.gate(x, w, 2, stream=s), lambda s: m.layer(x, w, 2, *ex, 16, stream=s), lambda s: m.project(*a, stream=s)):
        call(torch.cuda.Stream())
        torch.cuda.synchronize()
        with pytest.raises(ValueError, match="stream"):
            call(OnDevice(1))

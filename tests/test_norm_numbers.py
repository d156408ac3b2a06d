"""The numbers of a block norm (scale, h_scale, eps) as the library gets them:
what they are at each call, without a GPU."""

import struct

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as m


class FakeLibrary:
    """Stands where the library is called: keeps the problems that it is given."""

    def __init__(self):
        self.problems = []

    def _keep(self, p, *_):
        f = p._obj
        self.problems.append(tuple(struct.pack("f", v) for v in (f.scale, f.h_scale, f.eps)))
        return m.OK

    moe_fp4_block_norm = moe_fp4_block_norm_grad = _keep


@pytest.fixture
def calls(monkeypatch):
    """(the fake library, the calls of both directions with a scale, h_scale and eps) on CPU tensors"""
    fake = FakeLibrary()
    monkeypatch.setattr(m, "_lib", fake)
    monkeypatch.setattr(m, "_dev", lambda t, name, dtypes: t)
    monkeypatch.setattr(m, "_current", lambda t, stream: t.device)
    monkeypatch.setattr(m, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(m, "_norm_grad_need", lambda T, H: 256)
    h, y, w = torch.ones(2, 8), torch.ones(2, 8).bfloat16(), torch.ones(8)
    return fake, (lambda **k: m.block_norm(h, y, pre_w=w, **k), lambda **k: m.block_norm_grad(h, y, h, y, pre_w=w, **k))


def f32(*v):
    return tuple(struct.pack("f", x) for x in v)


@pytest.mark.parametrize("direction", [0, 1])
def test_a_tensor_that_changes_in_place(calls, direction):
    """A learned residual scale: every call takes the value that it has then."""
    fake, call = calls[0], calls[1][direction]
    s, c = torch.nn.Parameter(torch.tensor(0.5)), torch.tensor([1.5])
    e = np.array(1e-6)
    call(scale=s.detach(), h_scale=c, eps=e)
    with torch.no_grad():
        s.fill_(2.0)
    call(scale=s.detach(), h_scale=c, eps=e)
    c.fill_(-3.0)
    e[()] = 1e-3
    call(scale=s.detach(), h_scale=c, eps=e)
    same = s.detach()
    call(scale=same, h_scale=c, eps=e)
    same.fill_(4.0)
    call(scale=same, h_scale=c, eps=e)
    assert fake.problems == [f32(0.5, 1.5, 1e-6), f32(2.0, 1.5, 1e-6), f32(2.0, -3.0, 1e-3), f32(2.0, -3.0, 1e-3), f32(4.0, -3.0, 1e-3)]


@pytest.mark.parametrize("direction", [0, 1])
def test_the_sign_of_zero(calls, direction):
    fake, call = calls[0], calls[1][direction]
    for a, b in ((0.0, 0.0), (-0.0, 0.0), (0.0, -0.0), (0, -0.0), (-0.0, 0)):
        call(scale=a, h_scale=b)
        assert fake.problems[-1] == f32(a, b, 1e-6)


@pytest.mark.parametrize("direction", [0, 1])
def test_no_tensor_is_kept(calls, direction):
    import gc
    import weakref
    s = torch.tensor(0.75)
    gone = weakref.ref(s)
    calls[1][direction](scale=s)
    del s
    gc.collect()
    assert gone() is None


@pytest.mark.parametrize("direction", [0, 1])
@pytest.mark.parametrize("bad", ["0.5", None, torch.ones(2), [1.0]], ids=["text", "none", "two", "list"])
def test_no_number(calls, direction, bad):
    for name in ("scale", "h_scale", "eps"):
        with pytest.raises((TypeError, ValueError)):
            calls[1][direction](**{name: bad})
    assert calls[0].problems == []


@pytest.mark.gpu
def test_a_learned_scale():
    """A scale on the device, changed between two calls, gives what its value gives as a number."""
    from helpers import require_gpu
    require_gpu()
    h, y, w = torch.randn(3, 64, device="cuda"), torch.randn(3, 64, device="cuda").bfloat16(), torch.ones(64, device="cuda")
    s = torch.tensor(0.5, device="cuda")
    for value in (0.5, 2.0, -1.25):
        s.fill_(value)
        for a, b in zip(m.block_norm(h, y, pre_w=w, scale=s, h_scale=s) + m.block_norm_grad(h, y, h, y, pre_w=w, scale=s, h_scale=s)[:2],
                        m.block_norm(h, y, pre_w=w, scale=value, h_scale=value) +
                        m.block_norm_grad(h, y, h, y, pre_w=w, scale=value, h_scale=value)[:2]):
            assert torch.equal(a, b)

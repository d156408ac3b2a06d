"""gran_k of the products grouped by expert as the library gets it, without a
GPU: a whole number at each call, whatever holds it."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as m


@pytest.fixture
def call(monkeypatch):
    """A call on CPU tensors, and the group sizes that the library was given."""
    given = []

    class FakeLibrary:
        def _keep(self, p, *_):
            given.append(p._obj.gran_k)
            return m.OK

        def moe_fp4_grouped_workspace_bytes(self, *_):
            return m.OK

        moe_fp4_grouped = moe_fp4_grouped_dx = _keep

    m._grouped_problem.cache_clear()
    monkeypatch.setattr(m, "_lib", FakeLibrary())
    monkeypatch.setattr(m, "_dev", lambda t, name, dtypes: t)
    monkeypatch.setattr(m, "_current", lambda t, stream: t.device)
    monkeypatch.setattr(m, "_raw_stream", lambda stream, device: 0)
    x, dy, w = torch.ones(4, 64).bfloat16(), torch.ones(4, 8).bfloat16(), torch.zeros(2, 8, 32, dtype=torch.uint8)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)

    def run(gran_k, groups):
        sf = torch.zeros(2, 8, groups, dtype=torch.uint8)
        m.grouped(x, w, off, w_sf=sf, gran_k=gran_k)
        m.grouped_dx(dy, w, off, w_sf=sf, gran_k=gran_k)
        return given[-2:]

    yield run
    m._grouped_problem.cache_clear()


def test_a_tensor_that_changes_in_place(call):
    """(a remembered 16 beside scales of 32 would be scales read behind their end)"""
    g = torch.tensor(16)
    assert call(g, 4) == [16, 16]
    g.fill_(32)
    assert call(g, 2) == [32, 32]
    with pytest.raises(ValueError):
        call(g, 4)


@pytest.mark.parametrize("kind", [int, float, np.int64, np.uint8], ids=lambda k: k.__name__)
def test_any_whole_number(call, kind):
    assert call(kind(16), 4) == [16, 16] and call(kind(32), 2) == [32, 32]


@pytest.mark.parametrize("bad", [8, 64, 16.5, "16", torch.tensor(48)], ids=str)
def test_others(call, bad):
    with pytest.raises(ValueError, match="gran_k"):
        call(bad, 4)

"""Workspace sizes of the router, the layer and the projection, without a GPU."""

import ctypes

import pytest

import block_scaled_fp4_topk_amd as m


def project_need(T, N, K, gran=16, adapters=0, rank=0):
    n = ctypes.c_size_t(0)
    p = m.Linear(T, N, K, gran, m.OUT_BF16, adapters, rank)
    assert m.lib().moe_fp4_project_workspace_bytes(ctypes.byref(p), ctypes.byref(n)) == m.OK, m.lib().moefp4_last_error()
    return n.value


@pytest.mark.parametrize("T", [1, 40, 128, 129, 300, 1000, 2048, 8192])
@pytest.mark.parametrize("N,K", [(4096, 6144), (16, 256), (6144, 2048)])
def test_project_always_needs_a_workspace(T, N, K):
    """A caller that allocates what the query says has memory to pass: the call refuses NULL."""
    for gran in (16, 32):
        for adapters in (0, 4):
            assert project_need(T, N, K, gran, adapters, 16) > 0

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


# batches around every border of the forms (8/9, 64/65, 128/129, 2048, 8192 tokens; whole tiles) and between them
BATCHES = sorted(set(range(1, 300)) | {b + d for b in (512, 1024, 2048, 4096, 6000, 8192, 16384, 32768, 65536) for d in
                                       (-1, 0, 1)} | set(range(320, 9000, 61)) | set(range(128, 8200, 128)))


def grows(need, batches=BATCHES):
    last, at = 0, 0
    for T in batches:
        n = need(T)
        assert n >= last, f"T={T} needs {n} bytes, T={at} {last}"
        last, at = n, T
    return last


@pytest.mark.parametrize("w_fmt", [m.GATE_W_BF16, m.GATE_W_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,H", [(256, 6144), (8, 64), (96, 2048), (130, 520), (512, 1000), (384, 7168)])
def test_gate_workspace_serves_smaller_batches(E, H, w_fmt):
    g = m.make_gate(4, w_fmt=w_fmt)
    n = ctypes.c_size_t(0)

    def need(T):
        assert m.lib().moe_fp4_gate_workspace_bytes(ctypes.byref(g), T, E, H, ctypes.byref(n)) == m.OK
        return n.value
    grows(need)


@pytest.mark.parametrize("gran,adapters,rank", [(16, 0, 0), (32, 0, 0), (16, 8, 16), (32, 16, 64), (16, 511, 128), (32, 1, 8)])
@pytest.mark.parametrize("N,K", [(4096, 6144), (16, 256), (1968, 2048), (6144, 2048), (16384, 4096), (48, 16384)])
def test_project_workspace_serves_smaller_batches(N, K, gran, adapters, rank):
    grows(lambda T: project_need(T, N, K, gran, adapters, rank))


@pytest.mark.parametrize("gran,act", [(16, m.ACT_BF16), (32, m.ACT_BF16), (32, m.ACT_BF16_QUANT_FP8_K32),
                                      (32, m.ACT_BF16_QUANT_FP4_K32)])
@pytest.mark.parametrize("E,k,shared,H,I", [(257, 8, 1, 6144, 2048), (8, 2, 0, 512, 512), (512, 1, 0, 512, 512),
                                            (512, 8, 0, 512, 512), (33, 20, 1, 1024, 512), (4, 1, 1, 7168, 512)])
def test_layer_workspace_serves_smaller_batches(E, k, shared, H, I, gran, act):
    n = ctypes.c_size_t(0)
    for w_fmt in (m.GATE_W_BF16, m.GATE_W_F32):
        g = m.make_gate(k, shared=shared, w_fmt=w_fmt)

        def need(T):
            p = m.Problem(T, E, k + shared, H, I, gran, act, 0, 0, 0)
            assert m.lib().moe_fp4_layer_workspace_bytes(ctypes.byref(p), ctypes.byref(g), ctypes.byref(n)) == m.OK
            return n.value
        grows(need)


@pytest.mark.parametrize("T", [40, 1000])
def test_project_refuses_an_output_over_its_inputs(T):
    """In place, or with one byte in common: the tiled form reads x while other workgroups store.  (Addresses that
    are never dereferenced.)"""
    L = m.lib()
    N = K = 512
    p = m.Linear(T, N, K, 16, m.OUT_BF16, 2, 8)
    size = dict(x=T * K * 2, w=N * K // 2, w_sf=N * K // 16, w_gs=4, a=2 * 8 * K * 2, b=2 * N * 8 * 2, id=T * 4, scale=8)
    base = {n: (1 << 30) + (i << 28) for i, n in enumerate(size)}
    out = T * N * 2

    def call(at):
        ptr = [ctypes.c_void_p(base[n]) for n in size]
        return L.moe_fp4_project(ctypes.byref(p), *ptr, ctypes.c_void_p(at), ctypes.c_void_p(1 << 40), 1 << 40, None)
    for n in size:
        first = max(0, base[n] - out + 16)
        last = base[n] + (size[n] - 1) // 16 * 16
        for at in (base[n], first, last):
            assert call(at) == m.EINVAL and b"overlaps" in L.moefp4_last_error(), n

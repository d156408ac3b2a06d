"""Router, whole layer and adapted projection without a GPU: the library
exports them, and every argument it documents as refused is refused with its
status before any launch (the pointers here are never dereferenced)."""

import ctypes
import os

import pytest
import torch

import block_scaled_fp4_topk_amd as m

Z = ctypes.c_void_p(0)
F = ctypes.c_void_p(1 << 20)      # aligned, never read
ODD = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 46


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        pytest.fail("libmoefp4.so is not built (python -m block_scaled_fp4_topk_amd.build)")
    return m.lib()


def gate_struct(**kw):
    d = dict(top_k=8, scoring="softmax", renormalize=False, scale=1.0, shared=0, w_fmt=m.GATE_W_BF16)
    d.update(kw)
    return m.make_gate(**d)


def gate_ws(L, g, T=64, E=256, H=6144):
    n = ctypes.c_size_t(0)
    return L.moe_fp4_gate_workspace_bytes(ctypes.byref(g), T, E, H, ctypes.byref(n)), n.value


def test_exports(L):
    for n in ("moe_fp4_gate", "moe_fp4_gate_workspace_bytes", "moe_fp4_layer", "moe_fp4_layer_workspace_bytes",
              "moe_fp4_project", "moe_fp4_project_workspace_bytes"):
        assert hasattr(L, n), n
    for n in ("gate", "layer", "project"):
        assert callable(getattr(m, n)) and n in m.__all__


@pytest.mark.parametrize("kw,size,status", [
    (dict(), dict(), m.OK),
    (dict(), dict(T=0), m.OK),
    (dict(), dict(T=1), m.OK),
    (dict(), dict(T=1 << 24, H=8), m.OK),
    (dict(top_k=1), dict(E=1, H=8), m.OK),
    (dict(top_k=64, shared=256), dict(), m.OK),
    (dict(), dict(T=-1), m.EINVAL),
    (dict(), dict(E=0), m.EINVAL),
    (dict(), dict(H=0), m.EINVAL),
    (dict(), dict(H=12), m.EINVAL),
    (dict(top_k=0), dict(), m.EINVAL),
    (dict(top_k=9), dict(E=8), m.EINVAL),
    (dict(shared=-1), dict(), m.EINVAL),
    (dict(scoring=2), dict(), m.EINVAL),
    (dict(w_fmt=2), dict(), m.EINVAL),
    (dict(), dict(E=513), m.EUNSUPPORTED),
    (dict(shared=257), dict(), m.EUNSUPPORTED),
    (dict(shared=(1 << 31) - 1), dict(), m.EUNSUPPORTED),
    (dict(top_k=65), dict(), m.EUNSUPPORTED),
    (dict(), dict(T=(1 << 24) + 1), m.EUNSUPPORTED),
    (dict(), dict(H=(1 << 24) + 8), m.EUNSUPPORTED),
    (dict(), dict(T=1 << 24, H=1 << 16), m.EUNSUPPORTED),
])
def test_gate_sizes(L, kw, size, status):
    st, n = gate_ws(L, gate_struct(**kw), **size)
    assert st == status
    assert status == m.OK or len(L.moefp4_last_error()) > 0


def test_gate_refuses_before_launch(L):
    g = gate_struct()
    need = gate_ws(L, g)[1]
    call = lambda x, w, b, i, wt, ws, n, T=64: L.moe_fp4_gate(ctypes.byref(g), T, 256, 6144, x, w, b, i, wt, ws, n, Z)
    assert L.moe_fp4_gate_workspace_bytes(ctypes.byref(g), 1, 8, 8, None) == m.EINVAL
    assert L.moe_fp4_gate(None, 1, 8, 8, F, F, Z, F, F, F, BIG, Z) == m.EINVAL
    for k in (0, 1, 3, 4):
        p = [F, F, Z, F, F]
        p[k] = Z
        assert call(*p, F, BIG) == m.EINVAL and b"non-NULL" in L.moefp4_last_error()
    for k in range(5):
        p = [F, F, F, F, F]
        p[k] = ctypes.c_void_p((1 << 20) + (8 if k < 2 else 2))
        assert call(*p, F, BIG) == m.EINVAL and b"aligned" in L.moefp4_last_error()
    if need:
        assert call(F, F, Z, F, F, F, need - 1) == m.EWORKSPACE
    assert call(F, F, Z, F, F, Z, BIG) == m.EWORKSPACE
    assert call(F, F, Z, F, F, ctypes.c_void_p((1 << 20) + 128), BIG) == m.EINVAL
    assert call(Z, Z, Z, Z, Z, Z, 0, T=0) == m.OK


def problem(**kw):
    d = dict(T=4, E=257, top_k=9, H=6144, I=2048, gran_k=16, act_fmt=m.ACT_BF16, w13_order=0, out_fmt=0, w_layout=0)
    d.update(kw)
    return m.Problem(**d)


def layer_ws(L, p, g):
    n = ctypes.c_size_t(0)
    return L.moe_fp4_layer_workspace_bytes(ctypes.byref(p), ctypes.byref(g), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,gkw,status", [
    (dict(), dict(shared=1), m.OK),
    (dict(T=0), dict(shared=1), m.OK),
    (dict(T=9), dict(shared=1), m.OK),
    (dict(T=8192), dict(shared=1), m.OK),
    (dict(gran_k=32, act_fmt=m.ACT_BF16_QUANT_FP8_K32), dict(shared=1), m.OK),
    (dict(top_k=8), dict(shared=1), m.EINVAL),                 # top_k counts the shared experts
    (dict(), dict(shared=0), m.EINVAL),
    (dict(), dict(shared=-1, top_k=10), m.EINVAL),
    (dict(E=9), dict(shared=9, top_k=0), m.EINVAL),            # no routed expert
    (dict(E=8, top_k=8), dict(shared=1, top_k=7), m.OK),
    (dict(act_fmt=m.ACT_FP8_UE8M0_K32, gran_k=32), dict(shared=1), m.EINVAL),
    (dict(act_fmt=m.ACT_FP4_UE8M0_K32, gran_k=32), dict(shared=1), m.EINVAL),
    (dict(H=6000), dict(shared=1), m.EINVAL),                  # not a multiple of 32
    (dict(H=6080), dict(shared=1), m.EUNSUPPORTED),            # of 32, not of 256
    (dict(T=-1), dict(shared=1), m.EINVAL),
    (dict(), dict(shared=1, scoring=7), m.EINVAL),
    (dict(top_k=66), dict(shared=1, top_k=65), m.EUNSUPPORTED),
])
def test_layer_sizes(L, kw, gkw, status):
    st, n = layer_ws(L, problem(**kw), gate_struct(**gkw))
    assert st == status, L.moefp4_last_error()
    assert status != m.OK or kw.get("T") == 0 or n > 0


@pytest.mark.parametrize("T", [1, 4, 40])
def test_layer_refuses_before_launch(L, T):
    p, g = problem(T=T), gate_struct(shared=1)
    need = layer_ws(L, p, g)[1]
    # x gate_w bias w13 w13_sf w13_gs w2 w2_sf w2_gs out ids wts
    call = lambda a, ws, n, q=p: L.moe_fp4_layer(ctypes.byref(q), ctypes.byref(g), *a, ws, n, Z)
    full = [F, F, Z, F, F, Z, F, F, Z, F, Z, Z]
    for k in (0, 1, 3, 4, 6, 7, 9):
        a = list(full)
        a[k] = Z
        assert call(a, F, BIG) == m.EINVAL and b"non-NULL" in L.moefp4_last_error()
    for k in range(12):
        a = list(full)
        a[k] = ODD
        assert call(a, F, BIG) == m.EINVAL and b"aligned" in L.moefp4_last_error()
    assert call(full, F, need - 1) == m.EWORKSPACE
    assert call(full, Z, BIG) == m.EWORKSPACE
    assert call(full, ctypes.c_void_p((1 << 20) + 16), BIG) == m.EINVAL
    assert call([Z] * 12, Z, 0, problem(T=0)) == m.OK
    assert L.moe_fp4_layer(None, ctypes.byref(g), *full, F, BIG, Z) == m.EINVAL
    assert L.moe_fp4_layer(ctypes.byref(p), None, *full, F, BIG, Z) == m.EINVAL


def linear(**kw):
    d = dict(T=40, N=4096, K=6144, gran_k=16, out_fmt=m.OUT_BF16, adapters=4, rank=16)
    d.update(kw)
    return m.Linear(**d)


def project_ws(L, p):
    n = ctypes.c_size_t(0)
    return L.moe_fp4_project_workspace_bytes(ctypes.byref(p), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", [
    (dict(), m.OK),
    (dict(T=0), m.OK),
    (dict(T=1, N=16, K=256, adapters=0, rank=0), m.OK),
    (dict(adapters=0, rank=-3), m.OK),                         # rank is ignored without adapters
    (dict(adapters=511, rank=128), m.OK),
    (dict(T=8192, adapters=16, rank=64), m.OK),
    (dict(T=(1 << 24) - 1, N=16, K=256), m.OK),
    (dict(T=-1), m.EINVAL),
    (dict(N=0), m.EINVAL),
    (dict(K=0), m.EINVAL),
    (dict(K=24), m.EINVAL),
    (dict(gran_k=64), m.EINVAL),
    (dict(out_fmt=2), m.EINVAL),
    (dict(adapters=-1), m.EINVAL),
    (dict(rank=0), m.EINVAL),
    (dict(rank=12), m.EINVAL),
    (dict(K=288), m.EUNSUPPORTED),
    (dict(N=4104), m.EUNSUPPORTED),
    (dict(adapters=512), m.EUNSUPPORTED),
    (dict(rank=136), m.EUNSUPPORTED),
    (dict(T=1 << 24), m.EUNSUPPORTED),
    (dict(N=1 << 20, K=1 << 12), m.EUNSUPPORTED),
    (dict(N=1 << 62, K=1 << 62), m.EUNSUPPORTED),
    (dict(N=1 << 19, K=256, adapters=511, rank=24), m.EUNSUPPORTED),
    (dict(T=1 << 23, N=1 << 20, K=256, adapters=0), m.EUNSUPPORTED),
])
def test_project_sizes(L, kw, status):
    st, n = project_ws(L, linear(**kw))
    assert st == status, L.moefp4_last_error()


@pytest.mark.parametrize("T", [1, 40, 1000])
@pytest.mark.parametrize("adapters", [0, 4])
def test_project_refuses_before_launch(L, T, adapters):
    p = linear(T=T, adapters=adapters)
    need = project_ws(L, p)[1]
    # x w w_sf w_gs a b id scale out
    call = lambda a, ws, n, q=p: L.moe_fp4_project(ctypes.byref(q), *a, ws, n, Z)
    full = [F, F, F, Z] + [F if adapters else Z] * 4 + [F]
    for k in (0, 1, 2, 8) + ((4, 5, 6, 7) if adapters else ()):
        a = list(full)
        a[k] = Z
        assert call(a, F, BIG) == m.EINVAL and b"non-NULL" in L.moefp4_last_error()
    if not adapters:
        for k in (4, 5, 6, 7):
            a = list(full)
            a[k] = F
            assert call(a, F, BIG) == m.EINVAL and b"NULL without adapters" in L.moefp4_last_error()
    for k in range(9):
        a = list(full)
        if a[k].value or k == 3:
            a[k] = ODD
            assert call(a, F, BIG) == m.EINVAL and b"aligned" in L.moefp4_last_error()
    if need:
        assert call(full, F, need - 1) == m.EWORKSPACE
    assert call(full, Z, BIG) == m.EWORKSPACE
    assert call(full, ctypes.c_void_p((1 << 20) + 16), BIG) == m.EINVAL
    assert call([Z] * 9, Z, 0, linear(T=0)) in (m.OK,)
    assert L.moe_fp4_project(None, *full, F, BIG, Z) == m.EINVAL


def test_binding_takes_gpu_tensors_only():
    x, w = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(4, 256, dtype=torch.bfloat16)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    with pytest.raises(TypeError):
        m.gate(x, w, 2)
    with pytest.raises(TypeError):
        m.layer(x, w, 2, u8(4, 512, 128), u8(4, 512, 16), None, u8(4, 256, 128), u8(4, 256, 16), None, 16)
    with pytest.raises(TypeError):
        m.project(x, u8(16, 128), u8(16, 16), None, 16)
    for call in (lambda: m.gate(None, w, 2), lambda: m.project(None, u8(16, 128), u8(16, 16), None, 16)):
        with pytest.raises(TypeError):
            call()


def test_make_gate():
    g = m.make_gate(4, "sigmoid", True, 2.5, 1, m.GATE_W_F32)
    assert (g.top_k, g.shared, g.scoring, g.renormalize, g.w_fmt, g.scale) == (4, 1, m.SCORE_SIGMOID, 1, m.GATE_W_F32, 2.5)
    with pytest.raises(ValueError):
        m.make_gate(4, "relu")

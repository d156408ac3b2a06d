"""Products grouped by expert and block norms without a GPU: the library
exports them, and every argument they document as refused is refused with its
status before any launch (the pointers here are never dereferenced)."""

import ctypes
import os

import pytest
import torch

import block_scaled_fp4_topk_amd as m

Z = ctypes.c_void_p(0)
BIG = 1 << 46


def far(i):
    """Addresses a TiB apart, aligned, never read."""
    return ctypes.c_void_p((i + 1) << 40)


def odd(i, by):
    return ctypes.c_void_p(((i + 1) << 40) + by)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(m.LIB_PATH):
        pytest.fail("libmoefp4.so is not built (python -m block_scaled_fp4_topk_amd.build)")
    return m.lib()


def test_exports(L):
    for n in ("moe_fp4_grouped", "moe_fp4_grouped_dx", "moe_fp4_grouped_dw", "moe_fp4_block_norm", "moe_fp4_block_norm_grad",
              "moe_fp4_block_norm_grad_workspace_bytes"):
        assert hasattr(L, n), n
    for n in ("grouped", "grouped_dx", "grouped_dw", "block_norm", "block_norm_grad"):
        assert callable(getattr(m, n)) and n in m.__all__


def problem(**kw):
    d = dict(M=0, N=64, K=128, E=8, gran_k=0, out_fmt=0)
    d.update(kw)
    return m.Grouped(*(d[n] for n in ("M", "N", "K", "E", "gran_k", "out_fmt")))


BAD_SIZES = [(dict(M=-1), m.EINVAL), (dict(E=0), m.EINVAL), (dict(N=0), m.EINVAL), (dict(K=0), m.EINVAL), (dict(N=12), m.EINVAL),
             (dict(K=12), m.EINVAL), (dict(gran_k=8), m.EINVAL), (dict(out_fmt=2), m.EINVAL), (dict(E=513), m.EUNSUPPORTED),
             (dict(M=(1 << 24) + 1), m.EUNSUPPORTED), (dict(N=(1 << 20) + 8), m.EUNSUPPORTED), (dict(K=(1 << 20) + 8), m.EUNSUPPORTED),
             (dict(M=1 << 24, N=1 << 16), m.EUNSUPPORTED), (dict(M=1 << 24, K=1 << 16), m.EUNSUPPORTED),
             (dict(E=512, N=1 << 16, K=1 << 15), m.EUNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_SIZES)
def test_grouped_sizes(L, kw, status):
    p = problem(**kw)
    calls = (lambda: L.moe_fp4_grouped(ctypes.byref(p), Z, Z, Z, Z, Z, Z, Z, 0, Z),
             lambda: L.moe_fp4_grouped_dx(ctypes.byref(p), Z, Z, Z, Z, Z, Z, Z, 0, Z),
             lambda: L.moe_fp4_grouped_dw(ctypes.byref(p), Z, Z, Z, Z, 0, Z, 0, Z))
    for call in calls:
        assert call() == status and len(L.moefp4_last_error()) > 0


def test_grouped_refuses_before_launch(L):
    for fn in (L.moe_fp4_grouped, L.moe_fp4_grouped_dx):
        assert fn(None, Z, Z, Z, Z, Z, Z, Z, 0, Z) == m.EINVAL
        p = problem()
        assert fn(ctypes.byref(p), Z, Z, Z, Z, Z, Z, Z, 0, Z) == m.OK  # no rows: nothing to do
        p = problem(gran_k=16, K=48)
        assert fn(ctypes.byref(p), Z, Z, Z, Z, Z, Z, Z, 0, Z) == m.EINVAL and b"32" in L.moefp4_last_error()
        for gran in (0, 32):
            p = problem(M=16, gran_k=gran)
            good = [far(0), far(1), far(2) if gran else Z, Z, far(4), far(5)]
            call = lambda a: fn(ctypes.byref(p), *a, far(9), BIG, Z)
            for k in (0, 1, 4, 5):
                a = list(good)
                a[k] = Z
                assert call(a) == m.EINVAL and b"non-NULL" in L.moefp4_last_error()
            for k, by in ((0, 8), (1, 8), (4, 2), (5, 8)):
                a = list(good)
                a[k] = odd(k, by)
                assert call(a) == m.EINVAL and b"aligned" in L.moefp4_last_error()
            a = list(good)
            a[2] = Z if gran else far(2)
            assert call(a) == m.EINVAL and b"w_sf" in L.moefp4_last_error()
            if not gran:
                a = list(good)
                a[3] = far(3)
                assert call(a) == m.EINVAL
            for k in (0, 1, 4):  # out over an input, at its start
                a = list(good)
                a[5] = a[k]
                assert call(a) == m.EINVAL and b"overlaps" in L.moefp4_last_error()


def test_grouped_dw_refuses_before_launch(L):
    fn = L.moe_fp4_grouped_dw
    assert fn(None, Z, Z, Z, Z, 0, Z, 0, Z) == m.EINVAL
    p = problem(gran_k=16)
    assert fn(ctypes.byref(p), Z, Z, Z, Z, 0, Z, 0, Z) == m.EINVAL
    p = problem(M=16)
    good = [far(0), far(1), far(2), far(3)]
    call = lambda a: fn(ctypes.byref(p), *a, 0, far(9), BIG, Z)
    for k in range(4):
        a = list(good)
        a[k] = Z
        assert call(a) == m.EINVAL and b"non-NULL" in L.moefp4_last_error()
        a[k] = odd(k, 2 if k == 2 else 8)
        assert call(a) == m.EINVAL and b"aligned" in L.moefp4_last_error()
        if k < 3:
            a = list(good)
            a[3] = a[k]
            assert call(a) == m.EINVAL and b"overlaps" in L.moefp4_last_error()
    p = problem(M=0)
    assert fn(ctypes.byref(p), Z, Z, far(2), Z, 0, Z, 0, Z) == m.EINVAL  # dw is written whole
    assert fn(ctypes.byref(p), Z, Z, far(2), far(2), 0, Z, 0, Z) == m.EINVAL and b"overlaps" in L.moefp4_last_error()


def grouped_ws(L, direction, **kw):
    n = ctypes.c_size_t(0)
    return L.moe_fp4_grouped_workspace_bytes(ctypes.byref(problem(**kw)), direction, ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", BAD_SIZES)
def test_grouped_workspace_sizes(L, kw, status):
    for d in range(3):
        assert grouped_ws(L, d, **kw)[0] == status
    assert grouped_ws(L, 3)[0] == m.EINVAL and grouped_ws(L, -1)[0] == m.EINVAL
    assert L.moe_fp4_grouped_workspace_bytes(ctypes.byref(problem()), 0, None) == m.EINVAL


def test_grouped_workspace_serves_smaller_batches(L):
    """What a call asks for is never more than the workspace of a larger batch.  (The calls are refused in any case: their
    out lies over an input.)"""
    asked = 0
    for N, K, E in ((4096, 4096, 1), (64, 4096, 1), (4096, 64, 3), (1024, 2048, 8), (2048, 1024, 60), (8, 6144, 64), (1 << 20, 64, 1),
                    (3200, 1280, 17)):
        for d in range(3):
            have = 0
            for M in (1, 2, 7, 13, 40, 64, 65, 96, 200, 700, 2000, 5000, 8191, 60000):
                st, n = grouped_ws(L, d, M=M, N=N, K=K, E=E)
                assert st == m.OK and have <= n <= 64 << 20 and n % 256 == 0, (d, M, N, K, E)
                have = n
                p = ctypes.byref(problem(M=M, N=N, K=K, E=E))
                call = lambda ws, by: (L.moe_fp4_grouped, L.moe_fp4_grouped_dx)[d](p, far(0), far(1), Z, Z, far(4), far(0), ws, by, Z) \
                    if d < 2 else L.moe_fp4_grouped_dw(p, far(0), far(1), far(4), far(0), 0, ws, by, Z)
                st = call(Z, 0)
                assert st in (m.EWORKSPACE, m.EINVAL)
                if st == m.EWORKSPACE:
                    asked += 1
                    need = int(L.moefp4_last_error().split()[2])
                    assert need <= n, (d, M, N, K, E)
                    assert call(far(9), need - 1) == m.EWORKSPACE
                    assert call(odd(9, 64), need) == m.EINVAL and b"256" in L.moefp4_last_error()
                    assert call(far(9), need) == m.EINVAL and b"out overlaps" in L.moefp4_last_error()
    assert asked > 20
    # FP4 weights choose other tiles, within the same workspace
    for gran, E in ((16, 1), (16, 8), (32, 3), (32, 40)):
        for N, K in ((4096, 4096), (64, 4096), (2048, 512), (8, 6144)):
            for d in range(2):
                for M in (1, 13, 15, 29, 40, 64, 65, 96, 200, 700, 2000, 5000):
                    size = dict(M=M, N=N, K=K, E=E, gran_k=gran)
                    n, p = grouped_ws(L, d, **size)[1], ctypes.byref(problem(**size))
                    call = (L.moe_fp4_grouped, L.moe_fp4_grouped_dx)[d]
                    assert call(p, far(0), far(1), far(2), Z, far(4), far(0), far(9), n, Z) == m.EINVAL
                    assert b"out overlaps" in L.moefp4_last_error(), (d, size)
    # the workspace over an input or out
    p = ctypes.byref(problem(M=60, N=4096, K=4096, E=1))
    for k in (0, 1, 4, 5):
        assert L.moe_fp4_grouped_dx(p, far(0), far(1), Z, Z, far(4), far(5), far(k), BIG, Z) == m.EINVAL
        assert b"workspace overlaps" in L.moefp4_last_error()


def norm(**kw):
    d = dict(T=4, H=64, h_fmt=0, post_fmt=0, pre_fmt=0, gate_fmt=0, gate_kind=0, gate_sigmoid=0, scale=1.0, h_scale=1.0, eps=1e-6)
    d.update(kw)
    return m.Norm(*d.values())


def norm_ws(L, p):
    n = ctypes.c_size_t(0)
    return L.moe_fp4_block_norm_grad_workspace_bytes(ctypes.byref(p), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), m.EINVAL), (dict(H=0), m.EINVAL), (dict(H=12), m.EINVAL), (dict(h_fmt=2), m.EINVAL), (dict(pre_fmt=-1), m.EINVAL),
    (dict(gate_kind=4), m.EINVAL), (dict(gate_sigmoid=2), m.EINVAL), (dict(eps=-1.0), m.EINVAL), (dict(eps=float("nan")), m.EINVAL),
    (dict(scale=float("inf")), m.EINVAL), (dict(h_scale=float("nan")), m.EINVAL), (dict(H=16392), m.EUNSUPPORTED),
    (dict(T=(1 << 24) + 1), m.EUNSUPPORTED), (dict(T=0), m.OK), (dict(H=16384, T=1 << 24), m.OK)])
def test_norm_sizes(L, kw, status):
    p = norm(**kw)
    st, n = norm_ws(L, p)
    assert st == status and (n >= 256 if status == m.OK else len(L.moefp4_last_error()) > 0)
    if status != m.OK:
        assert L.moe_fp4_block_norm(ctypes.byref(p), *[Z] * 7, Z) == status
        assert L.moe_fp4_block_norm_grad(ctypes.byref(p), *[Z] * 13, 0, Z) == status


def test_norm_workspace_serves_smaller_batches(L):
    for H in (8, 512, 520, 6144, 16384):
        sizes = [norm_ws(L, norm(T=T, H=H))[1] for T in (0, 1, 5, 300, 700, 5000, 1 << 24)]
        assert sizes == sorted(sizes)


def test_block_norm_refuses_before_launch(L):
    p = norm(gate_kind=1)
    good = [far(i) for i in range(7)]  # h, y, post_w, gate, pre_w, h_out, n
    call = lambda a, q=p: L.moe_fp4_block_norm(ctypes.byref(q), *a, Z)
    for k in (0, 1, 3, 4, 5, 6):
        a = list(good)
        a[k] = Z
        assert call(a) == m.EINVAL, k
    for k in range(7):
        a = list(good)
        a[k] = odd(k, 8)
        assert call(a) == m.EINVAL and b"aligned" in L.moefp4_last_error()
    assert call([far(0), Z, far(2), Z, far(4), Z, far(6)], norm()) == m.EINVAL   # post_w without y
    assert call([far(0), Z, Z, far(3), far(4), Z, far(6)], norm(gate_kind=2)) == m.EINVAL
    assert call([far(0), Z, Z, Z, Z, Z, Z], norm()) == m.EINVAL                  # neither y nor pre_w
    assert call([far(0), far(1), Z, far(3), far(4), far(5), far(6)], norm()) == m.EINVAL  # a gate without a kind
    for out in (5, 6):
        for k in range(7):
            if k == out or (out, k) == (5, 0):
                continue
            a = list(good)
            a[out] = a[k]
            assert call(a) == m.EINVAL and b"overlaps" in L.moefp4_last_error(), (out, k)
    a = list(good)
    a[5] = odd(0, 64)  # not h itself, but into it
    assert call(a) == m.EINVAL
    assert call([Z] * 7, norm(T=0)) == m.OK


def test_block_norm_grad_refuses_before_launch(L):
    p = norm(gate_kind=1)
    need = norm_ws(L, p)[1]
    # dh, dn, h, y, post_w, gate, pre_w, d_h, d_y, d_post_w, d_gate, d_pre_w, workspace
    good = [far(i) for i in range(13)]
    call = lambda a, q=p, n=BIG: L.moe_fp4_block_norm_grad(ctypes.byref(q), *a, n, Z)
    for k in range(1, 13):
        a = list(good)
        a[k] = Z
        assert call(a) == (m.EWORKSPACE if k == 12 else m.EINVAL), k
    for k in range(13):
        a = list(good)
        a[k] = odd(k, 128 if k == 12 else 8)
        assert call(a) == m.EINVAL and b"aligned" in L.moefp4_last_error()
    assert call(good, n=need - 1) == m.EWORKSPACE
    for out in range(7, 13):
        for k in range(13):
            if k == out or (out, k) in ((7, 0), (7, 7)):
                continue
            a = list(good)
            a[out] = a[k]
            want = b"overlaps" if not (k == 0 and out == 7) else b""
            assert call(a) == m.EINVAL and want in L.moefp4_last_error(), (out, k)
    a = [Z] + good[1:]
    a[1] = a[2] = a[6] = a[11] = Z  # nothing to differentiate
    assert call(a) == m.EINVAL
    # no rows: the sums over rows are written all the same
    assert call([Z] * 13, norm(T=0)) == m.EWORKSPACE


def test_python_refuses():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    off = torch.zeros(9, dtype=torch.int32)
    w = torch.zeros((8, 16, 64), dtype=torch.bfloat16)
    for call in (lambda: m.grouped(x, w, off), lambda: m.grouped_dx(x, w, off), lambda: m.grouped_dw(x, x, off),
                 lambda: m.block_norm(x, x), lambda: m.block_norm_grad(x, None, None, y=x), lambda: m.grouped(None, w, off),
                 lambda: m.block_norm(None)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="go with pre_w"):
        m.block_norm_grad(x, x, None, y=x)


@pytest.mark.parametrize("eps,status", [(0.0, m.EINVAL), (9e-21, m.EINVAL), (1.01, m.EINVAL), (float("inf"), m.EINVAL), (1.01e-20, m.OK), (1.0, m.OK)])
def test_norm_eps(L, eps, status):
    assert norm_ws(L, norm(eps=eps))[0] == status

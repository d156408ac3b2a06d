"""Products grouped by expert: every form of the tiled kernel over sums long
enough for its loop to run as it does in large calls (all its buffers in turn
several times), with ragged sums, rows and columns, the output types, and adding
to what is there.  The bounds are those of test_gpu_grouped.py.  Which form a
size takes is asserted, so that another rule of choice cannot leave one untested."""

import ctypes

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu
from test_gpu_grouped import U32, Case, offsets_of, rows_of

NT, NN, TN = 0, 1, 2


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("few", "tile", "parts", "many", "far")]


def plan(form, M, E, N, K, gran=0):
    """moefp4::grouped_plan of csrc/kernels.h"""
    f = moe.lib()["_ZN6moefp412grouped_planEixxxxi"]
    f.restype, f.argtypes = Plan, [ctypes.c_int] + [ctypes.c_longlong] * 4 + [ctypes.c_int]
    p = f(form, M, E, N, K, gran)
    return {n: getattr(p, n) for n, _ in Plan._fields_}


def spread(M, E):
    return rows_of(((M, E), 0, 0))


TWO = [2100, 2000]
SHORT = [700, 1, 0, 513, 255, 128, 1100, 384, 65, 0, 833, 129]  # last tiles of every length
# form, gran, rows, N, K, tile (far: of the FP4 codes)
TILES = [(NT, 0, TWO, 4104, 456, 256), (NT, 0, TWO, 4104, 1024, 256), (NT, 0, (4000, 40), 2056, 392, 256), (NT, 0, SHORT, 5128, 584, 256),
         (NT, 16, TWO, 4104, 480, 256), (NT, 32, TWO, 4104, 480, 256), (NT, 16, (9000, 40), 1096, 416, 256), (NT, 32, SHORT, 5128, 608, 256),
         (NT, 16, TWO, 4104, 1024, 256), (NT, 32, TWO, 4104, 1024, 256),
         (NT, 0, (1111, 40), 1000, 696, 128), (NT, 0, (1111, 40), 1000, 712, 128), (NT, 0, (1111, 40), 1000, 1024, 128),
         (NT, 16, (1500, 40), 1096, 416, 128), (NT, 32, (1500, 40), 1096, 480, 128), (NT, 16, (1500, 40), 1096, 1024, 128),
         (NT, 0, [150, 0, 90, 60], 520, 456, 64), (NT, 16, (900, 40), 1096, 416, 64), (NT, 32, (900, 40), 1096, 480, 64),
         (NN, 0, TWO, 456, 4104, 256), (NN, 0, SHORT, 584, 5128, 256), (NN, 16, TWO, 456, 4128, 256), (NN, 32, TWO, 520, 4128, 256),
         (NN, 16, SHORT, 584, 5152, 256), (NN, 32, SHORT, 1024, 5152, 256),
         (NN, 0, (1111, 40), 456, 1000, 128), (NN, 16, (3000, 40), 456, 1056, 128), (NN, 32, (3000, 40), 648, 1056, 128),
         (NN, 0, [150, 0, 90, 60], 456, 520, 64), (NN, 16, (900, 40), 456, 1056, (64, 1)), (NN, 32, (900, 40), 456, 1056, (64, 1)),
         (NN, 16, (1500, 40), 456, 2080, (64, 0)), (NN, 32, (1500, 40), 584, 2080, (64, 0))]


AROUND = 3  # rows in front and behind that belong to no expert; the rule counts them


def rows_in(rows):
    return rows if isinstance(rows, list) else spread(*rows)


def expect(form, gran, rows, N, K, tile):
    rows = rows_in(rows)
    for M in (int(sum(rows)), int(sum(rows)) + AROUND):
        p = plan(form, M, len(rows), N, K, gran)
        size, far = tile if isinstance(tile, tuple) else (tile, p["far"])
        assert p == dict(few=0, tile=size, parts=1, many=0, far=far), p


@pytest.mark.parametrize("case", TILES, ids=str)
def test_which_form(case):
    expect(*case)


@pytest.mark.gpu
@pytest.mark.parametrize("case", TILES, ids=str)
def test_steady_state(case):
    require_gpu()
    form, gran, rows, N, K, _ = case
    c = Case(rows_in(rows), N, K, gran, gs=gran == 16, first=1, behind=AROUND - 1)
    (c.product if form == NT else c.dx)()


# weight gradients: rows, N, K, tile
DW = [([900, 0, 571, 3], 2056, 2568, 256), ([900, 0, 448, 3], 2056, 2568, 256), ([900, 333, 0], 520, 264, 128), ((900, 40), 2056, 40, 64),
      ((900, 40), 40, 2056, 64)]


@pytest.mark.parametrize("rows,N,K,tile", DW, ids=str)
def test_which_form_of_dw(rows, N, K, tile):
    expect(TN, 0, rows, N, K, tile)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,N,K,tile", DW, ids=str)
def test_dw_steady_state(rows, N, K, tile):
    """Set, and added to what is there: the same sums, one FP32 addition, an expert without rows kept bit for bit."""
    require_gpu()
    c = Case(rows_in(rows), N, K, first=1, behind=AROUND - 1)
    ref = c.dw()
    old = torch.randn((c.E, N, K), device="cuda")
    old[:, ::3] = -0.0
    for dtype, as_int in ((torch.float32, torch.int32), (torch.bfloat16, torch.int16)):
        start = old.to(dtype)
        out = moe.grouped_dw(c.dy, c.x, c.off, out=start.clone(), accumulate=True)
        torch.cuda.synchronize()
        for e, a, b in c.ranges():
            want = start[e] if a == b else (start[e].float() + ref[e]).to(dtype)
            assert torch.equal(out[e].view(as_int), want.view(as_int)), e


# float32 outputs beyond 256 MiB, which are stored past the caches
BIG = [(NT, TWO, 16640, 136), (NN, TWO, 136, 16640), (TN, [300, 200], 4104, 8200)]


@pytest.mark.parametrize("form,rows,N,K", BIG, ids=str)
def test_which_form_of_large_outputs(form, rows, N, K):
    expect(form, 0, rows, N, K, 256)
    assert 4 * (sum(rows) * (N if form == NT else K) if form != TN else len(rows) * N * K) > 256 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("form,rows,N,K", BIG, ids=str)
def test_large_outputs(form, rows, N, K):
    require_gpu()
    E, M, off = len(rows), sum(rows), offsets_of(rows)
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    x, dy, w = r(M, K), r(M, N), r(E, N, K)
    f = {NT: lambda **k: moe.grouped(x, w, off, **k), NN: lambda **k: moe.grouped_dx(dy, w, off, **k), TN: lambda **k: moe.grouped_dw(dy, x, off, **k)}[form]
    outs = [f(out_dtype=torch.float32), f()]
    if form == TN:
        outs.append(f(out=torch.ones((E, N, K), device="cuda"), accumulate=True) - 1)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        X, D, W = x[a:b].double(), dy[a:b].double(), w[e].double()
        P, Q, at, terms = {NT: (X, W.T, slice(a, b), K), NN: (D, W, slice(a, b), N), TN: (D.T, X, e, b - a)}[form]
        ref, bound = P @ Q, (terms + 16) * U32 * (P.abs() @ Q.abs())
        assert bool(((outs[0][at].double() - ref).abs() <= bound).all())
        assert torch.equal(outs[1][at], outs[0][at].bfloat16())
        if form == TN:  # (one addition of 1 and one subtraction: half a step of each result)
            assert bool(((outs[2][at].double() - ref).abs() <= bound + 2 * U32 * (1 + ref.abs() + bound)).all())
        del ref, bound, P, Q


@pytest.mark.gpu
@pytest.mark.parametrize("gran", [0, 16, 32])
@pytest.mark.parametrize("form", [NT, NN])
def test_neighbours_stay_outside(form, gran):
    """NaN and infinities in every other expert's rows, weights or scales, and in rows of no expert, reach no row of the
    others: ragged sums and short last tiles of the largest form, whose loads run into them."""
    require_gpu()
    N, K = (5128, 608) if form == NT else (584, 5152)
    expect(form, gran, SHORT, N, K, 256)
    c = Case(SHORT, N, K, gran, gs=gran == 16, first=1, behind=AROUND - 1)
    f = (lambda a, w, **k: moe.grouped(a, w, c.off, **k)) if form == NT else (lambda a, w, **k: moe.grouped_dx(a, w, c.off, **k))
    a, kw = c.x if form == NT else c.dy, dict(c.kw(), out_dtype=torch.float32)
    ref = f(a, c.w, **kw)
    bad, w, clean = a.clone(), c.w.clone(), torch.zeros(c.M, dtype=torch.bool, device="cuda")
    if gran:
        kw["w_sf"] = c.w_sf.clone()
    bad[:1], bad[-2:] = float("nan"), float("inf")
    for e, s, t in c.ranges():
        if e % 2:
            bad[s:t] = float("nan") if e % 4 == 1 else float("inf")
            if gran:
                kw["w_sf"][e] = 0x7F if gran == 16 else 0xFF
            else:
                w[e] = float("nan")
        else:
            clean[s:t] = True
    out = f(bad, w, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out[clean], ref[clean]) and not bool(torch.isfinite(out[~clean][1:-2]).any())

"""The router (moe_fp4_gate) against a plain FP64 implementation: expert ids
equal, weights within the error of an FP32 logit.

Inputs lie on a grid whose products sum without rounding in FP32 (integers up
to 127 or 2047 times powers of two, sums below 2^24), so the logits, and with
them the selection, are exact in any order of summation; ties (equal logits
are common on the grid, and whole ties are planted) go to the lower index.

Tolerance of the weights: the kernel evaluates exp of an exact argument z and
one division in FP32.  exp and the division are good to 2 ulp each, the sum
over E <= 512 scores adds E 2^-24 at most, renormalisation two roundings:
(E + 16) 2^-24 relative, plus 2^-24 |z| for the rounding of z - max(z)."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu

pytestmark = pytest.mark.gpu


def plain_gate(x, w, top_k, bias=None, scoring="softmax", renormalize=False, scale=1.0, shared=0):
    """numpy FP64; x [T, H], w [E, H] float64."""
    z = x @ w.T
    T, E = z.shape
    ok = np.isfinite(z)
    zf = np.where(ok, z, -np.inf)
    with np.errstate(all="ignore"):
        if scoring == "softmax":
            m = np.max(zf, 1, keepdims=True)
            p = np.where(ok, np.exp(zf - np.where(np.isfinite(m), m, 0)), 0.0)
            s = p.sum(1, keepdims=True)
            p = np.where(s > 0, p / np.where(s > 0, s, 1), 0.0)
        else:
            p = np.where(ok, 1 / (1 + np.exp(-zf)), 0.0)
    # (without a bias both scores grow with the logit, which is compared)
    sel = zf.copy() if bias is None else p + bias[None, :]
    sel[~ok | ~(sel > -np.inf)] = -np.inf
    ids = np.argsort(-sel, axis=1, kind="stable")[:, :top_k].astype(np.int32)
    left = np.take_along_axis(sel, ids, 1) > -np.inf
    wt = np.where(left, np.take_along_axis(p, ids, 1), 0.0)
    if renormalize:
        s = wt.sum(1, keepdims=True)
        wt = np.where(s > 0, wt / np.where(s > 0, s, 1), 0.0)
    wt = wt * scale
    ids = np.where(left, ids, -1)
    ids = np.concatenate([ids, np.tile(E + np.arange(shared, dtype=np.int32), (T, 1))], 1)
    return ids, np.concatenate([wt, np.ones((T, shared))], 1)


def grid_inputs(T, E, H, wf32, seed):
    rng = np.random.default_rng([seed, T, E, H])
    x = np.clip(np.rint(rng.standard_normal((T, H)) * 16), -127, 127) / 16
    unit = 2.0 ** -round(np.log2(np.sqrt(H)))
    if wf32:
        w = np.clip(np.rint(rng.standard_normal((E, H)) * 256), -2047, 2047) * (unit / 256)
    else:
        w = np.clip(np.rint(rng.standard_normal((E, H)) * 16), -127, 127) * (unit / 16)
    return x, w


def run(x, w, wf32, top_k, bias=None, **kw):
    xd = torch.from_numpy(x).bfloat16().cuda()
    wd = torch.from_numpy(w).to(torch.float32 if wf32 else torch.bfloat16).cuda()
    assert torch.equal(wd.double().cpu().nan_to_num(7), torch.from_numpy(w).nan_to_num(7))
    bd = None if bias is None else torch.from_numpy(bias).cuda()
    ids, wt = moe.gate(xd, wd, top_k, bias=bd, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), wt.cpu().numpy().astype(np.float64)


def check(got, want, zmax, E):
    ids, wt = got
    rids, rwt = want
    assert np.array_equal(ids, rids)
    tol = (E + 16 + np.ceil(zmax)) * 2.0 ** -24
    assert np.all(np.abs(wt - rwt) <= tol * np.abs(rwt)), np.max(np.abs(wt - rwt) / np.maximum(np.abs(rwt), 1e-300))


SHAPES = [(1, 8, 64), (2, 1, 8), (16, 256, 6144), (17, 256, 6144), (3, 257, 520), (40, 65, 2048), (129, 130, 72),
          (300, 512, 1000), (1, 384, 2048), (64, 64, 512), (1000, 96, 8)]


@pytest.mark.parametrize("wf32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d-E%d-H%d" % s)
def test_gate(shape, scoring, wf32):
    require_gpu()
    T, E, H = shape
    x, w = grid_inputs(T, E, H, wf32, 1)
    rng = np.random.default_rng(5)
    for top_k in sorted({1, min(8, E), min(E, 64)}):
        for bias in (None, (0.05 * rng.standard_normal(E)).astype(np.float32)):
            for renorm, scale, shared in ((False, 1.0, 0), (True, 2.5, min(1, 512 - E))):
                kw = dict(scoring=scoring, renormalize=renorm, scale=scale, shared=shared)
                b64 = None if bias is None else bias.astype(np.float64)
                check(run(x, w, wf32, top_k, bias, **kw), plain_gate(x, w, top_k, b64, **kw),
                      np.abs(x @ w.T).max() * 2, E)


@pytest.mark.parametrize("T", [4, 40])
def test_ties_take_the_lower_index(T):
    require_gpu()
    x, w = grid_inputs(T, 96, 256, False, 2)
    w[48:] = w[:48]          # every expert has a double
    w[10] = w[20] = w[5]
    for bias in (None, np.zeros(96, np.float32)):
        for sc in ("softmax", "sigmoid"):
            check(run(x, w, False, 9, bias, scoring=sc),
                  plain_gate(x, w, 9, None if bias is None else bias.astype(np.float64), scoring=sc), 20, 96)
    ids, _ = run(np.zeros((T, 256)), w, False, 5)
    assert np.array_equal(ids, np.tile(np.arange(5, dtype=np.int32), (T, 1)))


@pytest.mark.parametrize("T", [4, 40])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_experts_and_rows(T, scoring):
    """Bias -inf / NaN masks experts, until none is left; the lowest finite bias does not."""
    require_gpu()
    x, w = grid_inputs(T, 70, 512, False, 3)
    for keep in (70, 5, 2, 0):
        bias = np.full(70, -np.inf, np.float32)
        bias[::2] = np.nan
        bias[np.random.default_rng(keep).permutation(70)[:keep]] = np.float32(0.25)
        got = run(x, w, False, 4, bias, scoring=scoring, renormalize=True)
        check(got, plain_gate(x, w, 4, bias.astype(np.float64), scoring=scoring, renormalize=True), 20, 70)
        if keep == 0:
            assert np.all(got[0] == -1) and np.all(got[1] == 0)
    low = np.full(70, np.finfo(np.float32).min, np.float32)
    low[7] = 0
    ids, _ = run(x, w, False, 3, low, scoring=scoring)
    # score + lowest rounds to lowest for every expert but 7: a tie
    assert np.array_equal(ids, np.tile(np.array([7, 0, 1], np.int32), (T, 1)))


@pytest.mark.parametrize("T", [4, 40])
def test_logits_that_are_not_finite(T):
    """A NaN or infinite router row is never taken and stays out of the softmax; a NaN token takes nothing."""
    require_gpu()
    x, w = grid_inputs(T, 70, 512, False, 4)
    x[:, 3] = 1.0
    w[11] = np.nan
    w[12, 3] = np.inf
    w[13, 3] = -np.inf
    x[1, 5] = np.nan
    for sc in ("softmax", "sigmoid"):
        got = run(x, w, False, 6, scoring=sc, renormalize=True, shared=1)
        want = plain_gate(x, w, 6, scoring=sc, renormalize=True, shared=1)
        check(got, want, 20, 70)
        assert np.all(got[0][1, :6] == -1) and got[0][1, 6] == 70


def test_empty_batch_outputs_and_stream():
    require_gpu()
    w = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    ids, wt = moe.gate(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), w, 2)
    assert ids.shape == (0, 2) and wt.shape == (0, 2)
    # outputs that the caller gives are written whole and nothing beside them
    x, wn = grid_inputs(5, 96, 256, False, 6)
    buf = torch.full((7, 4), -77, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    xd, wd = torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(wn).bfloat16().cuda()
    s.wait_stream(torch.cuda.current_stream())
    ids, wt = moe.gate(xd, wd, 4, topk_ids=buf[1:6], stream=s)
    s.synchronize()
    want = plain_gate(x, wn, 4)
    assert np.array_equal(buf[1:6].cpu().numpy(), want[0]) and ids.data_ptr() == buf[1:6].data_ptr()
    assert bool((buf[0] == -77).all()) and bool((buf[6] == -77).all())


@pytest.mark.parametrize("T", [3, 150])
def test_captured_and_replayed(T):
    require_gpu()
    x, w = grid_inputs(T, 96, 256, False, 7)
    xd, wd = torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(w).bfloat16().cuda()
    moe.gate(xd, wd, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, wt = moe.gate(xd, wd, 4)
    for k in range(4):
        xn = np.roll(x, k, axis=0)
        xd.copy_(torch.from_numpy(xn).bfloat16())
        g.replay()
        torch.cuda.synchronize()
        check((ids.cpu().numpy(), wt.cpu().numpy().astype(np.float64)), plain_gate(xn, w, 4), 20, 96)
        moe.gate(xd, wd, 3)


def test_routes_the_forward():
    """gate -> forward with shared experts: the ids index the stacked weight tensors."""
    require_gpu()
    x, w = grid_inputs(20, 7, 512, False, 8)
    ids, wt = run(x, w, False, 2, scoring="sigmoid", renormalize=True, shared=1)
    p = moe.make_problem(20, 8, 3, 512, 256, 16)
    counts, offsets, _, _ = moe.route(p, torch.from_numpy(ids).cuda())
    assert int(offsets[-1]) == 60 and int(counts[7]) == 20

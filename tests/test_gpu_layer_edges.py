"""The whole layer's two-launch form at the ends of its ranges."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu

pytestmark = pytest.mark.gpu

HREL = {16: mp.U16, 32: 2.0 ** -17}


@pytest.mark.parametrize("gran,T", [(16, 1), (16, 8), (32, 1), (32, 2)])
def test_h_near_the_largest_float(gran, T):
    """h is finite in FP32, but rounded to bfloat16 it would be infinite: its products with small weights are
    ordinary numbers, those with zero are zero."""
    require_gpu()
    H = I = 256
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    x[:, 0] = 181 / 128 * 2.0 ** 63
    w13 = np.zeros((1, 2 * I, H // 2), np.uint8)
    w13[0, 3, 0] = 2          # gate row 3: 1.0 at column 0
    w13[0, I + 3, 0] = 4      # up row 3: 2.0
    one = 0x38 if gran == 16 else 127
    w13_sf = np.full((1, 2 * I, H // gran), one, np.uint8)
    rng = np.random.default_rng(1)
    w2 = rng.integers(0, 256, (1, H, I // 2), dtype=np.uint8)
    w2[0, 17] = 0
    small = 2.0 ** -100
    w2_sf = np.full((1, H, I // gran), one if gran == 16 else 27, np.uint8)
    gs = torch.tensor([small], device="cuda") if gran == 16 else None
    d = lambda v: torch.from_numpy(v).cuda()
    gw = torch.zeros((1, H), dtype=torch.bfloat16, device="cuda")
    out = moe.layer(x.cuda(), gw, 1, d(w13), d(w13_sf), None, d(w2), d(w2_sf), gs, gran, out_dtype=torch.float32)
    torch.cuda.synchronize()
    h = 2 * (181 / 128) ** 2 * 2.0 ** 126
    assert mp.weight(w13[0], w13_sf[0], None, gran)[3, 0] == 1 and h < np.finfo(np.float32).max
    V = mp.weight(w2[0], w2_sf[0], None if gs is None else small, gran)[:, 3]
    want = np.tile(h * V, (T, 1))
    got = out.double().cpu().numpy()
    # silu and the product 16 half steps, h's rounding, one product and the sum over zeros
    assert np.all(np.abs(got - want) <= (HREL[gran] + (16 + 64) * mp.U32) * np.abs(want)), np.abs(got - want).max()
    assert np.all(got[:, 17] == 0)


@pytest.mark.parametrize("gran,T", [(16, 1), (16, 8), (32, 2)])
def test_a_wait_that_is_given_up_shows_in_the_output(gran, T):
    """Every wait given up at once (the kernel itself runs to its end): no output of an unfinished FC1 looks like a
    number, and the calls after it are whole again."""
    require_gpu()
    from test_gpu_layer import Layer
    L = Layer(16, 1024, 512, gran, 41)
    x, gw = L.args(T, 0)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    want = moe.layer(x, gw, 4, *L.d, gran, workspace=ws)
    assert moe.abandoned_waits(ws) == 0 and bool(want.isfinite().all())
    torch.cuda.synchronize()
    try:
        moe.set_wait_looks(0)
        for dt in (torch.bfloat16, torch.float32):
            out = moe.layer(x, gw, 4, *L.d, gran, workspace=ws, out_dtype=dt)
            torch.cuda.synchronize()
            assert moe.abandoned_waits(ws) > 0 and bool(out.isnan().all())
    finally:
        moe.set_wait_looks(-1)
    assert torch.equal(moe.layer(x, gw, 4, *L.d, gran, workspace=ws), want) and moe.abandoned_waits(ws) == 0


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("gran,T", [(16, 8), (32, 2)])
def test_sixteen_experts_per_token_all_different(gran, T, shared):
    """The most experts that the two-launch form holds: 16 per token, with no routed one in common."""
    require_gpu()
    from test_gpu_layer import Layer
    E, k = 16 * T + shared, 16 - shared
    L = Layer(E, 512, 256, gran, 42, gs=gran == 16, T=T)
    L.gw[:] = 0
    for e in range(E - shared):
        L.gw[e, e // 16 if e < 16 * T else 0] = 8 + (e % 16) / 8
    L.x[:, :T] = np.eye(T)
    out = L.check(T, k, shared, renormalize=True)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("I", [2304, 4096, 6400])
def test_long_intermediate_rows(I, gran):
    """More than 8 chunks of an expert's rows in FC2: a step's 8 waves end inside one."""
    require_gpu()
    from test_gpu_layer import Layer
    L = Layer(5, 512, I, gran, 43, gs=gran == 16, T=8)
    for T in (1, 2, 8):
        L.check(T, 3, 1, scoring="sigmoid", renormalize=True)


@pytest.mark.parametrize("gran", [16, 32])
def test_512_experts(gran):
    require_gpu()
    from test_gpu_layer import Layer
    L = Layer(512, 256, 256, gran, 44, gs=gran == 16, T=8)
    for T in (1, 2, 8):
        L.check(T, 8, 2, renormalize=True)


@pytest.mark.parametrize("gran,T", [(16, 1), (16, 8), (32, 2), (16, 12)])
@pytest.mark.parametrize("E", [20, 300])
def test_renormalised_weights_of_scores_below_fp32(E, gran, T):
    """The layer's selection gives the router's weights, also where their scores are beyond FP32's range."""
    require_gpu()
    from test_gpu_gate_edges import check, planted
    rng = np.random.default_rng(45)
    H = I = 256
    z = -95 - (rng.permutation(E) + 16) / 64
    x, gw = (torch.from_numpy(v).bfloat16().cuda() for v in planted(T, z, H))
    d = [torch.from_numpy(v).cuda() for v in (*mp.fp4_tensor(rng, E, 2 * I, H, gran), *mp.fp4_tensor(rng, E, H, I, gran))]
    ids = torch.empty((T, 5), dtype=torch.int32, device="cuda")
    wts = torch.empty((T, 5), device="cuda")
    out = moe.layer(x, gw, 5, d[0], d[1], None, d[2], d[3], None, gran, scoring="sigmoid", renormalize=True, scale=2.5,
                    topk_ids=ids, topk_w=wts, out_dtype=torch.float32)
    rids, rwts = moe.gate(x, gw, 5, scoring="sigmoid", renormalize=True, scale=2.5)
    assert torch.equal(ids, rids) and torch.equal(wts, rwts) and abs(float(wts[0].sum()) - 2.5) < 1e-5
    check(T, z, False, 5, None, "sigmoid", 2.5)
    assert bool(out.isfinite().all()) and bool((out != 0).any())

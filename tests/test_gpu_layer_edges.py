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

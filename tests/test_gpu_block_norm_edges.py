"""The gradient of the block norms at its edges."""

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("H", [64, 512, 1024, 4096, 6144, 8192, 8200])
def test_a_branch_without_a_norm_has_its_gradient_whatever_it_holds(H, gate):
    """d_y = scale act(gate) D does not contain y where there is no norm after the layer: infinities and NaN of y leave
    every bit of d_y (0 times one of them would be NaN)."""
    require_gpu()
    T, inf, nan = 5, float("inf"), float("nan")
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    for stream in (torch.float32, torch.bfloat16):
        dh, y = r(T, H).to(stream), r(T, H).bfloat16()
        kw = dict(scale=0.5, h_scale=2.0, gate=None if gate is None else r(*{"channel": (H,), "token": (T,), "full": (T, H)}[gate]))
        for act in (None, "sigmoid"):
            want = moe.block_norm_grad(dh, None, None, y, gate_act=act, **kw)
            bad = y.clone()
            bad[0, 3], bad[1, H - 1], bad[2, 7], bad[4, :] = inf, -inf, nan, inf
            got = moe.block_norm_grad(dh, None, None, bad, gate_act=act, **kw)
            torch.cuda.synchronize()
            assert bool(torch.isfinite(want[1]).all())
            assert torch.equal(got[0], want[0]) and torch.equal(got[1].view(torch.int16), want[1].view(torch.int16)), (stream, act)


def test_a_closed_gate():
    """sigmoid of the types' lowest values and of -infinity is 0: nothing of y enters h', and no gradient y."""
    require_gpu()
    for H in (64, 1024, 8200):
        h, y = torch.zeros((4, H), device="cuda"), torch.full((4, H), 3e30, device="cuda").bfloat16()
        w = torch.ones(H, device="cuda")
        for dtype in (torch.bfloat16, torch.float32):
            g = torch.tensor([-float("inf"), torch.finfo(dtype).min, -200.0, -105.0], device="cuda").to(dtype)
            for gate in (g, g[:, None].expand(4, H).contiguous()):
                out, n = moe.block_norm(h, y, gate=gate, gate_act="sigmoid", pre_w=w)
                _, dy, _, dg, _ = moe.block_norm_grad(torch.ones_like(h), None, None, y, gate=gate, gate_act="sigmoid")
                assert not bool(out.any()) and not bool(n.any()) and not bool(dy.any()) and not bool(dg.any())

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


# sigmoid(g) = 1 / (1 + e) and its slope e / (1 + e)^2, e = exp(-g), in half steps of FP32 (2^-24): the exponential 4 (the
# instruction 2, its correction's addition and argument 1 each), the sum 1, the reciprocal 2, each product 1.  A relative
# error of e enters the slope times |1 - 2 e / (1 + e)| <= 1, those of the sum and the reciprocal twice.
SLOPE = (4 + 2 * (1 + 2) + 2) * 2.0 ** -24
TINY = 2.0 ** -125  # (smaller values are 0)


def slope64(g):
    e = torch.exp(-g.double().abs())
    return e / (1 + e) ** 2


def gates(n):
    g = torch.linspace(-110, 110, n - 8, device="cuda")
    return torch.cat([g, torch.tensor([0.0, 11.5, 17.4, -17.4, 3.0e38, -3.0e38, float("inf"), -float("inf")], device="cuda")])


@pytest.mark.parametrize("T,H", [(40, 64), (40, 1024), (3, 8192), (3, 8200), (2, 16384)])
def test_gate_gradient_over_the_whole_range(T, H):
    """The slope keeps its relative accuracy on both sides: of large gates 1 - sigmoid is what is left of the exponential.
    (D, y and scale are 1: the sums of D a are whole numbers, and the gradient's one rounding is that of the product.)"""
    require_gpu()
    dh, y = torch.ones((T, H), device="cuda"), torch.ones((T, H), device="cuda").bfloat16()

    def check(gate, terms):
        d = moe.block_norm_grad(dh, None, None, y, gate=gate, gate_act="sigmoid")[3]
        want = slope64(gate)
        err = (d.double() / terms - want).abs()
        bound = (SLOPE + (terms + 1) * 2.0 ** -24) * want + TINY
        if d.dtype is torch.bfloat16:
            bound = bound + 2.0 ** -8 * (want + bound)
        assert bool((err <= bound).all()), ((err / bound).max().item(), gate.flatten()[(err / bound).argmax()].item())

    full = gates(T * H).view(T, H)
    check(full, 1)
    check(full.bfloat16(), 1)
    check(gates(H), T)  # (the sum over T rows of equal values)
    for some in gates(80).split(T):
        per = torch.zeros(T, device="cuda")
        per[:some.numel()] = some
        check(per, H)


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

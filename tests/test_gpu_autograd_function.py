"""The grouped products and block norms inside a torch.autograd.Function, as a
trainer uses them: outside of one their results need no gradient; inside of one
the leaves get the gradients of the formulas (FP64)."""

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu
from test_gpu_block_norm import Case
from test_gpu_grouped import offsets_of

pytestmark = pytest.mark.gpu
U32, UBF = 2.0 ** -24, 2.0 ** -8


class Grouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, off):
        ctx.save_for_backward(x, w, off)
        return moe.grouped(x, w, off)

    @staticmethod
    def backward(ctx, dy):
        x, w, off = ctx.saved_tensors
        dy = dy.contiguous()
        return moe.grouped_dx(dy, w, off), moe.grouped_dw(dy, x, off), None


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, y, post, pre):
        h, n = moe.block_norm(h, y, post_w=post, pre_w=pre, scale=0.5)
        ctx.save_for_backward(h, y, post, pre)
        return h, n

    @staticmethod
    def backward(ctx, dh, dn):
        h, y, post, pre = ctx.saved_tensors
        d_h, d_y, d_post, _, d_pre = moe.block_norm_grad(dh.contiguous(), dn.contiguous(), h, y, post_w=post, pre_w=pre, scale=0.5)
        return d_h, d_y, d_post, d_pre


def leaves(*shapes, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").bfloat16().requires_grad_() for s in shapes]


def test_results_need_no_gradient():
    require_gpu()
    x, w, dy = leaves((6, 64), (2, 16, 64), (6, 16))
    off = offsets_of([2, 4])
    h, post = leaves((4, 64), (64,))
    for t in (moe.grouped(x, w, off), moe.grouped_dx(dy, w, off), moe.grouped_dw(dy, x, off), *moe.block_norm(h, h, post_w=post, pre_w=post)):
        assert not t.requires_grad and t.grad_fn is None


@pytest.mark.parametrize("rows", [[2, 0, 5], [70, 130, 9]], ids=str)
def test_grouped(rows):
    """dx and dW are sums of S exact products, off by (S + 16) half steps of FP32 of their magnitudes, rounded once."""
    require_gpu()
    M, E, N, K = sum(rows), len(rows), 136, 96
    x, w = leaves((M, K), (E, N, K))
    dy, = leaves((M, N), seed=1)
    off = offsets_of(rows)
    Grouped.apply(x, w, off).backward(dy.detach())
    o, X, W, D = off.tolist(), x.detach().double(), w.detach().double(), dy.detach().double()
    for e in range(E):
        s = slice(o[e], o[e + 1])
        for got, ref, mag, terms in ((x.grad[s], D[s] @ W[e], D[s].abs() @ W[e].abs(), N), (w.grad[e], D[s].T @ X[s], D[s].abs().T @ X[s].abs(), rows[e])):
            b = (terms + 16) * U32 * mag
            assert bool(((got.double() - ref).abs() <= b + UBF * (ref.abs() + b)).all())


def test_norm():
    """Against the formulas at the h' that the forward gave, with their bounds on every element."""
    require_gpu()
    c = Case(20, 264, stream=torch.float32, wt=torch.float32, scale=0.5, h_scale=1.0)
    h, y, post, pre = (t.clone().requires_grad_() for t in (c.h, c.y, c.post, c.pre))
    a, n = Norm.apply(h, y, post, pre)
    torch.autograd.backward((a, n), (c.dh, c.dn))
    c.h = a.detach()
    ref = c.backward()
    for name, t in (("d_h", h), ("d_y", y), ("d_post_w", post), ("d_pre_w", pre)):
        c.within(name, t.grad, *ref[name])

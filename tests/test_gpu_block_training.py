"""A block as it is trained, from the operators together: norm, router, products
grouped by expert, the gated norm behind them, and the gradient of all of it.

Every step's result is held against the formula in FP64 on what the step before gave,
with a bound on every element from the arithmetic (roundings carried on over the whole
block would bound nothing), and the formulas one after the other against autograd's
gradient of the block in FP64: the steps are right, and they are the right steps.

The bound: a value v that is off by up to d gives a product off by |a| db + |b| da +
da db, and so on, and every operation adds its own: half a step of FP32 (2^-24), S + 18
of them of the sum of the magnitudes for a sum of S terms, half a step of bfloat16
(2^-8) for a result in that.  The router's choices and weights are taken as they are
(they are constants of the block here)."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu

pytestmark = pytest.mark.gpu
U32, UBF = mp.U32, mp.UBF


class B:
    """FP64 values and how far what a kernel holds may be from them."""

    def __init__(self, v, d=None):
        self.v = v.double()
        self.d = torch.zeros_like(self.v) if d is None else d

    def __mul__(self, o):
        if not isinstance(o, B):
            return B(self.v * o, self.d * abs(o) + 2 * U32 * (self.v * o).abs())
        v = self.v * o.v
        d = self.v.abs() * o.d + (o.v.abs() + o.d) * self.d
        return B(v, d * (1 + U32) + U32 * v.abs())

    def __add__(self, o):
        v, d = self.v + o.v, self.d + o.d
        return B(v, d * (1 + U32) + U32 * v.abs())

    def __matmul__(self, o):
        mag = (self.v.abs() + self.d) @ (o.v.abs() + o.d)
        d = (self.v.abs() + self.d) @ o.d + self.d @ o.v.abs()
        return B(self.v @ o.v, d + (self.v.shape[1] + 18) * U32 * mag)

    def t(self):
        return B(self.v.T, self.d.T)

    def sum(self, dim, keepdim=False):
        n, mag = self.v.shape[dim], (self.v.abs() + self.d).sum(dim, keepdim=keepdim)
        return B(self.v.sum(dim, keepdim=keepdim), self.d.sum(dim, keepdim=keepdim) + (n + 18) * U32 * mag)

    def __getitem__(self, i):
        return B(self.v[i], self.d[i])

    def through(self, f, slope):
        """f, whose slope is at most `slope`, evaluated to 16 half steps of itself and of 1"""
        v = f(self.v)
        return B(v, slope * self.d + 16 * U32 * (1 + v.abs() + slope * self.d))

    def rms(self, eps):
        """1 / sqrt(mean of squares + eps), from the ends of the mean's range"""
        H = self.v.shape[1]
        ms = (self.v ** 2).mean(1, keepdim=True) + eps
        dm = (2 * self.v.abs() * self.d + self.d ** 2).mean(1, keepdim=True) + (H + 18) * U32 * ms
        r = ms ** -0.5
        assert bool((dm < ms).all())
        return B(r, (ms - dm) ** -0.5 - r + 8 * U32 * r)

    def check(self, name, got):
        assert got.shape == self.v.shape, name
        b = self.d + U32 * self.v.abs()
        if got.dtype is torch.bfloat16:
            b = self.d + UBF * (self.v.abs() + self.d)
        err = (got.double() - self.v).abs()
        assert bool((err <= b).all()), f"{name}: {(err / b.clamp_min(1e-300)).max().item():.3g} of the bound"
        # (a bound so wide that zeros would pass finds nothing)
        assert bool((self.v.norm() > 4 * b.norm())), f"{name}: the bound is {(b.norm() / self.v.norm()).item():.3g} of the values"


def silu_grad(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


SILU = torch.nn.functional.silu
EPS, SCALE, H_SCALE = 1e-5, 0.5, 0.75


def plain(h, pre0, w13, w2, post, gate, pre1, ids, wt):
    """The block in FP64, differentiable: (h', n')."""
    rms = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    n = rms(h) * pre0
    y = torch.zeros_like(n)
    for j in range(ids.shape[1]):
        for e in ids[:, j].unique().tolist():
            t = (ids[:, j] == e).nonzero()[:, 0]
            g, u = (n[t] @ w13[e].T).chunk(2, 1)
            y = y.index_add(0, t, wt[t, j:j + 1] * ((SILU(g) * u) @ w2[e].T))
    h1 = H_SCALE * h + SCALE * torch.sigmoid(gate) * rms(y) * post
    return h1, rms(h1) * pre1


class Block:
    def __init__(self, T, H, I, E, k, stream, seed=0, idle=()):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 1009 + 31 * T + H)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.h = r(T, H).to(stream)
        self.pre0, self.pre1, self.post = (1 + 0.2 * r(H) for _ in range(3))
        self.gate = r(H)
        self.gate_w = (r(E, H) / H ** 0.5).bfloat16()
        self.bias = torch.zeros(E, device="cuda")
        self.bias[list(idle)] = float("-inf")  # (experts without rows)
        self.w13, self.w2 = (r(E, 2 * I, H) / H ** 0.5).bfloat16(), (r(E, H, I) / I ** 0.5).bfloat16()
        self.dh, self.dn = r(T, H).to(stream), r(T, H).bfloat16()

    def tail(self):
        return dict(post_w=self.post, gate=self.gate, gate_act="sigmoid", scale=SCALE, h_scale=H_SCALE, pre_w=self.pre1, eps=EPS)

    def route(self, n):
        ids, wt = moe.gate(n, self.gate_w, self.k, bias=self.bias, renormalize=True)
        p = moe.make_problem(self.T, self.E, self.k, 256, 256, 16)
        _, off, sa, so = moe.route(p, ids)
        return ids, wt, off, sa.long(), so.long()

    def run(self):
        """Forward and backward by the operators."""
        k, T, H = self.k, self.T, self.H
        r = {}
        _, r["n"] = moe.block_norm(self.h, pre_w=self.pre0, eps=EPS)
        ids, wt, off, sa, so = self.route(r["n"])
        w = wt.view(-1)[sa][:, None]
        x = r["n"][sa // k]
        r["a"] = moe.grouped(x, self.w13, off)
        g, u = r["a"].float().chunk(2, 1)
        r["act"] = (SILU(g) * u).bfloat16()
        r["o"] = moe.grouped(r["act"], self.w2, off)
        r["y"] = (w * r["o"].float())[so].view(T, k, H).sum(1).bfloat16()
        r["h1"], r["n1"] = moe.block_norm(self.h, r["y"], **self.tail())
        back = moe.block_norm_grad(self.dh, self.dn, r["h1"], r["y"], **self.tail())
        r["dh1"], r["dy"], r["d_post"], r["d_gate"], r["d_pre1"] = back
        r["do"] = (w * r["dy"].float()[sa // k]).bfloat16()
        r["d_act"] = moe.grouped_dx(r["do"], self.w2, off)
        r["d_w2"] = moe.grouped_dw(r["do"], r["act"], off, out_dtype=torch.float32)
        d = r["d_act"].float()
        r["da"] = torch.cat([d * u * silu_grad(g), d * SILU(g)], 1).bfloat16()
        r["dx"] = moe.grouped_dx(r["da"], self.w13, off)
        r["d_w13"] = moe.grouped_dw(r["da"], x, off, out_dtype=torch.float32)
        r["dn"] = r["dx"].float()[so].view(T, k, H).sum(1).bfloat16()
        # (the first norm passes h itself on: its gradient is what the second one's is)
        r["dh"], _, _, _, r["d_pre0"] = moe.block_norm_grad(r["dh1"], r["dn"], self.h, pre_w=self.pre0, eps=EPS)
        return r, (ids, wt, off, sa, so)

    def steps(self, routed, given=None):
        """run()'s results by the formulas, each from the ones before it: given's, or these themselves."""
        ids, wt, off, sa, so = routed
        k, T, H, I = self.k, self.T, self.H, self.I
        per = lambda f: [f(e, slice(a, b)) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))]
        cat = lambda bs, dim=0: B(torch.cat([b.v for b in bs], dim), torch.cat([b.d for b in bs], dim))
        stack = lambda bs: B(torch.stack([b.v for b in bs]), torch.stack([b.d for b in bs]))
        out = {}

        def is_(name, b):
            out[name] = b
            return B(b.v if given is None else given[name])

        def spread(b):  # rows by expert -> sums over a token's
            return B(b.v[so].view(T, k, H), b.d[so].view(T, k, H)).sum(1)

        def rms_grad(D, u, v, r):  # D + r (u - v r mean(u v r))
            vr = v * r
            m = (u * vr).sum(1, keepdim=True) * (1 / H)
            return D + r * (u + vr * m * -1.0)

        h, pre0, pre1, post, gate = B(self.h), B(self.pre0), B(self.pre1), B(self.post), B(self.gate)
        w13, w2, w = B(self.w13), B(self.w2), B(wt.view(-1)[sa][:, None])
        r0 = h.rms(EPS)
        x = is_("n", h * r0 * pre0)[sa // k]
        a = is_("a", cat(per(lambda e, i: x[i] @ w13[e].t())))
        g, u = a[:, :I], a[:, I:]
        s, sg = g.through(SILU, 1.1), g.through(silu_grad, 0.5)
        act = is_("act", s * u)
        o = is_("o", cat(per(lambda e, i: act[i] @ w2[e].t())))
        y = is_("y", spread(w * o))
        ry, sig = y.rms(EPS), gate.through(torch.sigmoid, 0.25)
        yy = y * ry
        pw = yy * post
        h1 = h * H_SCALE + sig * pw * SCALE
        is_("n1", h1 * h1.rms(EPS) * pre1)  # (of h' before its rounding)
        h1 = is_("h1", h1)
        r1, dn = h1.rms(EPS), B(self.dn)
        is_("d_pre1", (dn * h1 * r1).sum(0))
        D = rms_grad(B(self.dh), dn * pre1, h1, r1)
        dh = is_("dh1", D * H_SCALE)
        # (1 - sigmoid is off by a step of 1)
        is_("d_gate", (D * B(sig.v * (1 - sig.v), 16 * U32 * sig.v) * pw * SCALE).sum(0))
        dpw = D * sig * SCALE
        is_("d_post", (dpw * yy).sum(0))
        dyy = dpw * post
        m = (dyy * yy).sum(1, keepdim=True) * (1 / H)
        dy = is_("dy", ry * (dyy + yy * m * -1.0))
        do = is_("do", w * dy[sa // k])
        d_act = is_("d_act", cat(per(lambda e, i: do[i] @ w2[e])))
        is_("d_w2", stack(per(lambda e, i: do[i].t() @ act[i])))
        da = is_("da", cat([d_act * u * sg, d_act * s], 1))
        dx = is_("dx", cat(per(lambda e, i: da[i] @ w13[e])))
        is_("d_w13", stack(per(lambda e, i: da[i].t() @ x[i])))
        dn = is_("dn", spread(dx))
        is_("d_pre0", (dn * h * r0).sum(0))
        is_("dh", rms_grad(dh, dn * pre0, h, r0))
        return out

    def gradients(self, routed):
        """Autograd's, in FP64."""
        ids, wt = routed[0], routed[1].double()
        leaves = [t.double().requires_grad_() for t in (self.h, self.pre0, self.w13, self.w2, self.post, self.gate, self.pre1)]
        h1, n1 = plain(*leaves, ids.long(), wt)
        ((h1 * self.dh.double()).sum() + (n1 * self.dn.double()).sum()).backward()
        names = ("dh", "d_pre0", "d_w13", "d_w2", "d_post", "d_gate", "d_pre1")
        return dict(zip(names, (t.grad for t in leaves)), h1=h1.detach(), n1=n1.detach())


CASES = [(1, 64, 32, 4, 2, torch.float32, ()), (5, 72, 24, 3, 1, torch.bfloat16, (1,)), (40, 64, 40, 5, 2, torch.float32, (0, 4)),
         (200, 136, 64, 4, 2, torch.bfloat16, (2,)), (700, 64, 32, 8, 4, torch.float32, ())]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d-H%d-I%d-E%d-k%d" % c[:5])
def test_a_block_and_its_gradient(case):
    require_gpu()
    b = Block(*case[:6], idle=case[6])
    got, routed = b.run()
    torch.cuda.synchronize()
    assert int(routed[2][-1]) == b.T * b.k and bool((routed[0] >= 0).all())
    for name, r in b.steps(routed, got).items():
        r.check(name, got[name])
    whole = b.steps(routed)
    for name, g in b.gradients(routed).items():
        assert bool(((whole[name].v - g).abs() <= 1e-9 * g.abs().max()).all()), name
    for e in case[6]:
        assert bool((got["d_w13"][e] == 0).all()) and bool((got["d_w2"][e] == 0).all())


def test_accumulated_over_two_batches():
    """Weight gradients added up in one buffer: the second batch's on top of the first's."""
    require_gpu()
    H, N = 64, 48
    w = torch.zeros((3, N, H), device="cuda")
    want = torch.zeros_like(w)
    for rows in ([4, 0, 30], [0, 9, 70]):
        off = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
        dy, x = torch.randn((sum(rows), N), device="cuda").bfloat16(), torch.randn((sum(rows), H), device="cuda").bfloat16()
        moe.grouped_dw(dy, x, off, out=w, accumulate=True)
        want += moe.grouped_dw(dy, x, off, out_dtype=torch.float32)
    assert torch.equal(w, want)


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("T", [1, 6, 150])
def test_fp4_experts_in_steps_and_at_once(T, gran):
    """A layer with FP4 experts from its single products, and forward(), which fuses them, from the same rows."""
    require_gpu()
    H, I, E, k = 256, 256, 6, 2
    rng = np.random.default_rng(T + gran)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda().bfloat16()
    (w13, s13), (w2, s2) = mp.fp4_tensor(rng, E, 2 * I, H, gran), mp.fp4_tensor(rng, E, H, I, gran)
    g13, g2 = (rng.uniform(0.5, 2, E).astype(np.float32) for _ in range(2))
    W13 = B(torch.from_numpy(np.stack([mp.weight(w13[e], s13[e], g13[e], gran) for e in range(E)])).cuda())
    W2 = B(torch.from_numpy(np.stack([mp.weight(w2[e], s2[e], g2[e], gran) for e in range(E)])).cuda())
    w13, s13, g13, w2, s2, g2 = (torch.from_numpy(t).cuda() for t in (w13, s13, g13, w2, s2, g2))
    ids, wt = moe.gate(x, torch.randn((E, H), device="cuda").bfloat16(), k, renormalize=True)
    _, off, sa, so = moe.route(moe.make_problem(T, E, k, H, I, gran), ids)
    sa, so = sa.long(), so.long()
    a = moe.grouped(x[sa // k], w13, off, w_sf=s13, w_gs=g13, gran_k=gran, out_dtype=torch.float32)
    g, u = a.chunk(2, 1)
    act = (SILU(g) * u).bfloat16()
    o = moe.grouped(act, w2, off, w_sf=s2, w_gs=g2, gran_k=gran, out_dtype=torch.float32)
    w = wt.view(-1)[sa][:, None]
    y = (w * o)[so].view(T, k, H).sum(1)
    fused = moe.forward(x, ids, wt, w13, s13, g13, w2, s2, g2, gran, out_dtype=torch.float32)
    rows = lambda f: [f(e, slice(p, q)) for e, (p, q) in enumerate(zip(off.tolist(), off.tolist()[1:]))]
    cat = lambda bs: B(torch.cat([b.v for b in bs]), torch.cat([b.d for b in bs]))
    xs = B(x)[sa // k]
    ref = cat(rows(lambda e, i: xs[i] @ W13[e].t())) * 1.0
    act = ref[:, :I].through(SILU, 1.1) * ref[:, I:]
    act = B(act.v, act.d + UBF * (act.v.abs() + act.d))
    ref = B(w) * (cat(rows(lambda e, i: act[i] @ W2[e].t())) * 1.0)
    ref = B(ref.v[so].view(T, k, H), ref.d[so].view(T, k, H)).sum(1)
    ref.check("in steps", y)
    # (its rounding between the products is at most bfloat16's, too)
    ref.check("fused", fused)

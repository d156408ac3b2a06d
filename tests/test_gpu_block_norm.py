"""Norms around a layer with gate and residual scale (moe_fp4_block_norm) and
their gradient against the formulas in FP64, with bounds on every element from
the arithmetic.

A sum of H FP32 terms is off by at most H half steps (2^-24) of the sum of their
magnitudes, in whatever order; 1 / sqrt of a mean of squares therefore by H / 2 + 4
half steps, a product or a sigmoid by a few (8 taken); what follows is propagated
to first order, and a rounding to bfloat16 is half of its steps, 2^-8 of the
value."""

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu

pytestmark = pytest.mark.gpu
U32, UBF = mp.U32, mp.UBF
TINY = 2.0 ** -133  # below bfloat16's and FP32's normal range: absolute


class Case:
    def __init__(self, T, H, post=True, gate="none", act=None, stream=torch.bfloat16, wt=torch.bfloat16, gt=torch.bfloat16, pre=True,
                 y=True, scale=0.75, h_scale=1.25, eps=1e-6, seed=0, size=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 1000003 + T * 131 + H)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.T, self.H, self.eps, self.act, self.kind = T, H, eps, act, gate
        self.scale, self.h_scale = scale, h_scale
        self.h = (3 * size * r(T, H)).to(stream)
        self.y = (0.5 * size * r(T, H)).bfloat16() if y else None
        self.post = (1 + 0.2 * r(H)).to(wt) if post and y else None
        self.pre = (1 + 0.2 * r(H)).to(wt) if pre else None
        shape = {"none": None, "channel": (H,), "token": (T,), "token1": (T, 1), "full": (T, H)}[gate]
        self.gate = None if shape is None or not y else (1.5 * r(*shape)).to(gt)
        self.dh, self.dn = (0.1 * r(T, H)).to(stream), (0.1 * r(T, H)).bfloat16() if pre else None

    def args(self):
        return dict(post_w=self.post, gate=self.gate, gate_act=self.act, scale=self.scale, h_scale=self.h_scale, pre_w=self.pre, eps=self.eps)

    def rms(self, v):
        return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + self.eps)

    def gate64(self):
        """(act(gate), its derivative), broadcast over [T, H]"""
        if self.gate is None:
            return torch.ones((1, 1), dtype=torch.float64, device="cuda"), torch.zeros((1, 1), dtype=torch.float64, device="cuda")
        g = self.gate.double()
        g = g.view(1, -1) if self.kind == "channel" else g.view(-1, 1) if self.kind in ("token", "token1") else g
        if self.act is None:
            return g, torch.ones_like(g)
        s = torch.sigmoid(g)
        return s, s * (1 - s)

    def forward(self):
        """(h', n) in FP64 and the bounds before a rounding to the output's type"""
        H, h = self.H, self.h.double()
        d = torch.zeros_like(h)
        if self.y is not None:
            a = self.y.double()
            if self.post is not None:
                a = a * self.rms(a) * self.post.double()
            b = self.scale * self.gate64()[0] * a
            d = U32 * ((H / 2 + 20) * b.abs() + 4 * (self.h_scale * h).abs())
            h = self.h_scale * h + b
        if self.pre is None:
            return h, None, d, None
        r, w = self.rms(h), self.pre.double()
        n = h * r * w
        dr = U32 * (H / 2 + 8) + (h.abs() * d).sum(1, keepdim=True) / (h * h).sum(1, keepdim=True).clamp_min(1e-300)
        return h, n, d, (r * w).abs() * d + n.abs() * (dr + 8 * U32)

    def check_forward(self, inplace=False):
        h = self.h.clone()
        kw = dict(h_out=h) if inplace else {}
        ho, n = moe.block_norm(h, self.y, **self.args(), **kw)
        torch.cuda.synchronize()
        rh, rn, dh, dn = self.forward()
        if self.y is None:
            assert ho is h
        else:
            self.within("h'", ho, rh, dh)
        assert inplace == (ho is h) or self.y is None
        if self.pre is None:
            assert n is None
        else:
            self.within("n", n, rn, dn)
        return ho, n

    @staticmethod
    def within(name, got, ref, bound):
        b = bound + TINY
        if got.dtype is torch.bfloat16:
            b = b * (1 + UBF) + UBF * ref.abs()
        else:
            b = b + U32 * ref.abs()
        err = (got.double() - ref).abs()
        assert bool((err <= b).all()), f"{name}: {(err / b).max().item():.3g} of the bound"

    def backward(self):
        """The formulas' gradients in FP64, with bounds: d_h, d_y, d_post_w, d_gate, d_pre_w (h here is h')."""
        T, H, c = self.T, self.H, (self.H + 32) * U32
        D = self.dh.double() if self.dh is not None else torch.zeros((T, H), dtype=torch.float64, device="cuda")
        mag = D.abs()
        out = {}
        if self.pre is not None:
            h, dn = self.h.double(), self.dn.double()
            r = self.rms(h)
            hh, u = h * r, dn * self.pre.double()
            D = D + r * (u - hh * (u * hh).mean(1, keepdim=True))
            mag = mag + r * (u.abs() + hh.abs() * (u * hh).abs().mean(1, keepdim=True))
            out["d_pre_w"] = (dn * hh).sum(0), (H / 2 + T + 24) * U32 * (dn * hh).abs().sum(0)
        dD = c * mag
        hs = self.h_scale if self.y is not None else 1.0
        out["d_h"] = hs * D, abs(hs) * dD + 2 * U32 * (hs * D).abs()
        if self.y is None:
            return out
        y, (act, slope) = self.y.double(), self.gate64()
        ry, w = (self.rms(y), self.post.double()) if self.post is not None else (torch.ones((T, 1), dtype=torch.float64, device="cuda"), 1.0)
        yy = y * ry
        a, s = yy * w, abs(self.scale)
        da, dda = self.scale * act * D, s * act.abs() * dD + c * (s * act * D).abs()
        if self.post is not None:
            out["d_post_w"] = (da * yy).sum(0), (dda * yy.abs()).sum(0) + (T + H) * U32 * (da * yy).abs().sum(0)
        if self.gate is not None:
            t = self.scale * slope * D * a
            # (1 - sigmoid is off by a step of 1: as much of the slope as 1 / (1 - sigmoid))
            dt = s * (slope * a).abs() * dD + c * t.abs() + 8 * U32 * (s * D * a * act).abs()
            dim = {"channel": 0, "token": 1, "token1": 1}.get(self.kind)
            if dim is not None:
                t, dt = t.sum(dim), dt.sum(dim) + (T + H + 8) * U32 * t.abs().sum(dim)
                if self.kind == "token1":
                    t, dt = t.view(-1, 1), dt.view(-1, 1)
            out["d_gate"] = t, dt
        v, dv = da * w, dda * (abs(w) if isinstance(w, float) else w.abs()) + 4 * U32 * (da * w).abs()
        if self.post is None:
            out["d_y"] = v, dv
        else:
            m, dm = (v * yy).mean(1, keepdim=True), (dv * yy.abs() + c * (v * yy).abs()).mean(1, keepdim=True)
            out["d_y"] = ry * (v - yy * m), ry * (dv + yy.abs() * dm + c * (v.abs() + (yy * m).abs()))
        return out

    def check_backward(self):
        got = moe.block_norm_grad(self.dh, self.dn, None if self.pre is None else self.h, self.y, **self.args())
        torch.cuda.synchronize()
        ref = self.backward()
        for name, o in zip(("d_h", "d_y", "d_post_w", "d_gate", "d_pre_w"), got):
            assert (o is None) == (name not in ref), name
            if o is not None:
                assert o.shape == ref[name][0].shape, name
                self.within(name, o, *ref[name])
        return got


SIZES = [(1, 8), (1, 6144), (3, 504), (5, 512), (2, 520), (4, 2048), (7, 2056), (6, 4104), (3, 8192), (2, 8200), (2, 16384)]
KINDS = [("none", None), ("channel", None), ("channel", "sigmoid"), ("token", "sigmoid"), ("token1", None), ("full", "sigmoid"), ("full", None)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-{k[1]}")
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "T%d-H%d" % s)
def test_block_norm(size, kind):
    require_gpu()
    f32, bf = torch.float32, torch.bfloat16
    for i, (stream, wt, gt) in enumerate(((bf, bf, bf), (f32, f32, f32), (f32, bf, bf), (bf, f32, bf))):
        c = Case(*size, gate=kind[0], act=kind[1], stream=stream, wt=wt, gt=gt, post=i != 2, seed=i)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("T,H", [(300, 6144), (1100, 520), (5000, 64), (600, 8200)])
def test_many_rows(T, H):
    """More rows than the gradient's workgroups."""
    require_gpu()
    for kind, act in (("channel", None), ("token", "sigmoid")):
        c = Case(T, H, gate=kind, act=act, stream=torch.float32)
        c.check_forward()
        c.check_backward()


def test_parts_that_are_not_there():
    require_gpu()
    for H in (64, 520, 8200):
        Case(5, H, y=False).check_forward()
        Case(5, H, y=False).check_backward()
        Case(5, H, pre=False, gate="channel").check_forward()
        Case(5, H, pre=False, gate="channel").check_backward()
        c = Case(5, H, gate="token")
        c.dh = None
        c.check_backward()
        c = Case(5, H, post=False)
        c.check_forward()
        c.check_backward()


def test_in_place():
    require_gpu()
    for H, stream in ((64, torch.float32), (2048, torch.bfloat16), (8200, torch.bfloat16)):
        c = Case(6, H, gate="channel", stream=stream)
        a, n = c.check_forward()
        b, m = c.check_forward(inplace=True)
        assert torch.equal(a, b) and torch.equal(n, m)
        want = moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args())
        d = c.dh.clone()
        got = moe.block_norm_grad(d, c.dn, c.h, c.y, **c.args(), d_h=d)
        assert got[0] is d and all(torch.equal(x, y) for x, y in zip(want, got))


def test_no_rows():
    require_gpu()
    c = Case(0, 64, gate="channel")
    h, n = moe.block_norm(c.h, c.y, **c.args())
    assert h.shape == (0, 64) and n.shape == (0, 64)
    _, _, post, gate, pre = moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args())
    assert all(bool((t == 0).all()) and t.shape == (64,) for t in (post, gate, pre))


def test_large_and_small_values():
    """Rows whose squares leave FP32's range, rows of zeros and single large elements."""
    require_gpu()
    for H in (512, 1024, 8200):
        for size in (1e30, 1e19, 1e-3):
            c = Case(4, H, gate="channel", stream=torch.float32, size=size)
            c.dh.zero_()
            c.check_forward()
            c.check_backward()
        c = Case(4, H, stream=torch.float32)
        c.h[1], c.y[1], c.h[2, 3], c.y[3, 5] = 0, 0, 2.0 ** 100, 2.0 ** 100
        c.check_forward()
        c.check_backward()


def test_special_values_stay_in_their_row():
    require_gpu()
    c = Case(6, 1032, gate="token", act="sigmoid")
    h0, n0 = moe.block_norm(c.h, c.y, **c.args())
    g0 = moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args())
    c.h[1, 5], c.y[3, 7] = float("nan"), float("inf")
    h1, n1 = moe.block_norm(c.h, c.y, **c.args())
    g1 = moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args())
    torch.cuda.synchronize()
    keep = [0, 2, 4, 5]
    for a, b in ((h0, h1), (n0, n1), (g0[0], g1[0]), (g0[1], g1[1])):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(n1[1]).all()) and bool(torch.isnan(n1[3]).any())


def test_sigmoid_over_the_whole_range():
    require_gpu()
    c = Case(8, 4096, post=False, gate="full", act="sigmoid", stream=torch.float32, gt=torch.float32, h_scale=0.0)
    c.gate.view(-1).copy_(torch.linspace(-110, 110, c.gate.numel(), device="cuda"))
    c.y.fill_(1)
    h, _ = moe.block_norm(c.h, c.y, **c.args())
    ref = 0.75 * torch.sigmoid(c.gate.double())
    # (below 2^-125, the end of the normal range, it is not resolved)
    assert bool(((h.double() - ref).abs() <= 12 * U32 * ref + 2.0 ** -125).all())
    c.gate[0, 0], c.gate[0, 1], c.gate[0, 2] = float("inf"), float("-inf"), float("nan")
    h, _ = moe.block_norm(c.h, c.y, **c.args())
    assert h[0, 0] == 0.75 and h[0, 1].abs() < 2.0 ** -124 and bool(torch.isnan(h[0, 2]))


def test_gradient_against_differences():
    """Central differences of the formula (FP64) along random directions: their error is the third derivative's, of the
    step's square; the kernel's own error is bounded as above (here by 1e-3 of the sum of magnitudes, far above both: what
    this finds is a wrong formula)."""
    require_gpu()
    for kind, act in KINDS:
        c = Case(3, 264, gate=kind, act=act, stream=torch.float32, wt=torch.float32, gt=torch.float32)
        rh = c.forward()[0]
        args = c.args()
        d_h, d_y, d_post, d_gate, d_pre = moe.block_norm_grad(c.dh, c.dn, rh.float(), c.y, **args)
        grads = dict(h=d_h, y=d_y, post=d_post, gate=d_gate, pre=d_pre)

        def loss():
            h, n, _, _ = c.forward()
            return ((h * c.dh.double()).sum() + (n * c.dn.double()).sum()).item()

        for name, g in grads.items():
            t = getattr(c, name)
            if t is None:
                continue
            base = t.double()
            v = torch.randn(base.shape, dtype=torch.float64, device="cuda")
            step = 1e-4
            vals = []
            for sgn in (1, -1):
                setattr(c, name, base + sgn * step * v)
                vals.append(loss())
            setattr(c, name, t)
            num = (vals[0] - vals[1]) / (2 * step)
            want = (g.double() * v.view(g.shape)).sum().item()
            mag = (g.double() * v.view(g.shape)).abs().sum().item()
            # d_y is bfloat16: half a step of each element
            assert abs(num - want) <= (1e-3 + (UBF if name == "y" else 0)) * mag, (kind, act, name, num, want, mag)


def test_python_refusals():
    require_gpu()
    c = Case(4, 64, gate="channel")
    a = c.args()
    for kw in (dict(gate=c.gate[:32].contiguous()), dict(gate_act="tanh"), dict(post_w=c.post[:32].contiguous()), dict(h_out=c.h[:2])):
        with pytest.raises(ValueError):
            moe.block_norm(c.h, c.y, **dict(a, **kw))
    for args, kw in (((c.h,), {}), ((c.h,), dict(pre_w=c.pre, post_w=c.post)), ((c.h,), dict(pre_w=c.pre, h_out=c.h)),
                     ((c.h, c.y), dict(n=c.h)), ((c.h, c.y[:2]), dict(pre_w=c.pre))):
        with pytest.raises(ValueError):
            moe.block_norm(*args, **kw)
    for kw in (dict(pre_w=c.pre.half()), dict(gate=c.gate.half())):
        with pytest.raises(TypeError):
            moe.block_norm(c.h, c.y, **dict(a, **kw))
    with pytest.raises(TypeError):
        moe.block_norm(c.h, c.y.float(), **a)
    with pytest.raises(moe.MoeFp4Error):
        moe.block_norm(c.h, c.y, **a, n=c.y)
    with pytest.raises(moe.MoeFp4Error):
        moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **a, workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))


def test_workspace_guard_and_smaller_batches():
    require_gpu()
    H = 1032
    need = moe._norm_grad_need(300, H)
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    at = (-buf.data_ptr()) % 256
    ws = buf[at:at + need]
    for T in (300, 7, 1):
        c = Case(T, H, gate="channel")
        want = moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args())
        got = moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args(), workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert bool((buf[:at] == 0x5A).all()) and bool((buf[at + need:] == 0x5A).all())


def test_streams_and_graphs():
    require_gpu()
    c = Case(40, 2056, gate="channel", act="sigmoid")
    f = lambda **k: (*moe.block_norm(c.h, c.y, **c.args(), **k), *moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args(), **k))
    want = f()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = f(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # two graphs with a workspace each, replayed in turn with eager calls between
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    for i in range(4):
        c.h.copy_(torch.randn_like(c.h.float()).bfloat16())
        c.dn.copy_(torch.randn_like(c.dn.float()).bfloat16())
        for g, out in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, f()))


def test_more_rows_than_a_grid_is_wide():
    """T beyond 2^20 workgroups (or 2^22 waves)."""
    require_gpu()
    for T, H in (((1 << 20) + 5, 520), ((1 << 22) + 9, 8)):
        c = Case(8, H, pre=True, y=False)
        h = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        h[:4], h[-4:] = c.h[:4], c.h[4:]
        _, n = moe.block_norm(h, pre_w=c.pre)
        want = moe.block_norm(c.h, pre_w=c.pre)[1]
        assert torch.equal(n[:4], want[:4]) and torch.equal(n[-4:], want[4:]) and not bool(n[4:-4].any())


def test_ends_of_eps():
    """Rows so small that eps counts, down to the least one, and the largest one beside ordinary and large rows."""
    require_gpu()
    for H in (64, 1024, 8200):
        for eps, sizes in ((1.1e-20, (1e-9, 1e-10, 1e-12)), (1.0, (1.0, 1e-3, 1e19))):
            for size in sizes:
                c = Case(4, H, gate="channel", stream=torch.float32, size=size, eps=eps)
                c.dh.zero_()
                c.check_forward()
                c.check_backward()


def test_operators_refuse_a_stream_of_another_device():
    require_gpu()
    from test_operator_streams import OnDevice
    c = Case(4, 64, gate="channel")
    w, off = torch.ones((1, 64, 64), device="cuda").bfloat16(), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for call in (lambda s: moe.block_norm(c.h, c.y, **c.args(), stream=s), lambda s: moe.block_norm_grad(c.dh, c.dn, c.h, c.y, **c.args(), stream=s),
                 lambda s: moe.grouped(c.y, w, off, stream=s), lambda s: moe.grouped_dx(c.y, w, off, stream=s),
                 lambda s: moe.grouped_dw(c.y, c.y, off, stream=s)):
        call(torch.cuda.Stream())
        torch.cuda.synchronize()
        with pytest.raises(ValueError, match="stream"):
            call(OnDevice(1))


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("H", [8, 1032, 3080, 5000, 7000, 8192, 8200])
def test_the_norm_before_the_first_layer(H, stream):
    require_gpu()
    c = Case(5, H, y=False, stream=stream)
    c.check_forward()
    c.check_backward()

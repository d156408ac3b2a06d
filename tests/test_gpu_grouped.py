"""Products grouped by expert (moe_fp4_grouped, _dx, _dw) against a plain FP64
implementation, with a bound on every element from the arithmetic.

The factors are bfloat16 (or FP4 codes times E4M3 or UE8M0 scales, which
bfloat16 holds exactly), so every product is exact in FP32 and a float32 output
of a sum of S products is off by at most (S + 16) half steps of FP32 (2^-24)
times the sum of the products' magnitudes, in whatever order they are added; the
global scale is one more factor (2 half steps).  A bfloat16 output is the
float32 one rounded to nearest, bit for bit."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu

pytestmark = pytest.mark.gpu
# half a step of FP32, 2^-24, and of bfloat16: its values in [1, 2) lie 2^-7 apart (8 significant bits), so that a
# rounding is off by up to 2^-8 of the value
U32, UBF = mp.U32, mp.UBF


def offsets_of(rows, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(rows)]), dtype=torch.int32, device="cuda")


def spread(rng, M, E):
    """M rows over E experts, some without any."""
    p = np.exp(rng.standard_normal(E))
    p[rng.random(E) < 0.2] = 0
    if p.sum() == 0:
        p[:] = 1
    return rng.multinomial(M, p / p.sum())


class Case:
    def __init__(self, rows, N, K, gran=0, seed=0, first=0, behind=0, gs=True):
        rng = np.random.default_rng([seed, N, K, gran, len(rows)])
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 17 * N + K)
        self.rows, self.N, self.K, self.gran, self.E = list(rows), N, K, gran, len(rows)
        self.off = offsets_of(rows, first)
        self.M = first + int(sum(rows)) + behind
        r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
        self.x, self.dy = r(self.M, K), r(self.M, N)
        self.w_sf = self.w_gs = None
        if gran:
            w, sf = mp.fp4_tensor(rng, self.E, N, K, gran)
            self.w, self.w_sf = torch.from_numpy(w).cuda(), torch.from_numpy(sf).cuda()
            if gs:
                self.w_gs = torch.from_numpy(rng.uniform(0.5, 2, self.E).astype(np.float32)).cuda()
            self.W = torch.from_numpy(np.stack([mp.weight(w[e], sf[e], None if self.w_gs is None else self.w_gs[e].item(), gran)
                                                for e in range(self.E)])).cuda()
        else:
            self.w = r(self.E, N, K)
            self.W = self.w.double()

    def kw(self):
        return dict(w_sf=self.w_sf, w_gs=self.w_gs, gran_k=self.gran or None)

    def ranges(self):
        o = self.off.tolist()
        return [(e, o[e], o[e + 1]) for e in range(self.E)]

    def check_rows(self, form, out, ref_of, terms):
        """out [M, C] float32 of rows guarded in front and behind; ref_of(e, rows) -> (reference, sum of magnitudes)."""
        worst = 0.0
        done = torch.zeros(self.M, dtype=torch.bool, device="cuda")
        for e, a, b in self.ranges():
            if a == b:
                continue
            ref, mag = ref_of(e, slice(a, b))
            bound = (terms + 18) * U32 * mag
            err = (out[a:b].double() - ref).abs()
            assert bool((err <= bound).all()), f"{form} expert {e}: {(err / bound.clamp_min(1e-300)).max().item():.3g} of the bound"
            worst = max(worst, (err / bound.clamp_min(1e-300)).max().item())
            done[a:b] = True
        assert bool((out[~done] == -77).all()), "a row outside the groups was written"
        print(f"[{form}] M={self.M} E={self.E} N={self.N} K={self.K} g{self.gran}: {worst:.2e} of the bound", flush=True)

    def product(self):
        buf = torch.full((self.M + 2, self.N), -77.0, device="cuda")
        out = moe.grouped(self.x, self.w, self.off, **self.kw(), out=buf[1:self.M + 1])
        b16 = moe.grouped(self.x, self.w, self.off, **self.kw(), out=torch.full((self.M, self.N), -77.0, device="cuda").bfloat16())
        torch.cuda.synchronize()
        self.check_rows("grouped", out, lambda e, s: (self.x[s].double() @ self.W[e].T, self.x[s].double().abs() @ self.W[e].abs().T),
                        self.K)
        assert bool((buf[0] == -77).all()) and bool((buf[-1] == -77).all())
        assert torch.equal(out.bfloat16().view(torch.int16), b16.view(torch.int16))
        return out

    def dx(self):
        buf = torch.full((self.M + 2, self.K), -77.0, device="cuda")
        out = moe.grouped_dx(self.dy, self.w, self.off, **self.kw(), out=buf[1:self.M + 1])
        b16 = moe.grouped_dx(self.dy, self.w, self.off, **self.kw(), out=torch.full((self.M, self.K), -77.0, device="cuda").bfloat16())
        torch.cuda.synchronize()
        self.check_rows("grouped_dx", out, lambda e, s: (self.dy[s].double() @ self.W[e], self.dy[s].double().abs() @ self.W[e].abs()),
                        self.N)
        assert bool((buf[0] == -77).all()) and bool((buf[-1] == -77).all())
        assert torch.equal(out.bfloat16().view(torch.int16), b16.view(torch.int16))
        return out

    def dw(self):
        buf = torch.full((self.E + 2, self.N, self.K), -77.0, device="cuda")
        out = moe.grouped_dw(self.dy, self.x, self.off, out=buf[1:self.E + 1])
        b16 = moe.grouped_dw(self.dy, self.x, self.off)
        torch.cuda.synchronize()
        worst = 0.0
        for e, a, b in self.ranges():
            ref = self.dy[a:b].double().T @ self.x[a:b].double()
            bound = (b - a + 16) * U32 * (self.dy[a:b].double().abs().T @ self.x[a:b].double().abs())
            err = (out[e].double() - ref).abs()
            assert bool((err <= bound).all()), f"grouped_dw expert {e} of {b - a} rows"
            if a < b:
                worst = max(worst, (err / bound).max().item())
        assert bool((buf[0] == -77).all()) and bool((buf[-1] == -77).all())
        assert torch.equal(out.bfloat16().view(torch.int16), b16.view(torch.int16))
        print(f"[grouped_dw] M={self.M} E={self.E} N={self.N} K={self.K}: {worst:.2e} of the bound", flush=True)
        return out


# (rows, experts or the rows of each, N, K): one row; few rows per expert; tiles of 64, 128 and 256; sums that are no
# multiple of a stage; sizes of a low-rank factor; more rows than a tile holds in one expert
SHAPES = [([1], 8, 32), ([1], 4096, 2080), ([3, 0, 2], 24, 96), ((8, 64), 520, 288), ((40, 60), 72, 1056), ((90, 9), 264, 160),
          ([17, 0, 1, 33], 136, 320), ([0, 300, 0], 1000, 704), ((700, 3), 1096, 224), ([63, 64, 65, 1], 256, 128),
          ([127, 128, 129, 0], 384, 64), ([255, 256, 257], 648, 96), ((1500, 12), 2056, 512), ([2100, 2000], 4104, 96),
          ((4000, 64), 32, 512), ((4000, 64), 512, 32), ([1000], 16, 2048), ([60], 2048, 4096),
          # short sums, many tiles per workgroup
          ((4000, 64), 72, 2080), ((4000, 64), 2056, 96), ((2000, 130), 1096, 128),
          # sums in parts: few tiles, long sums; fewer stages than parts in one expert
          ([5000], 64, 256), ([1300, 0, 20], 1320, 1184), ([33], 1096, 2080)]


def rows_of(shape, seed=0):
    return shape[0] if isinstance(shape[0], list) else spread(np.random.default_rng(seed + shape[1]), shape[0][0], shape[0][1])


@pytest.mark.parametrize("gran", [0, 16, 32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_rows(shape, gran):
    require_gpu()
    c = Case(rows_of(shape), shape[1], shape[2], gran, gs=gran == 16, first=3, behind=5)
    c.product()
    c.dx()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dw(shape):
    require_gpu()
    Case(rows_of(shape), shape[1], shape[2] + 8, first=3, behind=5).dw()


@pytest.mark.parametrize("gran", [0, 32])
@pytest.mark.parametrize("rows", [[2] * 40, [7, 9, 12, 3], [30, 40, 20, 0, 35], [130] * 6, [300, 20, 257]], ids=str)
def test_gradients_are_the_products_adjoints(rows, gran):
    """<dy, W x> = <dx, x> = <dW, W>, each side from its own kernel: the change of the output along any change of x or W
    (the product is linear in both, so that differences are exact)."""
    require_gpu()
    c = Case(rows, 264, 544, gran, seed=3)
    y = moe.grouped(c.x, c.w, c.off, **c.kw(), out_dtype=torch.float32).double()
    dx = moe.grouped_dx(c.dy, c.w, c.off, **c.kw(), out_dtype=torch.float32).double()
    dw = moe.grouped_dw(c.dy, c.x, c.off, out_dtype=torch.float32).double()
    a, b, d = (y * c.dy.double()).sum().item(), (dx * c.x.double()).sum().item(), (dw * c.W).sum().item()
    # each element's bound as above, times what it is multiplied with
    mag = sum((c.dy[s:t].double().abs() * (c.x[s:t].double().abs() @ c.W[e].abs().T)).sum().item() for e, s, t in c.ranges())
    bound = 2 * (max(544, 300) + 18) * U32 * mag
    assert abs(a - b) <= bound and abs(a - d) <= bound, (a, b, d, bound)


def test_values_outside_a_group_stay_outside():
    """NaN and infinities in other experts' rows, weights and in rows of no expert reach no output of a clean expert."""
    require_gpu()
    for rows, N, K, gran in (([5, 3, 70], 40, 72, 0), ([100, 30, 130], 264, 200, 0), ([300, 257, 65], 520, 136, 0), ([9, 3, 14], 48, 96, 16),
                             ([300, 257, 65], 520, 160, 32), ([700, 2, 900], 2056, 1032, 0)):
        c = Case(rows, N, K, gran, first=2, behind=3)
        ref = [f(out_dtype=torch.float32) for f in (lambda **k: moe.grouped(c.x, c.w, c.off, **c.kw(), **k),
                                                    lambda **k: moe.grouped_dx(c.dy, c.w, c.off, **c.kw(), **k),
                                                    lambda **k: moe.grouped_dw(c.dy, c.x, c.off, **k))]
        (_, a0, b0), (_, a1, b1), (_, a2, b2) = c.ranges()
        x, dy = c.x.clone(), c.dy.clone()
        for t in (x, dy):
            t[:a0] = float("nan")
            t[a1:b1] = float("inf")
            t[b2:] = float("nan")
        w, sf = c.w.clone(), c.w_sf
        if gran:
            sf = c.w_sf.clone()
            sf[1] = 0x7F if gran == 16 else 0xFF  # NaN scales
        else:
            w[1] = float("nan")
        kw = dict(c.kw(), w_sf=sf, out_dtype=torch.float32)
        y, dx, dw = moe.grouped(x, w, c.off, **kw), moe.grouped_dx(dy, w, c.off, **kw), moe.grouped_dw(dy, x, c.off, out_dtype=torch.float32)
        torch.cuda.synchronize()
        for a, b in ((a0, b0), (a2, b2)):
            assert torch.equal(y[a:b], ref[0][a:b]) and torch.equal(dx[a:b], ref[1][a:b])
        assert torch.equal(dw[0], ref[2][0]) and torch.equal(dw[2], ref[2][2])
        assert not bool(torch.isfinite(y[a1:b1]).all())


def test_special_values_in_a_group():
    """An infinity or NaN of x or dy shows where the formula has it, and nowhere else."""
    require_gpu()
    for rows, N, K in (([6], 40, 200), ([150, 20], 264, 136), ([600], 2056, 1032)):
        c = Case(rows, N, K)
        c.w.abs_()
        c.x[2, 5], c.x[4, 7] = float("inf"), float("nan")
        y = moe.grouped(c.x, c.w, c.off, out_dtype=torch.float32)
        dw = moe.grouped_dw(c.dy.abs(), c.x, c.off, out_dtype=torch.float32)
        torch.cuda.synchronize()
        bad = torch.zeros(c.M, dtype=torch.bool, device="cuda")
        bad[[2, 4]] = True
        assert bool((y[2] == float("inf")).all()) and bool(torch.isnan(y[4]).all()) and bool(torch.isfinite(y[~bad]).all())
        assert bool((dw[0, :, 5] == float("inf")).all()) and bool(torch.isnan(dw[0, :, 7]).all())
        dw[0, :, [5, 7]] = 0
        assert bool(torch.isfinite(dw).all())


def test_dw_accumulates():
    require_gpu()
    for rows, N, K in (([5, 0, 70], 40, 72), ([300, 0, 65], 520, 136), ([2000, 0], 2056, 2056), ([4000, 0, 9000], 72, 136)):
        c = Case(rows, N, K)
        ref = moe.grouped_dw(c.dy, c.x, c.off, out_dtype=torch.float32)
        old = torch.randn((c.E, N, K), device="cuda")
        out = old.clone()
        assert moe.grouped_dw(c.dy, c.x, c.off, out=out, accumulate=True) is out
        o16 = old.bfloat16()
        p16 = o16.clone()
        moe.grouped_dw(c.dy, c.x, c.off, out=p16, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(out, old + ref)  # one FP32 addition
        assert torch.equal(p16, (o16.float() + ref).bfloat16())
        assert torch.equal(out[1], old[1]) and torch.equal(p16[1], o16[1])


def test_no_rows():
    require_gpu()
    w = torch.randn((3, 16, 64), device="cuda").bfloat16()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty((0, 64), device="cuda").bfloat16(), torch.empty((0, 16), device="cuda").bfloat16()
    assert moe.grouped(x, w, off).shape == (0, 16) and moe.grouped_dx(dy, w, off).shape == (0, 64)
    assert bool((moe.grouped_dw(dy, x, off) == 0).all())
    keep = torch.ones((3, 16, 64), device="cuda")
    assert bool((moe.grouped_dw(dy, x, off, out=keep, accumulate=True) == 1).all())
    # rows, but none of an expert's
    x, dy = torch.ones((5, 64), device="cuda").bfloat16(), torch.ones((5, 16), device="cuda").bfloat16()
    out = torch.full((5, 16), 7.0, device="cuda")
    moe.grouped(x, w, off, out=out)
    assert bool((out == 7).all()) and bool((moe.grouped_dw(dy, x, off) == 0).all())


def test_offsets_beyond_the_rows_are_taken_within():
    require_gpu()
    c = Case([4, 6, 10], 72, 136)
    off = torch.tensor([-3, 4, 10, 1 << 30], dtype=torch.int32, device="cuda")
    f32 = dict(out_dtype=torch.float32)
    for a, b in ((moe.grouped(c.x, c.w, off, **f32), moe.grouped(c.x, c.w, c.off, **f32)),
                 (moe.grouped_dx(c.dy, c.w, off, **f32), moe.grouped_dx(c.dy, c.w, c.off, **f32)),
                 (moe.grouped_dw(c.dy, c.x, off, **f32), moe.grouped_dw(c.dy, c.x, c.off, **f32))):
        assert torch.equal(a, b)


def test_workspace_guard_and_smaller_batches():
    """Sums in parts stay within the workspace that is asked for, which serves smaller batches too."""
    require_gpu()
    for d, (N, K) in enumerate(((64, 2048), (2048, 64), (64, 264))):
        big = Case([4000], N, K)
        need = moe._grouped_need(d, 4000, N, K, 1, 0, 1)
        assert need > 0
        buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        at = (-buf.data_ptr()) % 256
        ws = buf[at:at + need]
        for rows in (4000, 700, 65, 33, 1):
            c = Case([rows], N, K)
            f = (lambda **k: moe.grouped(c.x, c.w, c.off, **k), lambda **k: moe.grouped_dx(c.dy, c.w, c.off, **k),
                 lambda **k: moe.grouped_dw(c.dy, c.x, c.off, **k))[d]
            assert torch.equal(f(), f(workspace=ws))
        with pytest.raises(moe.MoeFp4Error, match="workspace"):
            c = big
            f(workspace=ws[:256])
        assert bool((buf[:at] == 0x5A).all()) and bool((buf[at + need:] == 0x5A).all())


def test_512_experts():
    require_gpu()
    c = Case([(i * 7) % 5 for i in range(512)], 40, 72)
    c.product()
    c.dx()
    c.dw()
    c = Case([(i * 7) % 90 for i in range(512)], 136, 64)
    c.product()
    c.dx()


def test_python_refusals():
    require_gpu()
    c = Case([4, 6], 32, 64, 16)
    b = Case([4, 6], 32, 64)
    for call in (lambda: moe.grouped(c.x, c.w, c.off), lambda: moe.grouped(b.x, b.w.float(), b.off), lambda: moe.grouped(b.x.float(), b.w, b.off),
                 lambda: moe.grouped(b.x, b.w, b.off.long()), lambda: moe.grouped(b.x, b.w, b.off, out_dtype=torch.float16),
                 lambda: moe.grouped_dw(b.dy, b.x.float(), b.off)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: moe.grouped(c.x, c.w, c.off, gran_k=16), lambda: moe.grouped(b.x, b.w, b.off, w_gs=c.w_gs),
                 lambda: moe.grouped(c.x, c.w, c.off, w_sf=c.w_sf, gran_k=8), lambda: moe.grouped(b.x[:, :32], b.w, b.off),
                 lambda: moe.grouped(b.x[:, :32].contiguous(), b.w, b.off), lambda: moe.grouped(b.x, b.w, b.off[:2]),
                 lambda: moe.grouped_dx(b.x, b.w, b.off), lambda: moe.grouped(b.x, b.w.transpose(0, 1), b.off),
                 lambda: moe.grouped_dw(b.dy, b.x, b.off, accumulate=True), lambda: moe.grouped_dw(b.dy, b.x[:4], b.off),
                 lambda: moe.grouped(b.x, b.w, b.off, out=torch.empty((9, 32), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(moe.MoeFp4Error, match="overlaps"):
        moe.grouped(b.x[:, :].view(10, 64), b.w.view(2, 32, 64), b.off, out=b.x.view(-1)[:320].view(10, 32))


def test_streams_and_graphs():
    """A call on another stream, and calls of every direction captured together and replayed on new inputs."""
    require_gpu()
    c = Case([30, 0, 200, 9], 264, 328)
    f = lambda: (moe.grouped(c.x, c.w, c.off), moe.grouped_dx(c.dy, c.w, c.off), moe.grouped_dw(c.dy, c.x, c.off, out_dtype=torch.float32))
    want = f()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (moe.grouped(c.x, c.w, c.off, stream=s), moe.grouped_dx(c.dy, c.w, c.off, stream=s),
           moe.grouped_dw(c.dy, c.x, c.off, out_dtype=torch.float32, stream=s))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    for i in range(4):
        c.x.copy_(torch.randn_like(c.x.float()).bfloat16())
        c.dy.copy_(torch.randn_like(c.dy.float()).bfloat16())
        c.off.copy_(offsets_of([[30, 0, 200, 9], [0, 239, 0, 0], [1, 1, 1, 1], [60, 60, 60, 59]][i]))
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        y = [torch.zeros_like(out[0]), torch.zeros_like(out[1])]
        moe.grouped(c.x, c.w, c.off, out=y[0])
        moe.grouped_dx(c.dy, c.w, c.off, out=y[1])
        dw = moe.grouped_dw(c.dy, c.x, c.off, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(out[0], y[0]) and torch.equal(out[1], y[1]) and torch.equal(out[2], dw)


@pytest.mark.parametrize("form", ["grouped", "dx", "dw"])
def test_offsets_past_32_bits(form):
    """Tensors of more than 2^31 elements: an expert's matrix or a row behind them."""
    require_gpu()
    if form == "dw":
        E, N, K, rows = 300, 2048, 4096, [0] * 298 + [40, 3]
    else:
        E, N, K, rows = 300, 2048, 4096, [2] + [0] * 297 + [40, 3]
    off = offsets_of(rows)
    M = sum(rows)
    x, dy = torch.randn((M, K), device="cuda").bfloat16(), torch.randn((M, N), device="cuda").bfloat16()
    if form == "dw":
        out = moe.grouped_dw(dy, x, off)
        ref = dy[40:].double().T @ x[40:].double()
        bound = (19 * U32 + UBF) * (dy[40:].double().abs().T @ x[40:].double().abs())
        assert bool(((out[299].double() - ref).abs() <= bound).all()) and bool((out[:298:50] == 0).all())
        return
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[298:].copy_(torch.randn((2, N, K), device="cuda"))
    out = moe.grouped(x, w, off, out_dtype=torch.float32) if form == "grouped" else moe.grouped_dx(dy, w, off, out_dtype=torch.float32)
    W = w[299].double()
    a = x[42:].double() if form == "grouped" else dy[42:].double()
    W = W.T if form == "grouped" else W
    ref, mag = a @ W, a.abs() @ W.abs()
    assert bool(((out[42:].double() - ref).abs() <= (max(N, K) + 18) * U32 * mag).all()) and bool((out[:2] == 0).all())


def test_more_tiles_than_a_grid_is_wide():
    """256 experts of a row each and N = 2^20: 2^23 workgroups of 512 threads and more."""
    require_gpu()
    E, N, K = 256, 1 << 20, 8
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[E - 1].copy_(torch.randn((N, K), device="cuda"))
    x = torch.randn((E, K), device="cuda").bfloat16()
    out = moe.grouped(x, w, offsets_of([1] * E))
    ref, mag = w[E - 1].double() @ x[E - 1].double(), w[E - 1].double().abs() @ x[E - 1].double().abs()
    b = (K + 18) * U32 * mag
    assert bool(((out[E - 1].double() - ref).abs() <= b + UBF * (ref.abs() + b)).all()) and not bool(out[:E - 1].any())


def test_two_calls_at_once():
    """Calls on two streams with a workspace each, sums in parts among them, give what they give one by one."""
    require_gpu()
    cases = [Case([60], 2048, 64, seed=1), Case([700], 64, 2048, seed=2), Case([33, 20], 2048, 256, 16, seed=3)]
    calls = [lambda c: moe.grouped_dx(c.dy, c.w, c.off, **c.kw()), lambda c: moe.grouped(c.x, c.w, c.off, **c.kw())]
    want = [[f(c) for f in calls] for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append([[f(c) for f in calls] for c in cases])
    torch.cuda.synchronize()
    for g in got:
        for r in g:
            assert all(torch.equal(a, b) for x, y in zip(r, want) for a, b in zip(x, y))


@pytest.mark.parametrize("gran", [0, 16, 32])
@pytest.mark.parametrize("rows", [(300, 420, 17), (100, 90, 65), (257, 256, 31)], ids=str)
def test_dx_of_wide_experts(rows, gran):
    """The larger tiles towards the rows, a sum that is no whole stages, tiles that end with an expert's rows."""
    require_gpu()
    for N in (200, 392):
        Case(rows, N, 32768, gran, seed=N).dx()


@pytest.mark.parametrize("K", [64, 128, 1088])
def test_rows_for_the_wider_stream(K):
    """6 to 12 rows per expert of bfloat16 weights, sums of whole lines."""
    require_gpu()
    Case([10, 8, 12, 7], 72, K).product()
    Case([0, 33, 1, 12, 2], 40, K).product()

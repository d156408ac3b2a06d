"""The FP4 projection with adapters (moe_fp4_project) against a plain FP64
implementation, with a bound on every element worked out from the arithmetic
(moe_plain.project)."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu

pytestmark = pytest.mark.gpu


def bf16(v):
    return torch.from_numpy(v.astype(np.float32)).bfloat16()


class Case:
    def __init__(self, T, N, K, gran, L, R, seed=0, gs=True, mix="each"):
        rng = np.random.default_rng([seed, T, N, K, gran, L, R])
        self.gran, self.L = gran, L
        w, sf = mp.fp4_tensor(rng, 1, N, K, gran)
        self.w, self.sf = w[0], sf[0]
        self.gs = rng.uniform(0.5, 2, 1).astype(np.float32) if gs else None
        self.x = bf16(rng.standard_normal((T, K)))
        self.a = self.b = self.id = self.scale = None
        if L:
            self.a = bf16(rng.standard_normal((L, R, K)) / np.sqrt(K))
            self.b = bf16(rng.standard_normal((L, N, R)))
            self.scale = rng.uniform(-2, 2, L).astype(np.float32)
            if mix == "each":
                self.id = rng.integers(-1, L + 1, T).astype(np.int32)  # (-1 and L: none)
            else:
                self.id = np.sort(rng.integers(-1, L, T)).astype(np.int32)

    def args(self):
        d = lambda v: None if v is None else (v if isinstance(v, torch.Tensor) else torch.from_numpy(v)).cuda()
        return [d(self.x), d(self.w), d(self.sf), d(self.gs), self.gran], dict(
            lora_a=d(self.a), lora_b=d(self.b), lora_id=d(self.id), lora_scale=d(self.scale))

    def ref(self):
        f = lambda v: None if v is None else v.double().numpy()
        return mp.project(f(self.x), self.w, self.sf, self.gs, self.gran, f(self.a), f(self.b), self.id,
                          None if self.scale is None else self.scale.astype(np.float64))

    def check(self):
        args, kw = self.args()
        T, N = self.x.shape[0], self.w.shape[0]
        buf = torch.full((T + 2, N), -77.0, device="cuda")
        f32 = moe.project(*args, **kw, out=buf[1:T + 1])
        b16 = moe.project(*args, **kw)
        torch.cuda.synchronize()
        ref, bound = self.ref()
        got = f32.cpu().numpy().astype(np.float64)
        err = np.abs(got - ref)
        print(f"[project] T={T} N={N} K={self.x.shape[1]} g{self.gran} L={self.L}: err "
              f"{err.max() / np.sqrt(np.mean(ref ** 2)):.2e} rms, {np.max(err / bound):.2e} of its bound", flush=True)
        assert np.all(err <= bound)
        assert bool((buf[0] == -77).all()) and bool((buf[T + 1] == -77).all())
        assert torch.equal(f32.bfloat16().view(torch.int16), b16.view(torch.int16))


SHAPES = [(1, 16, 256, 1, 8), (1, 4096, 6144, 8, 16), (5, 48, 2304, 3, 24), (16, 272, 2048, 5, 128), (17, 144, 512, 2, 8),
          (33, 16, 1024, 7, 16), (48, 400, 2048, 24, 32), (64, 128, 768, 4, 64), (65, 128, 256, 3, 8),
          (130, 1968, 512, 6, 40), (257, 272, 1024, 9, 16), (300, 144, 2304, 3, 128)]


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d-N%d-K%d-L%d-R%d" % s)
def test_project(shape, gran):
    require_gpu()
    T, N, K, L, R = shape
    Case(T, N, K, gran, L, R, gs=gran == 16).check()
    if T > 1:
        Case(T, N, K, gran, L, R, seed=1, gs=gran == 32, mix="runs").check()


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("K", [256, 2304])
@pytest.mark.parametrize("T", [1, 17, 37, 128])
def test_few_tokens_many_rows(T, K, gran):
    """32 rows per workgroup, the last workgroup with 16."""
    require_gpu()
    Case(T, 4112, K, gran, 3, 8, seed=9).check()


@pytest.mark.parametrize("gran", [16, 32])
def test_few_tokens_grouped_by_adapter(gran):
    """Long rows of high rank: few tokens' low-rank activations with matrix instructions too."""
    require_gpu()
    Case(40, 64, 16384, gran, 3, 128, seed=7).check()
    Case(200, 48, 4096, gran, 4, 96, seed=8).check()


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("shape", [(4090, 2032, 256, 5, 24), (4101, 2064, 256, 3, 8), (4101, 2064, 512, 0, 8)],
                         ids=lambda s: "T%d-N%d-K%d-L%d-R%d" % s)
def test_many_tokens(shape, gran):
    """Tiles of 128 x 128 and of 256 x 256, the last of both sides ragged."""
    require_gpu()
    T, N, K, L, R = shape
    Case(T, N, K, gran, L, R, seed=6, mix="sorted" if L == 3 else "each").check()


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("T", [1, 40, 100, 300])
def test_no_adapters(T, gran):
    require_gpu()
    Case(T, 144, 768, gran, 0, 0).check()


@pytest.mark.parametrize("T", [3, 30, 90, 400])
def test_an_adapter_of_nan_stays_with_its_tokens(T):
    require_gpu()
    c = Case(T, 144, 512, 16, 3, 16)
    c.id[:] = np.arange(T) % 4 - 1
    args, kw = c.args()
    want = moe.project(*args, **kw)
    for name in ("lora_a", "lora_b"):
        for bad in (float("nan"), float("inf")):
            k2 = dict(kw)
            k2[name] = kw[name].clone()
            k2[name][1] = bad
            got = moe.project(*args, **k2)
            mine = torch.from_numpy(c.id == 1).cuda()
            assert torch.equal(got[~mine], want[~mine]) and not bool(got[mine].isfinite().any())
    # a token of NaN stays alone too
    x = args[0].clone()
    x[T // 2, 7] = float("nan")
    got = moe.project(x, *args[1:], **kw)
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(got[keep], want[keep]) and bool(got[T // 2].isnan().all())


@pytest.mark.parametrize("T", [4, 70])
def test_rows_of_very_different_sizes(T):
    require_gpu()
    c = Case(T, 48, 512, 16, 2, 8)
    c.x = (c.x.double() * torch.exp2(torch.linspace(-60, 60, T).round().double())[:, None]).bfloat16()
    c.check()


@pytest.mark.parametrize("T", [4, 70, 300])
def test_repeats_captured_and_replayed(T):
    require_gpu()
    c = Case(T, 272, 1024, 32, 4, 16)
    args, kw = c.args()
    other = torch.roll(args[0], 1, 0).contiguous()
    want = [moe.project(v, *args[1:], **kw) for v in (args[0], other)]
    for fill in (0, 255):
        ws = torch.full((8 << 20,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(moe.project(*args, **kw, workspace=ws), want[0])
    buf = args[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = moe.project(buf, *args[1:], **kw)
    for k in range(5):
        buf.copy_((args[0], other)[k & 1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k & 1])
        moe.project(*args, **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = moe.project(*args, **kw, stream=st)
    st.synchronize()
    assert torch.equal(got, want[0])


def test_empty_batch():
    require_gpu()
    args, kw = Case(0, 48, 512, 16, 2, 8).args()
    assert moe.project(*args, **kw).shape == (0, 48)


def test_a_layer_with_an_adapted_shared_expert():
    """gate -> routed experts, the shared expert's two projections with adapters beside it, as one layer's output."""
    require_gpu()
    from test_gpu_gate import plain_gate
    from test_gpu_layer import Layer
    T, E, H, I, k, gran = 11, 6, 512, 256, 2, 16
    L = Layer(E, H, I, gran, 21)
    up, down = Case(T, 2 * I, H, gran, 3, 8, seed=5), Case(T, H, I, gran, 3, 8, seed=6)
    down.id = up.id
    x, gw = L.args(T, 0)
    routed = moe.layer(x, gw, k, *L.d, gran, scoring="sigmoid", renormalize=True, out_dtype=torch.float32)
    (_, w, sf, gs, _), kw = up.args()
    g = moe.project(x, w, sf, gs, gran, **kw, out_dtype=torch.float32)
    h = (torch.nn.functional.silu(g[:, :I]) * g[:, I:]).bfloat16()
    (_, w, sf, gs, _), kw = down.args()
    out = routed + moe.project(h, w, sf, gs, gran, **kw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    ids, wt = plain_gate(L.x[:T], L.gw, k, scoring="sigmoid", renormalize=True)
    want, b0 = mp.layer(L.x[:T], ids, wt, L.w13, L.w13_sf, L.w13_gs, L.w2, L.w2_sf, L.w2_gs, gran, "gate_up", mp.U16)
    up.x, down.x = x.cpu(), h.cpu()
    y, b1 = up.ref()
    assert np.all(np.abs(g.double().cpu().numpy() - y) <= b1)
    y, b2 = down.ref()  # (from the h that went in)
    assert np.all(np.abs(out.double().cpu().numpy() - want - y) <= b0 + b2 + mp.U32 * np.abs(want + y))

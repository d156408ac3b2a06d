"""The whole layer (moe_fp4_layer) against a plain FP64 implementation, with
a bound on every element worked out from the arithmetic (moe_plain.layer): up
to FEW tokens in the two-launch form (h to 11 bits or more), more tokens as
gate + forward (h to bfloat16)."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu
from test_gpu_gate import grid_inputs, plain_gate

pytestmark = pytest.mark.gpu

HREL = {16: mp.U16, 32: 2.0 ** -17}
FEW = {16: 8, 32: 2}


class Layer:
    def __init__(self, E, H, I, gran, seed, wf32=False, gs=True, T=16):
        rng = np.random.default_rng([seed, E, H, I, gran])
        self.E, self.H, self.I, self.gran, self.wf32 = E, H, I, gran, wf32
        self.x, self.gw = grid_inputs(T, E, H, wf32, seed)
        self.w13, self.w13_sf = mp.fp4_tensor(rng, E, 2 * I, H, gran)
        self.w2, self.w2_sf = mp.fp4_tensor(rng, E, H, I, gran)
        self.w13_gs = rng.uniform(0.5, 2, E).astype(np.float32) if gs else None
        self.w2_gs = rng.uniform(0.5, 2, E).astype(np.float32) if gs else None
        d = lambda v: None if v is None else torch.from_numpy(v).cuda()
        self.d = [d(v) for v in (self.w13, self.w13_sf, self.w13_gs, self.w2, self.w2_sf, self.w2_gs)]

    def args(self, T, shared):
        x = torch.from_numpy(self.x[:T]).bfloat16().cuda()
        gw = torch.from_numpy(self.gw[:self.E - shared]).to(torch.float32 if self.wf32 else torch.bfloat16).cuda()
        return x, gw

    def check(self, T, top_k, shared=0, bias=None, order="gate_up", hrel=None, **kw):
        x, gw = self.args(T, shared)
        b = None if bias is None else torch.from_numpy(bias).cuda()
        ids = torch.full((T, top_k + shared), -9, dtype=torch.int32, device="cuda")
        wts = torch.full((T, top_k + shared), -9.0, device="cuda")
        run = lambda **o: moe.layer(x, gw, top_k, *self.d, self.gran, bias=b, shared=shared, w13_order=order, **kw, **o)
        f32 = run(out_dtype=torch.float32, topk_ids=ids, topk_w=wts)
        b16 = run()
        torch.cuda.synchronize()
        rids, rw = plain_gate(self.x[:T], self.gw[:self.E - shared], top_k,
                              None if bias is None else bias.astype(np.float64), shared=shared, **kw)
        assert np.array_equal(ids.cpu().numpy(), rids)
        assert np.allclose(wts.cpu().numpy(), rw, rtol=1024 * mp.U32, atol=0)
        if hrel is None:
            hrel = HREL[self.gran] if T <= FEW[self.gran] else mp.UBF
        ref, bound = mp.layer(self.x[:T], rids, rw, self.w13, self.w13_sf, self.w13_gs, self.w2, self.w2_sf,
                              self.w2_gs, self.gran, order, hrel)
        got = f32.cpu().numpy().astype(np.float64)
        err = np.abs(got - ref)
        rms = max(np.sqrt(np.mean(ref ** 2)), 1e-30)
        print(f"[layer] T={T} E={self.E} k={top_k}+{shared} H={self.H} I={self.I} g{self.gran}: "
              f"err {err.max() / rms:.2e} rms, {np.max(err / np.maximum(bound, 1e-300)):.2e} of its bound", flush=True)
        assert np.all(err <= bound), (np.argmax(err - bound), err.max(), bound.max())
        assert torch.equal(f32.bfloat16().view(torch.int16), b16.view(torch.int16))
        return f32


SHAPES = [(8, 512, 256, 2, 0), (8, 256, 256, 1, 1), (33, 768, 512, 5, 1), (5, 2048, 1536, 3, 2), (300, 512, 256, 8, 0),
          (12, 6144, 256, 4, 0), (6, 4096, 2048, 2, 1)]


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "E%d-H%d-I%d-k%d+%d" % s)
def test_few_tokens(shape, gran):
    require_gpu()
    E, H, I, k, shared = shape
    L = Layer(E, H, I, gran, 1, gs=gran == 16)
    bias = (0.05 * np.random.default_rng(2).standard_normal(E - shared)).astype(np.float32)
    L.check(1, k, shared)
    L.check(2, k, shared, bias=bias)
    L.check(3, k, shared, order="up_gate", scoring="sigmoid", renormalize=True, scale=2.5)
    L.check(8, k, shared, bias=bias, renormalize=True)
    L.check(16, k, shared, bias=bias, scoring="sigmoid")


def test_router_weights_f32_and_no_global_scale():
    require_gpu()
    L = Layer(20, 1024, 512, 16, 3, wf32=True, gs=False)
    for T in (1, 2, 7, 16):
        L.check(T, 3, renormalize=True)
    Layer(20, 1024, 512, 32, 3, wf32=True, gs=True).check(5, 20)


@pytest.mark.parametrize("gran", [16, 32])
def test_more_tokens_run_gate_and_forward(gran):
    require_gpu()
    L = Layer(9, 512, 256, gran, 4, T=130)
    for T in (17, 130):
        L.check(T, 2, 1, hrel=mp.UBF, scoring="sigmoid", renormalize=True)


def test_wide_layer_runs_gate_and_forward():
    """H beyond the two-launch form's range."""
    require_gpu()
    Layer(3, 6400, 256, 32, 5).check(2, 2, hrel=mp.UBF)


@pytest.mark.parametrize("gran", [16, 32])
def test_masked_experts(gran):
    """Few experts left, fewer than top_k, none: the missing terms are zero."""
    require_gpu()
    L = Layer(12, 512, 256, gran, 6)
    for keep in (3, 1, 0):
        bias = np.full(12, -np.inf, np.float32)
        bias[5:5 + keep] = 0.1
        for T in (1, 9):
            out = L.check(T, 2, bias=bias, renormalize=True)
            if keep == 0:
                assert bool((out == 0).all())


@pytest.mark.parametrize("gran", [16, 32])
def test_a_token_of_nan_stays_alone(gran):
    require_gpu()
    L = Layer(12, 512, 256, gran, 7)
    x, gw = L.args(5, 0)
    want = moe.layer(x, gw, 3, *L.d, gran)
    bad = x.clone()
    bad[2, 17] = float("nan")
    ids = torch.empty((5, 3), dtype=torch.int32, device="cuda")
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    got = moe.layer(bad, gw, 3, *L.d, gran, topk_ids=ids, workspace=ws)
    keep = torch.tensor([0, 1, 3, 4], device="cuda")
    assert torch.equal(got[keep], want[keep]) and bool((got[2] == 0).all()) and ids[2].tolist() == [-1] * 3
    assert moe.dropped_assignments(ws) == 3
    inf = x.clone()
    inf[2, 17] = float("inf")  # logits +-inf: no expert either
    got = moe.layer(inf, gw, 3, *L.d, gran)
    assert torch.equal(got[keep], want[keep]) and bool((got[2] == 0).all())


@pytest.mark.parametrize("gran", [16, 32])
def test_h_of_very_different_sizes(gran):
    """Blocks of h far apart in size (group16 keeps them with a shared power of two per 16 values)."""
    require_gpu()
    L = Layer(4, 512, 512, gran, 8, T=4)
    if gran == 32:
        L.w13_sf[:, ::3] = 127 + 20
        L.w13_sf[:, 1::3] = 127 - 40
    else:
        L.w13_sf[:, ::3] = 0x7E   # 448
        L.w13_sf[:, 1::3] = 0x01  # 2^-9
    L.d[1] = torch.from_numpy(L.w13_sf).cuda()
    L.x *= np.array([1, 2.0 ** -20, 2.0 ** 10, 2.0 ** -3])[:, None]
    L.check(4, 2)


def test_workspace_holds_anything_and_results_repeat():
    require_gpu()
    L = Layer(16, 1024, 512, 16, 9)
    x, gw = L.args(6, 0)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((16 << 20,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            out = moe.layer(x, gw, 4, *L.d, 16, workspace=ws)
            first = out if first is None else first
            assert torch.equal(out, first)
        assert int(ws[4:8].view(torch.int32)) == 0


@pytest.mark.parametrize("gran,T", [(16, 4), (32, 2), (32, 4)])
def test_captured_and_replayed(gran, T):
    require_gpu()
    L = Layer(16, 1024, 512, gran, 10)
    x, gw = L.args(T, 0)
    other = torch.roll(x, 1, 0).contiguous()
    want = [moe.layer(v, gw, 3, *L.d, gran) for v in (x, other)]
    buf = x.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = moe.layer(buf, gw, 3, *L.d, gran)
    for k in range(6):
        buf.copy_((x, other)[k & 1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k & 1])
        moe.layer(x, gw, 2, *L.d, gran)


def test_two_streams_at_once():
    """Layers on two streams with their own workspaces: neither waits for workgroups the other keeps out."""
    require_gpu()
    L = Layer(24, 2048, 512, 16, 11)
    x, gw = L.args(8, 0)
    xs = [x, torch.roll(x, 3, 0).contiguous()]
    want = [moe.layer(v, gw, 4, *L.d, 16) for v in xs]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for i in (0, 1):
            outs[i].append(moe.layer(xs[i], gw, 4, *L.d, 16, stream=st[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_empty_batch():
    require_gpu()
    L = Layer(4, 512, 256, 16, 12)
    x, gw = L.args(0, 0)
    assert moe.layer(x, gw, 2, *L.d, 16).shape == (0, 512)

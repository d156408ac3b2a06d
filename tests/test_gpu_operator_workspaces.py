"""Calls with workspaces of exactly the size that the queries give."""

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu
from test_gpu_project import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 48, 512, 0, 0), (1000, 4096, 1024, 0, 0), (2048, 4096, 256, 0, 0), (300, 144, 2304, 3, 16)],
                         ids=lambda s: "T%d-N%d-K%d-L%d-R%d" % s)
def test_project(shape):
    require_gpu()
    T, N, K, L, R = shape
    c = Case(T, N, K, 32, L, R, seed=31)
    args, kw = c.args()
    want = moe.project(*args, **kw)
    ws = torch.full((moe._project_need(T, N, K, 32, moe.OUT_BF16, L, R),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.project(*args, **kw, workspace=ws), want)


GUARD = 4096


def serves(need, call, batches):
    """One workspace, of the size that the largest batch needs: every batch runs in it, in what its own query says,
    and leaves what lies behind alone."""
    big = torch.empty(need(max(batches)) + GUARD, dtype=torch.uint8, device="cuda")
    for T in batches:
        print(f"T={T}", flush=True)
        n = need(T)
        want = call(T, None)
        for size in (n, big.numel() - GUARD):
            big.fill_(255)
            got = call(T, big[:size])
            assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((big[size:] == 255).all())


@pytest.mark.parametrize("w_fmt", [moe.GATE_W_BF16, moe.GATE_W_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("E,H", [(96, 2048), (300, 1000)])
def test_gate_batches_in_one_workspace(E, H, w_fmt):
    require_gpu()
    torch.manual_seed(1)
    x = torch.randn((4000, H), device="cuda").bfloat16()
    w = torch.randn((E, H), device="cuda").to(torch.float32 if w_fmt else torch.bfloat16)
    serves(lambda T: moe._gate_need(4, 0, "softmax", w_fmt, T, E, H), lambda T, ws: moe.gate(x[:T], w, 4, workspace=ws),
           [1, 8, 9, 64, 65, 128, 300, 1000, 4000])


@pytest.mark.parametrize("gran,N,K,L,R", [(16, 528, 4096, 3, 16), (32, 528, 4096, 5, 64), (32, 2064, 512, 0, 0)])
def test_project_batches_in_one_workspace(gran, N, K, L, R):
    require_gpu()
    c = Case(4101, N, K, gran, L, R, seed=32)
    (x, *args), kw = c.args()
    ids = kw["lora_id"]

    def call(T, ws):
        if L:
            kw["lora_id"] = ids[:T]
        return [moe.project(x[:T], *args, **kw, workspace=ws)]
    serves(lambda T: moe._project_need(T, N, K, gran, moe.OUT_BF16, L, R), call,
           [1, 16, 17, 64, 128, 129, 300, 600, 1100, 2048, 2049, 4101])


@pytest.mark.parametrize("gran", [16, 32])
def test_layer_batches_in_one_workspace(gran):
    require_gpu()
    from test_gpu_layer import Layer
    E, H, I, k = 12, 512, 256, 2
    L = Layer(E, H, I, gran, 33, T=1100)
    x, gw = L.args(1100, 0)
    need = lambda T: moe._layer_need(x.device, k, 0, "softmax", moe.GATE_W_BF16, T, E, k, H, I, gran, moe.ACT_BF16, 0,
                                     moe.OUT_BF16, moe.W_RAW)
    serves(need, lambda T, ws: [moe.layer(x[:T], gw, k, *L.d, gran, workspace=ws)], [1, 2, 3, 8, 9, 16, 96, 97, 300, 1100])

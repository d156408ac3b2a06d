"""The binding's checks of gate / layer / project arguments, and their calls
side by side: on two streams, over workspaces that hold anything, into given
outputs."""

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def rnd(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def codes(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()


def scales(gran, *shape):
    return torch.full(shape, 0x30 if gran == 16 else 122, dtype=torch.uint8, device="cuda")


def experts(E, H, I, gran):
    return [codes(1, E, 2 * I, H // 2), scales(gran, E, 2 * I, H // gran), torch.ones(E, device="cuda"),
            codes(2, E, H, I // 2), scales(gran, E, H, I // gran), torch.ones(E, device="cuda")]


def adapted(T, N, K, gran, L=3, R=16):
    ids = torch.arange(T, dtype=torch.int32).remainder(L + 1).sub(1).cuda()
    return [rnd(3, T, K), codes(4, N, K // 2), scales(gran, N, K // gran), torch.ones(1, device="cuda"), gran,
            rnd(5, L, R, K, scale=0.05), rnd(6, L, N, R), ids, torch.ones(L, device="cuda")]


def test_gate_refusals():
    require_gpu()
    x, w, b = rnd(0, 4, 512), rnd(1, 8, 512), torch.zeros(8, device="cuda")
    ok = lambda **k: moe.gate(x, w, 2, **k)
    ok(bias=b)
    for bad, err in ((lambda: moe.gate(x.float(), w, 2), TypeError), (lambda: moe.gate(x, w.half(), 2), TypeError),
                     (lambda: moe.gate(x[:, ::2], w[:, ::2], 2), ValueError), (lambda: moe.gate(x[0], w, 2), ValueError),
                     (lambda: moe.gate(x, w[:, :256].contiguous(), 2), ValueError),
                     (lambda: ok(bias=b[:7]), ValueError), (lambda: ok(bias=b.bfloat16()), TypeError),
                     (lambda: ok(bias=b.cpu()), TypeError), (lambda: ok(scoring="relu"), ValueError),
                     (lambda: ok(topk_ids=torch.zeros(4, 3, dtype=torch.int32, device="cuda")), ValueError),
                     (lambda: ok(topk_ids=torch.zeros(4, 2, dtype=torch.int64, device="cuda")), TypeError),
                     (lambda: ok(topk_w=torch.zeros(4, 2, dtype=BF, device="cuda")), TypeError),
                     (lambda: ok(workspace=torch.zeros(64, device="cuda")), TypeError),
                     (lambda: moe.gate(x, w, 9), moe.MoeFp4Error), (lambda: moe.gate(x, w, 0), moe.MoeFp4Error)):
        with pytest.raises(err):
            bad()
    # a view that starts off a 16-byte boundary
    flat = rnd(2, 4 * 512 + 1)
    with pytest.raises(moe.MoeFp4Error):
        moe.gate(flat[1:].view(4, 512), w, 2)
    with pytest.raises(moe.MoeFp4Error) as e:
        moe.gate(rnd(0, 200, 512), w, 2, workspace=torch.zeros(16, dtype=U8, device="cuda"))
    assert e.value.status == moe.EWORKSPACE


def test_layer_refusals():
    require_gpu()
    x, w, ex = rnd(0, 4, 512), rnd(1, 8, 512), experts(8, 512, 256, 16)
    run = lambda *e, **k: moe.layer(x, w, 2, *(e or ex), 16, **k)
    run()
    swap = lambda i, t: ex[:i] + [t] + ex[i + 1:]
    for bad, err in ((lambda: run(*swap(0, ex[0][:7])), ValueError), (lambda: run(*swap(0, ex[0].to(torch.int8))), TypeError),
                     (lambda: run(*swap(1, ex[1][..., ::2].contiguous())), ValueError),
                     (lambda: run(*swap(2, ex[2][:7])), ValueError), (lambda: run(*swap(3, ex[3].transpose(1, 2))), ValueError),
                     (lambda: run(*swap(4, ex[4].cpu())), TypeError), (lambda: run(shared=1), ValueError),
                     (lambda: run(out=torch.zeros(4, 256, dtype=BF, device="cuda")), ValueError),
                     (lambda: run(out_dtype=torch.float16), TypeError), (lambda: run(quantize_x="int8"), ValueError),
                     (lambda: run(topk_ids=torch.zeros(4, 3, dtype=torch.int32, device="cuda")), ValueError),
                     (lambda: moe.layer(x, w, 2, *ex, 8), ValueError),
                     (lambda: moe.layer(x, w, 9, *ex, 16), moe.MoeFp4Error)):
        with pytest.raises(err):
            bad()
    with pytest.raises(moe.MoeFp4Error) as e:
        run(workspace=torch.zeros(256, dtype=U8, device="cuda"))
    assert e.value.status == moe.EWORKSPACE


def test_project_refusals():
    require_gpu()
    a = adapted(5, 64, 512, 16)
    moe.project(*a)
    swap = lambda i, t: a[:i] + [t] + a[i + 1:]
    for bad, err in ((lambda: moe.project(*swap(0, a[0].float())), TypeError), (lambda: moe.project(*swap(1, a[1][:, :128])), ValueError),
                     (lambda: moe.project(*swap(2, a[2][:32])), ValueError), (lambda: moe.project(*swap(3, torch.ones(2, device="cuda"))), ValueError),
                     (lambda: moe.project(*swap(4, 8)), ValueError), (lambda: moe.project(*swap(5, None)), ValueError),
                     (lambda: moe.project(*swap(6, None)), ValueError), (lambda: moe.project(*swap(7, None)), ValueError),
                     (lambda: moe.project(*swap(8, None)), ValueError), (lambda: moe.project(*swap(5, a[5][0])), ValueError),
                     (lambda: moe.project(*swap(5, a[5][:0])), ValueError), (lambda: moe.project(*swap(6, a[6][:2])), ValueError),
                     (lambda: moe.project(*swap(7, a[7].long())), TypeError), (lambda: moe.project(*swap(7, a[7][:4])), ValueError),
                     (lambda: moe.project(*a, out_dtype=torch.float16), TypeError),
                     (lambda: moe.project(*a, workspace=torch.zeros(16, dtype=U8, device="cuda")), moe.MoeFp4Error)):
        with pytest.raises(err):
            bad()


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("T", [1, 20, 100, 150, 700, 2100])
def test_project_streams_workspaces_and_outputs(T, gran):
    """The same result into a given output, over a workspace of any content, and on two streams at once."""
    require_gpu()
    a = adapted(T, 528, 1024, gran)
    want = moe.project(*a)
    wide = moe.project(*a, out_dtype=F32)
    assert torch.equal(wide.bfloat16(), want)
    for fill in (0, 127, 255):
        ws = torch.full((64 << 20,), fill, dtype=U8, device="cuda")
        out = torch.full_like(want, float("nan"))
        assert moe.project(*a, out=out, workspace=ws) is out and torch.equal(out, want)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [moe.project(*a, stream=st[i & 1]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("T", [1, 16, 17, 300])
def test_gate_streams_and_workspaces(T):
    require_gpu()
    x, w = rnd(0, T, 1024), rnd(1, 100, 1024, dtype=F32)
    ids, wt = moe.gate(x, w, 6, shared=2)
    for fill in (0, 127, 255):
        ws = torch.full((32 << 20,), fill, dtype=U8, device="cuda")
        i2, w2 = torch.full_like(ids, -7), torch.full_like(wt, float("nan"))
        r = moe.gate(x, w, 6, shared=2, workspace=ws, topk_ids=i2, topk_w=w2)
        assert r[0] is i2 and r[1] is w2 and torch.equal(i2, ids) and torch.equal(w2, wt)
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [moe.gate(x, w, 6, shared=2, stream=st[i & 1]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(i, ids) and torch.equal(v, wt) for i, v in outs)


@pytest.mark.parametrize("quant", ["fp8", "fp4"])
@pytest.mark.parametrize("T", [1, 6, 90])
def test_layer_of_quantised_activations_is_gate_and_forward(T, quant):
    require_gpu()
    x, w, ex = rnd(0, T, 512), rnd(1, 8, 512), experts(8, 512, 512, 32)
    ids, wt = moe.gate(x, w, 2, renormalize=True)
    want = moe.forward(x, ids, wt, *ex, 32, quantize_x=quant)
    assert torch.equal(moe.layer(x, w, 2, *ex, 32, renormalize=True, quantize_x=quant), want)


def test_layers_of_two_sizes_share_a_workspace():
    """One after the other on one stream, captured into two graphs that are replayed in turn."""
    require_gpu()
    w, ex = rnd(1, 8, 512), experts(8, 512, 256, 16)
    xs = [rnd(7, 3, 512), rnd(8, 40, 512)]
    want = [moe.layer(x, w, 2, *ex, 16) for x in xs]
    ws = torch.empty(32 << 20, dtype=U8, device="cuda")
    outs = [torch.empty_like(o) for o in want]
    graphs = []
    for x, o in zip(xs, outs):
        moe.layer(x, w, 2, *ex, 16, out=o, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.layer(x, w, 2, *ex, 16, out=o, workspace=ws)
        graphs.append(g)
    for k in range(6):
        for o in outs:
            o.zero_()
        for g in graphs if k & 1 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))

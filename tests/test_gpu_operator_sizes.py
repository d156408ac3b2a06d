"""The router and the projection at the far ends of their sizes, where 32-bit
arithmetic would wrap; results are compared with FP64 in sampled places."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
import moe_plain as mp
from helpers import require_gpu

pytestmark = pytest.mark.gpu


def sampled(rng, n, count):
    return np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, count)]))


def check_project(T, N, K, gran, L, R, seed):
    print(f"T={T} N={N} K={K} gran={gran} L={L} R={R}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(117, 126, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8) if gran == 32 else \
        torch.randint(0x10, 0x30, (N, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    kw, ids = {}, None
    if L:
        a = (torch.randn((L, R, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
        b = torch.empty((L, N, R), device="cuda", dtype=torch.bfloat16)
        b.normal_(generator=g)
        ids = rng.integers(-1, L, T).astype(np.int32)
        ids[-1] = L - 1
        kw = dict(lora_a=a, lora_b=b, lora_id=torch.from_numpy(ids).cuda(),
                  lora_scale=torch.linspace(0.5, 1.5, L, device="cuda"))
    out = moe.project(x, w, sf, None, gran, **kw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    t, n = sampled(rng, T, 30), sampled(rng, N, 60)
    td, nd = torch.from_numpy(t).cuda(), torch.from_numpy(n).cuda()
    f = lambda v: v.double().cpu().numpy()
    if L:
        used = np.unique(ids[t][ids[t] >= 0])
        ud = torch.from_numpy(used).cuda()
        pos = np.full(L + 1, -1)
        pos[used] = np.arange(len(used))
        lora = (f(a[ud]), f(b[ud][:, nd]), pos[ids[t]], f(kw["lora_scale"][ud]))
    else:
        lora = (None,) * 4
    ref, bound = mp.project(f(x[td]), w[nd].cpu().numpy(), sf[nd].cpu().numpy(), None, gran, *lora)
    err = np.abs(f(out[td][:, nd]) - ref)
    print(f"[project] T={T} N={N} K={K} L={L} R={R}: {np.max(err / bound):.2e} of the bound", flush=True)
    assert np.all(err <= bound)
    assert bool(out.isfinite().all())
    return out


@pytest.mark.parametrize("T", [2, 100, 150])
def test_project_matrix_of_nearly_2_to_the_32_elements(T):
    require_gpu()
    check_project(T, (1 << 20) - 16, 3840, 32, 0, 0, 1)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [3, 70, 400])
def test_project_adapters_of_nearly_2_to_the_32_elements(T):
    require_gpu()
    check_project(T, (1 << 16) - 16, 256, 16, 511, 128, 2)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("L", [0, 3])
def test_project_of_many_tokens(L):
    require_gpu()
    check_project((1 << 22) + 13, 272, 256, 32, L, 8, 3)  # T * N past 2^30, T * K past 2^30
    torch.cuda.empty_cache()


def test_project_of_long_rows():
    require_gpu()
    for T in (2, 130):
        check_project(T, 16, 1 << 20, 16, 2, 8, 4)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("wf32", [False, True], ids=["bf16", "f32"])
def test_gate_of_many_tokens(wf32):
    """Logits of 2 GB and more: rows behind 2^31 bytes are as right as the first."""
    require_gpu()
    T, E, H, k = (1 << 21) + 77, 300, 64, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    # (a grid whose products sum exactly)
    x = torch.randint(-8, 9, (T, H), generator=g, device="cuda").bfloat16()
    w = (torch.randint(-64, 65, (E, H), generator=g, device="cuda") / 128).to(torch.float32 if wf32 else torch.bfloat16)
    ids, wt = moe.gate(x, w, k, scoring="sigmoid", renormalize=True)
    torch.cuda.synchronize()
    rng = np.random.default_rng(6)
    t = sampled(rng, T, 500)
    td = torch.from_numpy(t).cuda()
    z = x[td].double().cpu().numpy() @ w.double().cpu().numpy().T
    want = np.argsort(-z, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids[td].cpu().numpy(), want)
    ls = -np.logaddexp(0, -np.take_along_axis(z, want, 1))
    p = np.exp(ls - ls.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    assert np.all(np.abs(wt[td].double().cpu().numpy() / p - 1) <= (k + 24) * 2.0 ** -24)
    assert int(ids.min()) >= 0 and int(ids.max()) < E and bool(wt.isfinite().all())


def test_gate_of_long_rows():
    require_gpu()
    T, E, H = 20, 5, 1 << 22
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randint(-1, 2, (T, H), generator=g, device="cuda").bfloat16()
    w = torch.randint(-1, 2, (E, H), generator=g, device="cuda").bfloat16()
    z = (x.double() @ w.double().T).cpu().numpy()  # whole numbers below 2^22: exact in FP32
    for n in (1, 20):
        ids, _ = moe.gate(x[:n], w, 3)
        assert np.array_equal(ids.cpu().numpy(), np.argsort(-z[:n], axis=1, kind="stable")[:, :3])

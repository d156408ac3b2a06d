"""The router where its scores leave FP32's range, against FP64.

Logits are planted: x holds 1 in two columns and the router's rows hold the
logit's integer and its 64ths there, so that every logit is exact."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu

pytestmark = pytest.mark.gpu


def planted(T, logits, H=64):
    """x [T, H], w [E, H] with x w^T = logits (multiples of 1/64) for every token; whole numbers up to 2^11 in
    columns 0 and 1 (bfloat16 holds 8 bits), 64ths in column 2."""
    whole = np.floor(logits)
    x, w = np.zeros((T, H)), np.zeros((len(logits), H))
    x[:, :3] = 1
    w[:, 0] = np.floor(whole / 16) * 16
    w[:, 1] = whole - w[:, 0]
    w[:, 2] = logits - whole
    return x, w


def log_score(z, scoring):
    """log of the score, whatever its size."""
    if scoring == "softmax":
        m = z.max()
        return z - m - np.log(np.exp(z - m).sum())
    return np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))


def renormalised(z, k, scoring, bias, scale):
    """ids by score (+ bias) in FP64, lower index first among equals; weights from the scores' logarithms."""
    ls = log_score(z, scoring)
    sel = z.copy() if bias is None else np.exp(ls) + bias
    ids = np.argsort(-sel, kind="stable")[:k]
    ids = ids[sel[ids] > -np.inf]
    e = np.exp(ls[ids] - ls[ids].max())
    return ids, e / e.sum() * scale


def run(T, z, wf32, k, bias, **kw):
    x, w = planted(T, z)
    xd = torch.from_numpy(x).bfloat16().cuda()
    wd = torch.from_numpy(w).to(torch.float32 if wf32 else torch.bfloat16).cuda()
    assert np.array_equal(xd.double().cpu().numpy() @ wd.double().cpu().numpy().T, np.tile(z, (T, 1)))
    bd = None if bias is None else torch.from_numpy(bias).cuda()
    ids, wt = moe.gate(xd, wd, k, bias=bd, renormalize=True, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), wt.double().cpu().numpy()


def check(T, z, wf32, k, bias, scoring, scale):
    """Tolerance: exp of an exact argument and a division, 2 ulp each, the sum over the selected scores and two
    roundings more: (k + 16) half steps, plus the E roundings of a softmax's sum where it counts."""
    ids, wt = run(T, z, wf32, k, bias, scoring=scoring, scale=scale)
    rids, rwt = renormalised(z, k, scoring, None if bias is None else bias.astype(np.float64), scale)
    n = len(rids)
    assert np.array_equal(ids[:, :n], np.tile(rids, (T, 1))) and np.all(ids[:, n:] == -1) and np.all(wt[:, n:] == 0)
    err = np.max(np.abs(wt[:, :n] / rwt - 1))
    print(f"[gate] T={T} {scoring} top logit {z.max()} scale {scale}: relative error {err:.2e}", flush=True)
    assert err <= (k + 16 + len(z)) * 2.0 ** -24


ROWS = [(3, False), (20, False), (3, True), (70, True)]  # dot and tiled, both weight formats


@pytest.mark.parametrize("top", [-20, -69, -70, -87, -88, -89, -95, -104, -110, -150, -1000])
@pytest.mark.parametrize("T,wf32", ROWS)
def test_renormalised_sigmoid_of_very_negative_logits(T, wf32, top):
    """Scores below FP32's range, whose ratios are ordinary numbers."""
    require_gpu()
    for E in (24, 100, 200, 400):  # 1, 2, 4 and 8 experts per lane
        sigmoid_case(T, wf32, top, E, 6)


def sigmoid_case(T, wf32, top, E, k):
    z = top - (np.random.default_rng(1).permutation(E) + 16) / 64
    check(T, z, wf32, k, None, "sigmoid", 2.5)
    # selected by the bias alone: its steps are far larger than the scores
    bias = (np.random.default_rng(2).permutation(E) / 4).astype(np.float32)
    check(T, z, wf32, k, bias, "sigmoid", 1.0)
    # fewer left than top_k
    bias[np.random.default_rng(3).permutation(E)[:E - 4]] = -np.inf
    check(T, z, wf32, k, bias, "sigmoid", 1.0)


@pytest.mark.parametrize("gap", [20, 69, 87, 89, 100, 110, 300, 700])
@pytest.mark.parametrize("T,wf32", ROWS)
def test_renormalised_softmax_behind_masked_experts(T, wf32, gap):
    """The experts that hold the softmax's mass are masked; those left share the weight."""
    require_gpu()
    for E in (40, 300):
        softmax_case(T, wf32, gap, E, 4)


def softmax_case(T, wf32, gap, E, k):
    z = 3.0 - gap - np.random.default_rng(4).permutation(E) / 64
    z[[2, 17, 39]] = [3.0, 2.5, 3.25]
    bias = np.zeros(E, np.float32)
    bias[[2, 17, 39]] = -np.inf
    check(T, z, wf32, k, bias, "softmax", 2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,wf32", ROWS)
def test_renormalised_with_a_large_factor(T, wf32, scoring):
    """A factor whose quotient with the scores' sum is beyond FP32, though the weights are not."""
    require_gpu()
    z = -2.0 - np.random.default_rng(5).permutation(64) / 64
    check(T, z, wf32, 4, None, scoring, float(np.float32(1e38)))


def unique(rng, shape, lo=0x3F800000, span=1 << 23):
    """Floats of one binade with all 24 bits in use, no two alike."""
    n = int(np.prod(shape))
    bits = (lo + rng.choice(span // 2, n, replace=False) * 2 + 1).astype(np.uint32)
    return bits.view(np.float32).reshape(shape)


@pytest.mark.parametrize("T", [3, 64, 65, 200])
def test_all_24_bits_of_fp32_weights_count(T):
    """Every token looks at one column, so that a logit is one weight, exactly; the experts' weights differ in their
    last bits only.  (Dot products up to 64 tokens, three bfloat16 planes beyond.)"""
    require_gpu()
    E, H, k = 96, 72, 10
    rng = np.random.default_rng(6)
    # 1 + 2^-8 + odd multiples of 2^-23 below 2^-15: the first two planes are the same for every expert
    w = np.stack([unique(rng, E, 0x3F808000, 1 << 8) for _ in range(H)], 1)
    rest = w - np.float32(1)
    assert np.all(rest.view(np.uint32) >> 16 == np.float32(2.0 ** -8).view(np.uint32) >> 16)
    assert all(len(np.unique(w[:, h])) == E for h in range(H))
    w = (w * np.where(np.arange(H) % 2, -1, 1)).astype(np.float32)
    x = np.zeros((T, H))
    x[np.arange(T), np.arange(T) % H] = np.where(np.arange(T) % 3, 2.0, -0.5)
    z = x @ w.astype(np.float64).T
    ids, wt = moe.gate(torch.from_numpy(x).bfloat16().cuda(), torch.from_numpy(w).cuda(), k, scoring="sigmoid")
    torch.cuda.synchronize()
    want = np.argsort(-z, axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids.cpu().numpy(), want)
    p = 1 / (1 + np.exp(-np.take_along_axis(z, want, 1)))
    # exp and division 2 ulp each, their sum a rounding
    assert np.all(np.abs(wt.double().cpu().numpy() / p - 1) <= 10 * 2.0 ** -24)


@pytest.mark.parametrize("T,E,H", [(64, 40, 520), (65, 40, 520), (130, 64, 6144), (300, 7, 64), (129, 33, 2056)])
def test_fp32_weights_of_24_bits_within_the_bound_of_an_fp32_sum(T, E, H):
    """All experts taken, so that no order is in question.  A logit is off by (H + 8) half steps of the sum of its
    products' sizes at most, a sigmoid relatively by as much as its logit (and 10 half steps of its own)."""
    require_gpu()
    rng = np.random.default_rng([7, T, E, H])
    w = (unique(rng, (E, H)) * rng.choice([-1, 1], (E, H)) * 2.0 ** -round(np.log2(np.sqrt(H)))).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, H))).bfloat16()
    ids, wt = moe.gate(x.cuda(), torch.from_numpy(w).cuda(), E, scoring="sigmoid")
    torch.cuda.synchronize()
    ids, wt = ids.cpu().numpy(), wt.double().cpu().numpy()
    assert np.array_equal(np.sort(ids, 1), np.tile(np.arange(E), (T, 1)))
    xd, wd = x.double().numpy(), w.astype(np.float64)
    p = 1 / (1 + np.exp(-xd @ wd.T))
    dz = (H + 8) * 2.0 ** -24 * (np.abs(xd) @ np.abs(wd).T)
    got = np.empty((T, E))
    np.put_along_axis(got, ids, wt, 1)
    ratio = np.abs(got / p - 1) / (np.expm1(dz) + 10 * 2.0 ** -24)
    print(f"[gate] T={T} E={E} H={H}: {ratio.max():.3f} of the bound", flush=True)
    assert ratio.max() <= 1


@pytest.mark.parametrize("wf32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 7, 8, 9, 63, 64, 65])
def test_around_the_border_of_the_dot_form(T, wf32):
    """8 tokens with bfloat16 weights, 64 with FP32 ones; odd numbers of experts, H no multiple of a stage."""
    require_gpu()
    import test_gpu_gate as g
    for E, H in ((97, 200), (130, 2056), (3, 8), (511, 72)):
        x, w = g.grid_inputs(T, E, H, wf32, 8)
        bias = (0.05 * np.random.default_rng(9).standard_normal(E)).astype(np.float32)
        k = min(8, E)
        for b, kw in ((None, dict(scoring="softmax")), (bias, dict(scoring="sigmoid", renormalize=True, scale=2.5, shared=1))):
            g.check(g.run(x, w, wf32, k, b, **kw), g.plain_gate(x, w, k, None if b is None else b.astype(np.float64), **kw),
                    np.abs(x @ w.T).max() * 2, E)

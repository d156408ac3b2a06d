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

"""The adapted projection at the ends of the number range: infinities in B,
products and low-rank activations past what bfloat16 or FP32 hold.  Every
batch size gives what the definition gives, whichever form runs it."""

import numpy as np
import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu
from test_gpu_project import Case, bf16

pytestmark = pytest.mark.gpu

F32MAX = float(np.finfo(np.float32).max)
# the few-token form; 64-token tiles, whole and with K in parts; tiles of 128 and of 256
SHAPES = [(40, 144, 512), (300, 144, 512), (300, 144, 2304), (4090, 2032, 256), (4101, 2064, 256)]
ids = lambda s: "T%d-N%d-K%d" % s


def one_hot_a(c, l):
    """A_l x = x's first elements, exactly."""
    a = np.zeros(tuple(c.a.shape[1:]))
    a[np.arange(a.shape[0]), np.arange(a.shape[0])] = 1
    c.a[l] = bf16(a)


@pytest.mark.parametrize("gran", [16, 32])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_infinities_of_b(shape, gran):
    """inf times a low-rank activation that is not zero is inf, of the product's sign; a product past FP32 is too;
    two of different sign, and NaN, are NaN; no other element is touched."""
    require_gpu()
    c = Case(*shape, gran, 3, 16, seed=11)
    one_hot_a(c, 0)
    one_hot_a(c, 1)   # low-rank activations of 8 bits
    c.scale[:] = (700.0, 1.0, 1.5)
    c.x[:, :16] = torch.where(c.x[:, :16] == 0, torch.ones(()).bfloat16(), c.x[:, :16])
    plain = c.ref()
    c.b[0, 13] = 0
    c.b[0, 13, 2] = 3e38      # times 700: past FP32
    c.b[0, 14] = 0
    c.b[0, 14, 1] = -3e38
    c.b[1, 5, 3] = float("inf")
    c.b[1, 7, 0] = -float("inf")
    c.b[1, 15, 15] = float("inf")
    c.b[1, 9, 2], c.b[1, 9, 4] = float("inf"), float("nan")
    c.b[2, 11, 1] = float("inf")
    c.b[2, 12, 6] = -float("inf")
    c.b[2, 40, 1] = c.b[2, 40, 2] = float("inf")
    args, kw = c.args()
    got = moe.project(*args, **kw, out_dtype=torch.float32)
    b16 = moe.project(*args, **kw)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    x, a, b = (v.double().numpy() for v in (c.x, c.a, c.b))
    want, bound = plain
    with np.errstate(all="ignore"):
        for l in range(3):
            t = np.nonzero(c.id == l)[0]
            u = c.scale[l].astype(np.float64) * (x[t] @ a[l].T)
            assert np.all(np.abs(u) > 0)
            n = np.nonzero(np.any(~np.isfinite(b[l]) | (np.abs(b[l]) > 1e38), axis=1))[0]
            s = np.zeros((len(t), len(n)))
            for r in range(16):   # (in turn: inf - inf is NaN in any order)
                s += u[:, r:r + 1] * b[l][n, r]
            s[s > F32MAX], s[s < -F32MAX] = np.inf, -np.inf
            want[np.ix_(t, n)] = np.where(np.abs(s) < 1e38, want[np.ix_(t, n)], s)
            if l == 0:  # (a product that stays within FP32)
                near = np.abs(s) < np.inf
                got_n = got[np.ix_(t, n)]
                assert np.all(np.abs(got_n[near] - s[near]) <= 2.0 ** -15 * np.abs(s[near]) + 1e6)
                want[np.ix_(t, n)] = np.where(near, got_n, s)
    fin = np.isfinite(want)
    assert (~fin).sum() > 3 * len(c.id) // 8
    assert np.array_equal(np.nan_to_num(got[~fin], nan=7.0, posinf=1, neginf=-1),
                          np.nan_to_num(want[~fin], nan=7.0, posinf=1, neginf=-1))
    assert np.all(np.abs(got[fin] - want[fin]) <= bound[fin])
    assert torch.equal(torch.from_numpy(got).float().bfloat16().nan_to_num(7), b16.cpu().nan_to_num(7))


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_low_rank_activations_near_the_largest_float(shape):
    """Finite, but rounded to bfloat16 they would be infinite."""
    require_gpu()
    c = Case(*shape, 32, 2, 8, seed=12, gs=False)
    one_hot_a(c, 0)
    one_hot_a(c, 1)
    c.x[:, :8] = torch.where(c.x[:, :8] < 0, -torch.ones(()), torch.ones(())).bfloat16()
    c.scale[:] = np.float32(3.4e38)
    c.b = (c.b.double() * 2.0 ** -110).bfloat16()
    c.b[:, 3] = 0
    c.check()

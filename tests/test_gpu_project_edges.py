"""The adapted projection at the ends of the number range: every batch size
gives what the definition gives, whichever form runs it."""

import numpy as np
import pytest
import torch

from helpers import require_gpu
from test_gpu_project import Case, bf16

pytestmark = pytest.mark.gpu

# the few-token form; 64-token tiles, whole and with K in parts; tiles of 128 and of 256
SHAPES = [(40, 144, 512), (300, 144, 512), (300, 144, 2304), (4090, 2032, 256), (4101, 2064, 256)]
ids = lambda s: "T%d-N%d-K%d" % s


def one_hot_a(c, l):
    """A_l x = x's first elements, exactly."""
    a = np.zeros(tuple(c.a.shape[1:]))
    a[np.arange(a.shape[0]), np.arange(a.shape[0])] = 1
    c.a[l] = bf16(a)


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

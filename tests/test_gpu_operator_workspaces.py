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

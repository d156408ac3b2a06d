"""Weight gradients added to what is there: an expert without rows keeps its
bits (a sum of nothing added would make -0.0 of 0.0 and quiet a NaN), in every
form of the kernel; an expert with rows gets one FP32 addition."""

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu
from test_gpu_grouped import offsets_of

pytestmark = pytest.mark.gpu

# tiles of 64 either way, 128 and 256; sums in parts
FORMS = [([5, 0, 70], 40, 136), ([5, 0, 70], 136, 40), ([300, 0, 65], 520, 136), ([0, 200, 0, 90], 2056, 2568), ([4000, 0, 9000], 72, 136),
         ([0, 3000], 264, 520)]


def bits(t):
    return t.view(torch.int32 if t.dtype is torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["float32", "bfloat16"])
@pytest.mark.parametrize("rows,N,K", FORMS, ids=str)
def test_accumulate_leaves_idle_experts(rows, N, K, dtype):
    require_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(N + K)
    M, E = sum(rows), len(rows)
    dy, x = (torch.randn((M, n), generator=g, device="cuda").bfloat16() for n in (N, K))
    old = torch.randn((E, N, K), generator=g, device="cuda").to(dtype)
    old[:, :, ::3] = -0.0
    # NaNs with bits of their own, a signalling one among them
    bits(old)[:, ::5, 1] = 0x7F800001 if dtype is torch.float32 else 0x7F81
    bits(old)[:, ::5, 2] = -3
    inside = offsets_of(rows)
    beyond = inside.clone()
    beyond[E] += 100  # (taken within the rows; a last expert behind them has none)
    behind = torch.cat([inside, inside[-1:] + 200])
    for off, start in ((inside, old), (beyond, old), (behind, torch.cat([old, old[:1]]))):
        off[-1] = max(int(off[-1]), M)
        out = start.clone()
        assert moe.grouped_dw(dy, x, off, out=out, accumulate=True) is out
        ref = moe.grouped_dw(dy, x, off, out_dtype=torch.float32)  # (the same number of experts: the same parts of the sums)
        torch.cuda.synchronize()
        for e in range(start.shape[0]):
            if e >= E or rows[e] == 0:
                assert torch.equal(bits(out[e]), bits(start[e])), f"expert {e} without rows has changed"
            else:
                want = (start[e].float() + ref[e]).to(dtype)
                assert torch.equal(torch.nan_to_num(out[e], nan=7.0), torch.nan_to_num(want, nan=7.0)), f"expert {e}"

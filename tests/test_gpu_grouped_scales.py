"""FP4 weights over the whole range of their scales: a code times its scale
enters the products exactly wherever it is below 2^128 (as bfloat16 it is a
subnormal at the lower end), and the NaN scale is NaN."""

import math

import pytest
import torch

import block_scaled_fp4_topk_amd as moe
from helpers import require_gpu

pytestmark = pytest.mark.gpu
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# every scale with all codes; 253 and 254 with the codes whose product stays below 2^128
UE8M0 = [(b, 8) for b in (0, 1, 2, 3, 64, 126, 127, 190, 251, 252)] + [(253, 6), (254, 4)]


# (rows: the stream of the weights; tiles of 64; of 256, of some experts)
@pytest.mark.parametrize("rows,E", [(1, 1), (100, 1), (300, 130)])
@pytest.mark.parametrize("byte,codes", UE8M0, ids=lambda v: str(v))
def test_group32(byte, codes, rows, E):
    """One element of x (dy) is a power of two that brings the products into FP32's range, so that every output is one
    exact product."""
    require_gpu()
    N, K = 520, 288
    code = (torch.arange(N) % codes) | 8 * ((torch.arange(N) // codes) & 1)
    w = (code | code << 4).to(torch.uint8).view(1, N, 1).expand(E, N, K // 2).contiguous().cuda()
    sf = torch.full((E, N, K // 32), byte, dtype=torch.uint8, device="cuda")
    off = (torch.arange(E + 1, device="cuda") * rows).int()
    M = E * rows
    up = 60 if byte < 64 else -60 if byte > 190 else 0
    want = torch.tensor([math.copysign(math.ldexp(E2M1[c & 7], byte - 127 + up), -1 if c & 8 else 1) for c in code.tolist()], device="cuda")
    at_k, at_n = torch.arange(M, device="cuda") % K, torch.arange(M, device="cuda") % N
    x = torch.zeros((M, K), device="cuda").scatter_(1, at_k[:, None], 2.0 ** up).bfloat16()
    dy = torch.zeros((M, N), device="cuda").scatter_(1, at_n[:, None], 2.0 ** up).bfloat16()
    y = moe.grouped(x, w, off, w_sf=sf, gran_k=32, out_dtype=torch.float32)
    dx = moe.grouped_dx(dy, w, off, w_sf=sf, gran_k=32, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(y, want.expand(M, N))
    assert torch.equal(dx, want[at_n][:, None].expand(M, K))


@pytest.mark.parametrize("rows", [1, 100])
def test_group16(rows):
    """E4M3 scales of every byte, subnormal, negative and NaN ones among them."""
    require_gpu()
    N, K = 256, 64
    w = torch.full((1, N, K // 2), 0x7D, dtype=torch.uint8, device="cuda")  # 3 and 6 in turn
    byte = torch.arange(N, device="cuda").to(torch.uint8)
    sf = byte.view(1, N, 1).expand(1, N, K // 16).contiguous()
    value = byte.view(torch.float8_e4m3fn).float()
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    x = torch.zeros((rows, K), device="cuda")
    x[:, 35] = 1
    y = moe.grouped(x.bfloat16(), w, off, w_sf=sf, gran_k=16, out_dtype=torch.float32)
    torch.cuda.synchronize()
    # (element 35 is the high nibble, 7: 6; low 0xD: -3)
    want = (6 * value).expand(rows, N)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y, nan=0.5), torch.nan_to_num(want, nan=0.5))


@pytest.mark.parametrize("rows", [1, 100])
def test_nan_scale(rows):
    require_gpu()
    w = torch.zeros((1, 8, 16), dtype=torch.uint8, device="cuda")
    sf = torch.full((1, 8, 1), 127, dtype=torch.uint8, device="cuda")
    sf[0, 3] = 255
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y = moe.grouped(torch.ones((rows, 32), device="cuda").bfloat16(), w, off, w_sf=sf, gran_k=32, out_dtype=torch.float32)
    torch.cuda.synchronize()
    nan = torch.isnan(y)
    assert bool(nan[:, 3].all()) and not bool(y[:, [0, 1, 2, 4, 5, 6, 7]].any())

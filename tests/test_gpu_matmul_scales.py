"""Dense e4m3 products whose scales meet at the borders of what the entry point
takes: products of two scales from 2^-126, the smallest normal binary32 number,
and up to below 2^128.  Tolerances are those of test_gpu_matmul.py."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import test_gpu_matmul as mm
from gpu_util import device

pytestmark = pytest.mark.gpu


def scales(rows, blocks, exponent, seed):
    """2^exponent times [1, 2), both ends of the range among them."""
    g = torch.Generator(device=device()).manual_seed(seed)
    s = 1 + torch.rand(rows, blocks, generator=g, device=device())
    s = s.clamp(max=2 - 2.0 ** -23)
    s.view(-1)[::3] = 1.0
    s.view(-1)[1::3] = 2 - 2.0 ** -23
    return s * 2.0 ** exponent


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 100), (33, 200), (70, 130), (300, 1030), (4100, 300)])
@pytest.mark.parametrize("ea,eb", [(-63, -63), (-120, -6), (20, -146), (63, 63), (100, 26), (0, 126)])
def test_border(M, N, dtype, rows, ea, eb):
    dev, K = device(), 384
    a, _ = mm.operand(M, K, 1, M + N, dev)
    b, _ = mm.operand(N, K, 1 if rows else 128, M + N + 1, dev)
    if ea + eb > 0:       # codes below 2^-6: a result of at most 2^128 K 2^-12, so that it is finite
        a, b = a & 0x87, b & 0x87
    sa, sb = scales(M, K // 128, ea, 1), scales(N if rows else -(-N // 128), K // 128, eb, 2)
    # 2^-146 [1, 2) itself has no more than three binary digits
    p = sa[:, None].double() * sb[None].double()
    keep = p.amin() >= 2.0 ** -126 and p.amax() < 2.0 ** 128
    assert keep
    mm.check(gl.matmul_e4m3(a, sa, b, sb, dtype=dtype), a, sa, b, sb, rows)

"""Head norms at the ends of binary32, for heads that fill their lanes and heads
that do not."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
from gpu_util import device

pytestmark = pytest.mark.gpu

HEADS = [8, 24, 32, 40, 72, 128, 136, 200, 256]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", HEADS)
def test_squares_past_the_range_give_zeros(D, interleaved):
    # 1e25 squared is past binary32: the inverse root is 0, and so is the head, its
    # gradient and what it adds to the weight's; the heads beside it are as ever
    dev, g = device(), torch.Generator().manual_seed(D)
    q, k = (torch.randn(3, h, D, generator=g).to(dev) for h in (5, 2))
    d_q, d_k = (torch.randn(3, h, D, generator=g).to(dev) for h in (5, 2))
    w, pos = torch.ones(D, device=dev), torch.arange(3, dtype=torch.int32, device=dev)
    rot = D // 16 * 16
    args = dict(positions=pos, inv_freq=gl.rope_frequencies(rot, 1e4, dev) if rot else None, interleaved=interleaved)
    y, _ = gl.qk_norm_rope(q, k, w, w, **args)
    for at in (0, D - 1):
        x = q.clone()
        x[1, 3, at] = 1e25
        big, _ = gl.qk_norm_rope(x, k, w, w, **args)
        got = gl.qk_norm_rope_backward(d_q, d_k, x, k, w, w, **args)
        assert (big[1, 3] == 0).all() and (got["d_q"][1, 3] == 0).all()
        big[1, 3] = y[1, 3]
        assert torch.equal(big, y)
        without = d_q.clone()
        without[1, 3] = 0
        want = gl.qk_norm_rope_backward(without, d_k, q, k, w, w, **args)
        assert torch.equal(got["d_q_weight"], want["d_q_weight"])
        assert torch.equal(got["d_k_weight"], want["d_k_weight"])


@pytest.mark.parametrize("eps", [1.2e-38, 1e-30, 1e-6])
@pytest.mark.parametrize("D", [24, 128])
def test_zeros_under_a_small_eps(D, eps):
    dev = device()
    q, w = torch.zeros(2, 3, D, device=dev), torch.ones(D, device=dev)
    y, _ = gl.qk_norm_rope(q, q, w, w, eps=eps)
    got = gl.qk_norm_rope_backward(q, q, q, q, w, w, eps=eps)
    assert (y == 0).all() and all((v == 0).all() for v in got.values())

"""The quantiser's quotients in three instructions against plain division, for
every significand of a block's largest value: the scale amax / 448 rounded to
binary32, and values on and beside the midpoints of neighbouring codes times
the scale, where a quotient off by one step changes the code.

The divisions are done in 64 bits and rounded to 24: a quotient of two 24-bit
numbers that is rounded to 53 bits first rounds to the same 24 bits (53 >= 2 *
24 + 2)."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
from gpu_util import device

pytestmark = pytest.mark.gpu

SLICE = 1 << 17


def codes_of(v, s):
    return (v.double() / s.double()[:, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


# the ends of the range that takes three instructions, the middle, and a block
# on each side that divides
@pytest.mark.parametrize("exponent", [-81, -80, -1, 0, 8, 89, 90, 110])
def test_every_significand(exponent):
    dev = device()
    c = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = ((c[:-1] + c[1:]) / 2).to(dev)
    col = torch.arange(126, device=dev)
    way = torch.tensor([0.0, float("inf"), 0.0], device=dev)
    for at in range(0, 1 << 23, SLICE):
        sig = torch.arange(at, at + SLICE, device=dev)
        amax = (sig | 127 << 23).to(torch.int32).view(torch.float32) * 2.0 ** exponent
        s = (amax.double() / 448).float()
        v = torch.empty(SLICE, 128, device=dev)
        v[:, :126] = mid * s[:, None]
        turn = (sig[:, None] + col) % 3
        beside = torch.nextafter(v[:, :126], way[turn])
        v[:, :126] = torch.where(turn < 2, beside, v[:, :126])
        v[:, 126], v[:, 127] = -v[:, 63], amax
        q, got, _, _ = gl.quant_e4m3_2d(v, transposed=False)
        assert torch.equal(got[:, 0], s), at
        assert torch.equal(q, codes_of(v, s)), at
        if at == 0:              # the card's own 64-bit divisions
            n = slice(0, 4096)
            assert torch.equal(q[n].cpu(), codes_of(v[n].cpu(), s[n].cpu()))

"""Scores of tokens and their gradient under caps above the logits, where z is near
l.  Tolerances are test_gpu_score_far's: past a cap of 66 a z is off by 20 u of
itself."""
import math

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
from gpu_util import device
from test_gpu_score_far import BF16, F32, U, check_gradient, parts

pytestmark = pytest.mark.gpu


CAPS = [(80.0, 1.0, 0.0), (1e3, 1.0, 0.0), (1e4, 1.0, 0.0), (1e4, 1.0, 8e3), (30.0, 3.0, 0.0), (400.0, 1.0, -390.0)]


def make(T, V, softcap, offset, dtype):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(T, V, generator=g) * 4 + offset).to(dtype)
    x[1, ::2] = -math.inf
    x[2] = (torch.randn(V, generator=g) * 3 * softcap).to(dtype)     # both of its ends
    t = torch.randint(0, V, (T,), generator=g)
    t[1] = 1
    return x, t, torch.randn(T, generator=g), torch.randn(T, generator=g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softcap,scale,offset", CAPS + [(1e30, 1.0, 0.0)])
@pytest.mark.parametrize("T,V", [(64, 1003), (3, 40003), (1100, 260)])
def test_scores(T, V, softcap, scale, offset, dtype):
    dev = device()
    x, t, _, _ = make(T, V, softcap, offset, dtype)
    r = ref.score(x, t, softcap, scale)
    dp, ls, dh = parts(r, softcap, scale)
    for top in (0, 3):
        got = gl.token_logprobs(x.to(dev), t.to(dev), softcap=softcap, scale=scale, top=top)
        room = 20 * U * (r["z"].gather(1, t[:, None])[:, 0].abs()) + dp + ls + 4 * U * r["logprobs"].abs()
        err = (got["logprobs"].cpu().double() - r["logprobs"]).abs()
        assert (err <= room).all(), f"logprobs {(err - room).max():.3e} over, at most {err.max():.3e} off"
        assert ((got["entropy"].cpu().double() - r["entropy"]).abs() <= dh).all()
        assert ((got["lse"].cpu().double() - r["lse"]).abs() <= dp + ls + 4 * U * r["lse"].abs()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softcap,scale,offset", CAPS)
@pytest.mark.parametrize("T,V", [(64, 1003), (3, 40003), (1100, 260)])
def test_gradient(T, V, softcap, scale, offset, dtype):
    dev = device()
    x, t, d_l, d_h = make(T, V, softcap, offset, dtype)
    got = gl.token_logprobs(x.to(dev), t.to(dev), softcap=softcap, scale=scale)
    d = gl.token_logprobs_backward(x.to(dev), got["lse"], got["entropy"], t.to(dev), d_l.to(dev), d_h.to(dev),
                                   softcap=softcap, scale=scale)
    keep = torch.arange(T) != 1
    check_gradient(x[keep], t[keep], d_l[keep], d_h[keep], d[keep.to(dev)], softcap, scale)
    assert (d[1, ::2] == 0).all() and torch.isfinite(d[1]).all()


@pytest.mark.parametrize("V", [50003, 1 << 24])
@pytest.mark.parametrize("softcap", [30.0, 66.0, 66.6, 1e3])
@pytest.mark.parametrize("sign", [1, -1])
def test_rows_at_the_cap(sign, softcap, V):
    # every word at an end of the cap: the largest and the smallest sums there are.  The
    # entropy of a small cap is a difference of its z's average, in which a thread's
    # chain of V / 256 terms (64 at most in pieces) and the joins count
    dev = device()
    x = torch.full((1, V), 1e5 * sign, device=dev)
    got = gl.token_logprobs(x, torch.tensor([V - 1], device=dev), softcap=softcap)
    room = (20 + 64 + 64) * U * (softcap + 20)
    assert abs(got["logprobs"].item() + math.log(V)) <= room and abs(got["entropy"].item() - math.log(V)) <= room
    assert abs(got["lse"].item() - sign * softcap - math.log(V)) <= room

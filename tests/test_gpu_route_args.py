"""Shapes of bias and logits that beam_moe_route's binding takes: their values
are read in order, so any shape of the right size, and a longer buffer for
logits that are written."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
from gpu_util import device
from synth import WORKLOADS, make_inputs, small_shape

pytestmark = pytest.mark.gpu


def setup():
    sh = small_shape()
    inp = make_inputs(WORKLOADS["prefill4k"], device=device(), tokens=23, shape=sh, seed=3)
    bias = torch.linspace(-0.05, 0.05, sh.n_experts, device=device())[torch.randperm(
        sh.n_experts, generator=torch.Generator().manual_seed(1)).to(device())].contiguous()
    return sh, inp, bias, gl.make_desc(sh, gl.BF16, gl.BF16)


def test_bias_and_logits_of_other_shapes():
    sh, inp, bias, d = setup()
    E, G = sh.n_experts, sh.n_groups
    want = gl.route(d, inp.x, inp.w_router, bias)
    for b in (bias[None], bias.view(G, E // G), bias.view(E, 1)):
        got = gl.route(d, inp.x, inp.w_router, b)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        lin = gl.with_flags(d, gl.ROUTE_LOGITS_IN)
        for lg in (want[2], want[2].view(-1, G, E // G), want[2][:, None]):
            got = gl.route(lin, None, None, b, lg)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] is lg


def test_preallocated_logits():
    sh, inp, bias, d = setup()
    want = gl.route(d, inp.x, inp.w_router, bias)
    for T in (23, 24, 64):
        room = torch.full((T, sh.n_experts), 7.0, device=device())
        idx, w, lg = gl.route(d, inp.x, inp.w_router, bias, logits=room)
        assert lg is room and torch.equal(idx, want[0]) and torch.equal(w, want[1])
        assert torch.equal(room[:23], want[2]) and (room[23:] == 7).all()


def test_refusals():
    sh, inp, bias, d = setup()
    E = sh.n_experts
    lin = gl.with_flags(d, gl.ROUTE_LOGITS_IN)
    lg = torch.zeros(23, E, device=device())
    for bad in (bias[:-1], torch.zeros(E + 1, device=device()), bias.double(), bias.cpu(), bias.bfloat16(),
                torch.zeros(2 * E, device=device())[::2]):
        with pytest.raises(ValueError, match="bias"):
            gl.route(lin, None, None, bad, lg)
    # given logits of more columns would be read as other rows
    for bad in (torch.zeros(23, 2 * E, device=device()), lg[:, :-1], lg.bfloat16()):
        with pytest.raises(ValueError, match="logits"):
            gl.route(lin, None, None, bias, bad)
    for bad in (torch.zeros(22, E, device=device()), torch.zeros(23, E, device=device(), dtype=torch.int32)):
        with pytest.raises(ValueError, match="logits"):
            gl.route(d, inp.x, inp.w_router, bias, logits=bad)

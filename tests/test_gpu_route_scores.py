"""Routing by softmax scores and unnormalised weights, and the gradient of the
routing weights, on the GPU against the 64-bit formulas.

Indices are equal: the selection compares binary32 scores that both sides
round from 64 bits.  A weight is off by at most its roundings: the score's, K
of the sum, the quotient's and the scale's, (K + 3) 2^-24 relative.

The gradient's factors: a score recomputed in binary32 is off by the rounding
of l - max (|l - max| 2^-24 in the exponent), the exponential's and quotient's
(under 6 half steps together) and the sum's (E/64 + 6 roundings); the sums
over K add K roundings.  With kappa the sum of these, doubled, a gradient is
off by at most kappa 2^-24 scale s (|dw| + sum |dw s|) with s the score or the
normalised score."""
import math

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import layer_ref as ref
from gpu_util import device
from synth import Shape

pytestmark = pytest.mark.gpu

# experts, groups, kept, top, top-n of the group score
SHAPES = [(256, 8, 4, 8, 2), (256, 8, 8, 8, 2), (39, 1, 1, 13, 2), (16, 4, 2, 4, 1),
          (1024, 16, 5, 16, 2), (78, 2, 2, 1, 2), (10, 10, 7, 7, 1), (130, 5, 3, 9, 2), (64, 1, 1, 16, 2)]


def desc(shape, softmax, normed, scale=2.5):
    e, g, tg, k, topn = shape
    sh = Shape(hidden=128, intermediate=128, n_experts=e, n_groups=g, topk_groups=tg, top_k=k,
               group_score_topn=topn, routed_scale=scale)
    flags = gl.ROUTE_LOGITS_IN | (gl.ROUTE_SOFTMAX if softmax else 0) | (0 if normed else gl.ROUTE_UNNORMED)
    return gl.make_desc(sh, gl.BF16, gl.BF16, flags)


def make(T, E, softmax, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(T, E, generator=g) * spread
    bias = (torch.rand(E, generator=g) * 2 - 1) * (0.5 / E if softmax else 0.02)
    return logits, bias


def check(shape, logits, bias, softmax, normed, seed=0):
    e, g, tg, k, topn = shape
    T = logits.shape[0]
    dev = device()
    d = desc(shape, softmax, normed)
    lg = logits.to(dev)
    idx, w, _ = gl.route(d, None, None, None if bias is None else bias.to(dev), lg)
    want = ref.select(logits, bias, g, tg, k, topn, softmax)
    assert torch.equal(idx.cpu(), want)
    ww = ref.weights(logits, want, 2.5, softmax, normed)
    err = (w.cpu().double() - ww).abs()
    # scores below the smallest normal binary32 value have a step of 2^-149
    s = ref.scores(logits, softmax).gather(1, want.long())
    den = s.sum(1, keepdim=True) if normed else torch.ones(T, 1, dtype=ref.F64)
    tiny = 2.5 * (k + 1) * 2.0 ** -149 / den.clamp_min(2.0 ** -148)
    assert (err <= (k + 3) * ref.U * ww + tiny).all(), (err / ww).max()

    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(seed + 1))
    got = gl.route_backward(d, lg, idx, dw.to(dev)).cpu().double()
    exact = ref.route_grad(logits, want, dw, 2.5, softmax, normed)
    assert (((got - exact).abs()) <= grad_bound(logits, want, dw, softmax, normed)).all(), \
        (got - exact).abs().max()
    return idx, w, got


def grad_bound(logits, idx, dw, softmax, normed, scale=2.5):
    T, E = logits.shape
    k = idx.shape[1]
    fin = logits.clamp(-200, 200)
    reach = (fin.amax(1, keepdim=True) - fin.gather(1, idx.long())) if softmax else fin.gather(1, idx.long()).abs()
    kappa = 2 * (reach.amax(1, keepdim=True).double() + 6 + E / 64 + 6 + 2 * k + 4)
    s_all = ref.scores(logits, softmax)
    s = s_all.gather(1, idx.long())
    if normed:
        q = s / s.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        q = s
    tot = (dw.double().abs() * q).sum(1, keepdim=True)
    per = q * (dw.double().abs() + tot)
    out = s_all * tot if (softmax and not normed) else torch.zeros(T, E, dtype=ref.F64)
    if softmax and not normed:
        kappa = 2 * (40 + 6 + E / 64 + 6 + 2 * k + 4)
    out = out.scatter_add(1, idx.long(), per)
    return scale * kappa * ref.U * out + 2.0 ** -120


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("softmax,normed", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T", [1, 7, 133])
def test_route_and_gradient(shape, softmax, normed, T):
    logits, bias = make(T, shape[0], softmax, 100 + T + shape[0])
    check(shape, logits, bias, softmax, normed)


@pytest.mark.parametrize("softmax,normed", [(True, True), (True, False), (False, True), (False, False)])
def test_no_bias_and_wide_logits(softmax, normed):
    logits, _ = make(40, 256, softmax, 7, spread=6.0)
    check((256, 8, 4, 8, 2), logits, None, softmax, normed)


@pytest.mark.parametrize("softmax", [True, False])
def test_ties_go_to_the_lower_index(softmax):
    logits = torch.zeros(5, 64)
    logits[1] = torch.arange(64) // 8 * 0.5          # groups of equal experts
    logits[2, 32:] = 1.0                              # equal groups
    logits[3] = -3.0
    logits[4, ::2] = 2.0
    check((64, 8, 4, 8, 2), logits, None, softmax, True)


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("normed", [True, False])
def test_masked_experts_and_rows(softmax, normed):
    # masked with -infinity or binary32's lowest value: some experts, all but
    # fewer than K of them, and whole rows
    g = torch.Generator().manual_seed(3)
    logits = torch.randn(9, 64, generator=g)
    low = torch.finfo(torch.float32).min
    logits[0, 5:] = -math.inf
    logits[1, 5:] = low
    logits[2] = -math.inf
    logits[3] = low
    logits[4, ::3] = -math.inf
    logits[5, 8:16] = low
    logits[6, 1:] = -math.inf
    logits[7] = -200.0
    logits[7, 3] = 0.0
    shape = (64, 8, 8, 8, 2)
    dev = device()
    d = desc(shape, softmax, normed)
    idx, w, _ = gl.route(d, None, None, None, logits.to(dev))
    want = ref.select(logits, None, 8, 8, 8, 2, softmax)
    assert torch.equal(idx.cpu(), want)
    ww = ref.weights(logits, want, 2.5, softmax, normed)
    # the scores themselves round to 0 below 2^-150
    assert ((w.cpu().double() - ww).abs() <= 11 * ref.U * ww + 2.0 ** -140).all()
    dw = torch.randn(9, 8, generator=g)
    got = gl.route_backward(d, logits.to(dev), idx, dw.to(dev)).cpu().double()
    exact = ref.route_grad(logits, want, dw, 2.5, softmax, normed)
    assert torch.isfinite(got).all()
    assert ((got - exact).abs() <= grad_bound(logits, want, dw, softmax, normed)).all()
    full = softmax and not normed        # a row of equal lowest logits is no masked row for a softmax
    assert (got[2] == 0).all() and (w[2].cpu() == 0).all()
    if not softmax:
        assert (w[3].cpu() == 0).all() and (got[3] == 0).all()
    assert full or (got[6] == 0).all() or not normed


def test_gradient_against_differences():
    # d/dl of sum dw w(l) with the selection held, by central differences of
    # the 64-bit forward: error of a difference h^2 f''' / 6 + 1e-16 / h
    h = 1e-5
    for softmax in (True, False):
        for normed in (True, False):
            logits, bias = make(3, 32, softmax, 50)
            shape = (32, 4, 2, 4, 2)
            d = desc(shape, softmax, normed)
            dev = device()
            idx, _, _ = gl.route(d, None, None, bias.to(dev), logits.to(dev))
            dw = torch.randn(3, 4, generator=torch.Generator().manual_seed(9))
            got = gl.route_backward(d, logits.to(dev), idx, dw.to(dev)).cpu().double()
            x = logits.double()
            for e in range(32):
                up, dn = x.clone(), x.clone()
                up[:, e] += h
                dn[:, e] -= h
                f = [(ref.weights(v, idx.cpu(), 2.5, softmax, normed) * dw).sum(1) for v in (up, dn)]
                diff = (f[0] - f[1]) / (2 * h)
                assert ((got[:, e] - diff).abs() <= 1e-5).all(), (softmax, normed, e)


def test_gradient_of_foreign_indices():
    # ids outside the experts add nothing, an id named twice counts twice
    logits, _ = make(4, 48, True, 12)
    idx = torch.tensor([[0, -1, 7, 48], [5, 5, 9, 1], [-5, -1, 100, 2**31 - 1], [3, 3, 3, 3]], dtype=torch.int32)
    dw = torch.randn(4, 4, generator=torch.Generator().manual_seed(2))
    dev = device()
    for softmax in (True, False):
        for normed in (True, False):
            d = desc((48, 4, 4, 4, 2), softmax, normed)
            got = gl.route_backward(d, logits.to(dev), idx.to(dev), dw.to(dev)).cpu().double()
            exact = ref.route_grad(logits, idx, dw, 2.5, softmax, normed)
            assert ((got - exact).abs() <= 100 * ref.U * 2.5 * 4).all()


@pytest.mark.parametrize("softmax", [True, False])
def test_long_batch_equals_its_rows(softmax):
    # the largest batch the boundary takes at these widths, against a slice
    shape = (256, 8, 8, 8, 2)
    T = 52001
    logits, bias = make(T, 256, softmax, 5)
    dev = device()
    d = desc(shape, softmax, False)
    lg, b = logits.to(dev), bias.to(dev)
    idx, w, _ = gl.route(d, None, None, b, lg)
    dw = torch.randn(T, 8, device=dev)
    g = gl.route_backward(d, lg, idx, dw)
    rows = slice(T - 37, T)
    i2, w2, _ = gl.route(d, None, None, b, lg[rows].contiguous())
    g2 = gl.route_backward(d, lg[rows].contiguous(), i2, dw[rows].contiguous())
    assert torch.equal(idx[rows], i2) and torch.equal(w[rows], w2) and torch.equal(g[rows], g2)
    assert torch.equal(idx[rows].cpu(), ref.select(logits[rows], bias, 8, 8, 8, 2, softmax))


def test_softmax_routes_the_whole_block():
    # logits computed from x inside the block, then the same routing
    import numpy as np
    import oracle
    from gpu_util import max_rel_err
    from synth import WORKLOADS, make_inputs, small_shape
    sh = small_shape()
    inp = make_inputs(WORKLOADS["prefill4k"], device=device(), tokens=60, shape=sh, seed=4)
    d = gl.make_desc(sh, gl.BF16, gl.BF16, gl.ROUTE_SOFTMAX | gl.ROUTE_UNNORMED)
    out, idx, w, lg = gl.forward(d, inp.x, inp.w_router, inp.bias, inp.w_gate_up, inp.w_down,
                                 return_routing=True)
    i2, w2, _ = gl.route(gl.with_flags(d, d.flags | gl.ROUTE_LOGITS_IN), None, None, inp.bias, lg)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    assert torch.equal(idx.cpu(), ref.select(lg.cpu(), inp.bias.cpu(), 8, 4, 8, 2, True))
    want = oracle.forward_tokens(sh, np.arange(60), inp.x.cpu(), idx.cpu().numpy(), w.cpu().numpy(),
                                 inp.w_gate_up.cpu(), inp.w_down.cpu())
    assert max_rel_err(out.float().cpu().numpy(), want) <= 2e-2      # the bf16 block's bar


def test_captured_and_on_another_stream():
    shape = (256, 8, 4, 8, 2)
    dev = device()
    d = desc(shape, True, True)
    logits, bias = make(300, 256, True, 8)
    lg, b, dw = logits.to(dev), bias.to(dev), torch.randn(300, 8, device=dev)
    idx, w, _ = gl.route(d, None, None, b, lg)
    g = gl.route_backward(d, lg, idx, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    i2, w2, _ = gl.route(d, None, None, b, lg, stream=side)
    g2 = gl.route_backward(d, lg, i2, dw, stream=side)
    side.synchronize()
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(g, g2)
    graph = torch.cuda.CUDAGraph()
    src = lg.clone()
    with torch.cuda.graph(graph):
        i3, w3, _ = gl.route(d, None, None, b, src)
        g3 = gl.route_backward(d, src, i3, dw)
    for _ in range(3):
        src.copy_(lg.flip(0))
        graph.replay()
        src.copy_(lg)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, i3) and torch.equal(w, w3) and torch.equal(g, g3)

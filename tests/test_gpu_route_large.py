"""Routing of batches past what the expert path holds, with the layer's own
descriptor, against the same rows alone."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import layer_ref as ref
from gpu_util import device
from synth import BEAM

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("flags", [0, gl.ROUTE_SOFTMAX | gl.ROUTE_UNNORMED])
@pytest.mark.parametrize("T", [52429, 65536, 8400003])       # the last: offsets past 2^31 elements
def test_training_batch(T, flags):
    dev = device()
    E, K = BEAM.n_experts, BEAM.top_k
    d = gl.make_desc(BEAM, gl.BF16, gl.BF16, flags | gl.ROUTE_LOGITS_IN)
    g = torch.Generator(device=dev).manual_seed(T)
    logits = torch.randn(T, E, generator=g, device=dev)
    bias = (torch.rand(E, generator=g, device=dev) - 0.5) / E
    dw = torch.randn(T, K, generator=g, device=dev)
    idx, w, _ = gl.route(d, None, None, bias, logits)
    grad = gl.route_backward(d, logits, idx, dw)
    for rows in (slice(0, 40), slice(T // 2, T // 2 + 40), slice(T - 37, T)):
        lg = logits[rows].contiguous()
        i2, w2, _ = gl.route(d, None, None, bias, lg)
        g2 = gl.route_backward(d, lg, i2, dw[rows].contiguous())
        assert torch.equal(idx[rows], i2) and torch.equal(w[rows], w2) and torch.equal(grad[rows], g2)
    want = ref.select(logits[-37:].cpu(), bias.cpu(), BEAM.n_groups, BEAM.topk_groups, K, 2, bool(flags))
    assert torch.equal(idx[-37:].cpu(), want)

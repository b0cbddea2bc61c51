"""Token counts that the routing entry points take: with given logits, and for
the gradient, no slots are held, so the layer's widths do not bound the batch.
Refusals come back before any GPU work, so these run without a GPU; a batch
within the bounds is told by the next check failing instead (null tensors)."""
import ctypes

import pytest

import group_limited_routing_sigmoid_amd as gl
from synth import BEAM

MOST = 4 * (2 ** 24 - 1)        # one wave of 64 a token, four a workgroup, fewer than 2^32 threads
NULLS = (None,) * 7


def route(T, flags, **kw):
    d = gl.make_desc(BEAM, gl.BF16, gl.BF16, flags)
    for k, v in kw.items():
        setattr(d, k, v)
    return gl.lib().beam_moe_route(ctypes.byref(d), T, *NULLS, 0, None)


def backward(T, flags=0, **kw):
    d = gl.make_desc(BEAM, gl.BF16, gl.BF16, flags)
    for k, v in kw.items():
        setattr(d, k, v)
    return gl.lib().beam_moe_route_backward(ctypes.byref(d), T, *(None,) * 5)


@pytest.mark.parametrize("T", [1, 52428, 52429, 65536, 1 << 20, MOST])
def test_layer_widths_do_not_bound_given_logits(T):
    assert route(T, gl.ROUTE_LOGITS_IN) == gl.ERR_INVALID_ARG
    assert route(T, gl.ROUTE_LOGITS_IN | gl.ROUTE_SOFTMAX | gl.ROUTE_UNNORMED) == gl.ERR_INVALID_ARG
    assert backward(T) == gl.ERR_INVALID_ARG
    assert backward(T, gl.ROUTE_SOFTMAX) == gl.ERR_INVALID_ARG


@pytest.mark.parametrize("T", [MOST + 1, 1 << 32, 1 << 62])
def test_more_tokens_than_a_launch_holds(T):
    assert route(T, gl.ROUTE_LOGITS_IN) == gl.ERR_UNSUPPORTED
    assert backward(T) == gl.ERR_UNSUPPORTED
    assert gl.validate(gl.make_desc(BEAM, gl.BF16, gl.BF16), T) == gl.ERR_UNSUPPORTED


def test_what_holds_slots_keeps_its_bound():
    d = gl.make_desc(BEAM, gl.BF16, gl.BF16)
    assert gl.validate(d, 52428) == gl.OK and gl.validate(d, 52429) == gl.ERR_UNSUPPORTED
    assert gl.validate(gl.with_flags(d, gl.ROUTE_LOGITS_IN), 52429) == gl.ERR_UNSUPPORTED
    assert route(52429, 0) == gl.ERR_UNSUPPORTED            # its logits' partial sums are in the workspace


@pytest.mark.parametrize("kw,status", [
    (dict(top_k=17), gl.ERR_UNSUPPORTED), (dict(n_experts=2048), gl.ERR_UNSUPPORTED), (dict(hidden=100), gl.ERR_UNSUPPORTED),
    (dict(routed_scale=0.0), gl.ERR_INVALID_ARG), (dict(flags=1 << 9), gl.ERR_INVALID_ARG)])
def test_fields_are_still_checked(kw, status):
    assert backward(1 << 20, **kw) == status
    if "flags" not in kw:
        assert route(1 << 20, gl.ROUTE_LOGITS_IN, **kw) == status

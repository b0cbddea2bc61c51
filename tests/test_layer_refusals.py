"""Host-side refusals of the operators around the expert block: bad arguments
come back as errors before any GPU work, so these run without a GPU."""
import ctypes

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
from synth import BEAM

GOOD, BAD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


def _desc(flags=0, **kw):
    d = gl.make_desc(BEAM, gl.BF16, gl.BF16, flags)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_score_flags_are_known():
    for f in (gl.ROUTE_SOFTMAX, gl.ROUTE_UNNORMED, gl.ROUTE_SOFTMAX | gl.ROUTE_UNNORMED | gl.ROUTE_LOGITS_IN):
        assert gl.validate(_desc(f), 64) == gl.OK


def test_route_backward_refuses():
    fn = gl.lib().beam_moe_route_backward
    d = _desc()
    ok = [GOOD] * 4
    assert fn(ctypes.byref(d), 0, None, None, None, None, None) == gl.OK
    assert fn(ctypes.byref(d), -1, *ok, None) == gl.ERR_INVALID_ARG
    assert fn(None, 4, *ok, None) == gl.ERR_INVALID_ARG
    for i in range(4):
        for bad in (None, BAD):
            args = list(ok)
            args[i] = bad
            assert fn(ctypes.byref(d), 4, *args, None) == gl.ERR_INVALID_ARG
    assert fn(ctypes.byref(_desc(top_k=17)), 4, *ok, None) == gl.ERR_UNSUPPORTED


def test_binding_checks_tensors_first():
    with pytest.raises(ValueError, match="GPU"):
        gl.route_backward(_desc(), torch.zeros(2, 256), torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 8),
                          out=torch.zeros(2, 256))

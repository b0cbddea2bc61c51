"""An eps below binary32's normal numbers has no inverse root in it, so that a head
of zeros would be NaN: refused before any GPU work."""
import pytest

import group_limited_routing_sigmoid_amd as gl
from test_serve_refusals import UNSUPPORTED, _rope, _rope_grad


@pytest.mark.parametrize("eps,status", [(1e-45, UNSUPPORTED), (1e-40, UNSUPPORTED), (1.17e-38, UNSUPPORTED),
                                        (1.18e-38, gl.OK), (1e-6, gl.OK)])
def test_head_norms_need_a_normal_eps(eps, status):
    assert _rope(T=0, eps=eps) == status
    if status != gl.OK:
        assert _rope_grad(T=0, eps=eps) == status
    else:      # past eps, the workspace comes next
        assert _rope_grad(eps=eps, ws=None) == gl.ERR_WORKSPACE

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


def _norm(**kw):
    a = dict(T=4, H=256, dtype=gl.BF16, o=GOOD, post=GOOD, gate=GOOD, cols=256, pre=GOOD, eps=1e-6, alpha=1.0,
             beta=1.0, res=GOOD, res_out=GOOD, x=GOOD, q=None, s=None)
    a.update(kw)
    return gl.lib().beam_moe_norm_residual(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), gl.ERR_INVALID_ARG), (dict(H=0), gl.ERR_INVALID_ARG), (dict(H=16385, cols=1), gl.ERR_UNSUPPORTED),
    (dict(dtype=gl.FP8_E4M3), gl.ERR_INVALID_ARG), (dict(eps=0.0), gl.ERR_INVALID_ARG),
    (dict(eps=-1.0), gl.ERR_INVALID_ARG), (dict(eps=float("nan")), gl.ERR_INVALID_ARG),
    (dict(alpha=float("inf")), gl.ERR_INVALID_ARG), (dict(beta=float("nan")), gl.ERR_INVALID_ARG),
    (dict(cols=2), gl.ERR_INVALID_ARG), (dict(cols=0), gl.ERR_INVALID_ARG),
    (dict(gate=None), gl.ERR_INVALID_ARG), (dict(o=None), gl.ERR_INVALID_ARG),
    (dict(post=None), gl.ERR_INVALID_ARG), (dict(res=None), gl.ERR_INVALID_ARG),
    (dict(res_out=None), gl.ERR_INVALID_ARG), (dict(x=None), gl.ERR_INVALID_ARG),
    (dict(pre=None), gl.ERR_INVALID_ARG), (dict(o=None, gate=None, cols=0, pre=None, x=None), gl.ERR_INVALID_ARG),
    (dict(q=GOOD), gl.ERR_INVALID_ARG), (dict(s=GOOD), gl.ERR_INVALID_ARG),
    (dict(H=200, cols=1, q=GOOD, s=GOOD), gl.ERR_UNSUPPORTED),
    (dict(o=BAD), gl.ERR_INVALID_ARG), (dict(gate=BAD), gl.ERR_INVALID_ARG), (dict(res=BAD), gl.ERR_INVALID_ARG),
    (dict(x=BAD), gl.ERR_INVALID_ARG), (dict(T=0, o=None, gate=None, res=None), gl.OK),
])
def test_norm_refuses(kw, status):
    assert _norm(**kw) == status


def _norm_grad(**kw):
    a = dict(T=4, H=256, dtype=gl.BF16, o=GOOD, post=GOOD, gate=GOOD, cols=1, pre=GOOD, eps=1e-6, alpha=1.0,
             beta=1.0, r=GOOD, d_r=GOOD, d_x=GOOD, d_res=GOOD, d_o=GOOD, d_gate=GOOD, d_pre=GOOD, d_post=GOOD,
             ws=GOOD, n=1 << 30)
    a.update(kw)
    return gl.lib().beam_moe_norm_residual_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), gl.ERR_INVALID_ARG), (dict(H=20000), gl.ERR_UNSUPPORTED), (dict(eps=0.0), gl.ERR_INVALID_ARG),
    (dict(cols=3), gl.ERR_INVALID_ARG), (dict(r=None), gl.ERR_INVALID_ARG),
    (dict(d_r=None, d_x=None), gl.ERR_INVALID_ARG), (dict(pre=None), gl.ERR_INVALID_ARG),
    (dict(d_pre=None), gl.ERR_INVALID_ARG), (dict(d_o=None), gl.ERR_INVALID_ARG),
    (dict(d_post=None), gl.ERR_INVALID_ARG), (dict(d_gate=None), gl.ERR_INVALID_ARG),
    (dict(d_res=None), gl.ERR_INVALID_ARG), (dict(ws=None), gl.ERR_WORKSPACE), (dict(n=100), gl.ERR_WORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10010)), gl.ERR_INVALID_ARG), (dict(d_x=BAD), gl.ERR_INVALID_ARG),
])
def test_norm_gradient_refuses(kw, status):
    assert _norm_grad(**kw) == status


def test_norm_binding_checks():
    f, r = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        gl.norm_residual(f, pre_weight=r)
    with pytest.raises(ValueError, match=r"\[T, H\]"):
        gl.norm_residual(torch.zeros(8), pre_weight=r)
    with pytest.raises(ValueError, match="belong to o"):
        gl.norm_residual(f, post_weight=r, pre_weight=r)
    with pytest.raises(ValueError, match="share one dtype"):
        gl.norm_residual(f, o=f, post_weight=r, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected torch.bfloat16"):
        gl.norm_residual(f, pre_weight=r, dtype=torch.float16)
    with pytest.raises(ValueError, match="post_weight"):
        gl.norm_residual(f, o=f)
    with pytest.raises(ValueError, match="pre_weight is needed"):
        gl.norm_residual_e4m3(f, o=f, post_weight=r)
    with pytest.raises(ValueError, match="one of"):
        gl.norm_residual_backward(f)
    with pytest.raises(ValueError):
        gl.residual_scale(0)


def _mm(**kw):
    a = dict(M=4, N=8, K=256, a=GOOD, sa=GOOD, sa_r=2, sa_k=1, b=GOOD, sb=GOOD, sb_r=2, sb_k=1, rows=0,
             dtype=gl.BF16, y=GOOD)
    a.update(kw)
    return gl.lib().beam_moe_matmul_e4m3(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), gl.ERR_INVALID_ARG), (dict(N=-1), gl.ERR_INVALID_ARG), (dict(K=-128), gl.ERR_INVALID_ARG),
    (dict(K=100), gl.ERR_UNSUPPORTED), (dict(K=1 << 23), gl.ERR_UNSUPPORTED), (dict(M=1 << 23), gl.ERR_UNSUPPORTED),
    (dict(N=1 << 40), gl.ERR_UNSUPPORTED), (dict(M=1 << 22, N=1 << 17), gl.ERR_UNSUPPORTED), (dict(rows=2), gl.ERR_INVALID_ARG),
    (dict(dtype=gl.FP8_E4M3), gl.ERR_INVALID_ARG), (dict(a=None), gl.ERR_INVALID_ARG),
    (dict(sa=None), gl.ERR_INVALID_ARG), (dict(b=None), gl.ERR_INVALID_ARG), (dict(sb=None), gl.ERR_INVALID_ARG),
    (dict(y=None), gl.ERR_INVALID_ARG), (dict(a=BAD), gl.ERR_INVALID_ARG), (dict(sb=BAD), gl.ERR_INVALID_ARG),
    (dict(y=BAD), gl.ERR_INVALID_ARG), (dict(sa_r=-1), gl.ERR_INVALID_ARG), (dict(sb_k=-4), gl.ERR_INVALID_ARG),
    (dict(M=0, a=None, sa=None, y=None), gl.OK), (dict(N=0, b=None), gl.OK),
])
def test_matmul_refuses(kw, status):
    assert _mm(**kw) == status


def _q2(**kw):
    a = dict(rows=4, cols=8, dtype=gl.BF16, block=0, v=GOOD, q=GOOD, s=GOOD, qt=GOOD, st=GOOD)
    a.update(kw)
    return gl.lib().beam_moe_quant_e4m3_2d(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), gl.ERR_INVALID_ARG), (dict(cols=-1), gl.ERR_INVALID_ARG), (dict(dtype=7), gl.ERR_INVALID_ARG),
    (dict(block=3), gl.ERR_INVALID_ARG), (dict(rows=1 << 40), gl.ERR_UNSUPPORTED), (dict(v=None), gl.ERR_INVALID_ARG),
    (dict(q=None), gl.ERR_INVALID_ARG), (dict(st=None), gl.ERR_INVALID_ARG),
    (dict(q=None, s=None, qt=None, st=None), gl.ERR_INVALID_ARG), (dict(qt=BAD), gl.ERR_INVALID_ARG),
    (dict(rows=0, v=None), gl.OK), (dict(cols=0, v=None), gl.OK),
])
def test_quant_2d_refuses(kw, status):
    assert _q2(**kw) == status


def test_matmul_binding_checks():
    a, s = torch.zeros(2, 128, dtype=torch.uint8), torch.ones(2, 1)
    with pytest.raises(ValueError, match="GPU"):
        gl.matmul_e4m3(a, s, a, s)
    with pytest.raises(ValueError, match="multiple of 128"):
        gl.matmul_e4m3(a[:, :100], s, a[:, :100], s)
    with pytest.raises(ValueError, match="expected torch.bfloat16"):
        gl.matmul_e4m3(a, s, a, s, dtype=torch.float16)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        gl.matmul_e4m3(a[0], s, a, s)
    with pytest.raises(ValueError, match="GPU"):
        gl.quant_e4m3_2d(torch.zeros(2, 3))


def test_gradient_of_nothing_is_refused():
    # without a block output and without x's gradient no kernel has work
    assert _norm_grad(o=None, post=None, gate=None, cols=0, d_x=None, pre=None) == gl.ERR_INVALID_ARG
    assert _norm_grad(o=None, post=None, gate=None, cols=0, d_x=None) == gl.ERR_INVALID_ARG
    f = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="d_x is needed"):
        gl.norm_residual_backward(f, d_residual_out=f, pre_weight=torch.zeros(8))


@pytest.mark.parametrize("H,threads", [(1, 64), (128, 64), (5120, 640), (16384, 1024), (16383, 1024), (4099, 576)])
def test_more_tokens_than_a_launch_holds(H, threads):
    # fewer than 2^32 threads a launch
    most = (2 ** 32 - 1) // threads
    n = ctypes.c_size_t()
    fn = gl.lib().beam_moe_norm_residual_workspace_bytes
    assert fn(most, H, ctypes.byref(n)) == gl.OK and n.value > 0 and n.value % (2 * H * 4) == 0
    assert fn(most + 1, H, ctypes.byref(n)) == gl.ERR_UNSUPPORTED
    assert _norm(T=most + 1, H=H, cols=1) == gl.ERR_UNSUPPORTED
    assert _norm_grad(T=most + 1, H=H) == gl.ERR_UNSUPPORTED


def test_more_tiles_than_a_launch_holds():
    assert _q2(rows=128 * 2 ** 23, cols=1) == gl.ERR_UNSUPPORTED
    assert _q2(rows=2 ** 20, cols=128 * 2 ** 10) == gl.ERR_UNSUPPORTED

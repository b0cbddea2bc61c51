"""Host-side refusals of the operators around a paged cache: bad arguments come
back as errors before any GPU work, so these run without a GPU."""
import ctypes

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl

GOOD, BAD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
NAN, INF = float("nan"), float("inf")
INVALID, UNSUPPORTED = gl.ERR_INVALID_ARG, gl.ERR_UNSUPPORTED


def _rope(**kw):
    a = dict(T=4, Hq=4, Hkv=2, D=128, dtype=gl.BF16, q=GOOD, q_s=1024, k=GOOD, k_s=1024, v=GOOD, v_s=1024, wq=GOOD,
             wk=GOOD, eps=1e-6, pos=GOOD, freq=GOOD, rot=128, inter=0, t_len=0.0, t_exp=0.0, q_out=GOOD, k_out=GOOD,
             kc=GOOD, vc=GOOD, ps=4096, ts=256, hs=128, pages=8, size=16, tables=GOOD, seqs=2, cols=4, rows=GOOD)
    a.update(kw)
    return gl.lib().beam_moe_qk_norm_rope(*a.values(), None)


ROPE_SHAPES = [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(dtype=2), INVALID),
    (dict(D=0), UNSUPPORTED), (dict(D=264), UNSUPPORTED), (dict(D=100), UNSUPPORTED), (dict(Hq=4097), UNSUPPORTED),
    (dict(Hkv=5000), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(rot=144), INVALID), (dict(rot=8), UNSUPPORTED),
    (dict(inter=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(t_len=-1.0), INVALID), (dict(t_len=NAN), INVALID), (dict(t_len=1.0, t_exp=INF), INVALID),
    (dict(T=1 << 25), UNSUPPORTED), (dict(T=1 << 24, Hq=300), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(wq=None), INVALID), (dict(wk=None), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(q=BAD), INVALID), (dict(k=BAD), INVALID), (dict(q_s=1021), INVALID), (dict(k_s=-8), INVALID),
    (dict(q_s=1020), INVALID)]


@pytest.mark.parametrize("kw,status", ROPE_SHAPES + [
    (dict(q_out=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(v=None), INVALID),
    (dict(tables=None), INVALID), (dict(kc=None, vc=None, k_out=None), INVALID), (dict(pages=0), INVALID),
    (dict(size=0), UNSUPPORTED), (dict(size=24), UNSUPPORTED), (dict(cols=1 << 28), UNSUPPORTED),
    (dict(pages=1 << 31), UNSUPPORTED), (dict(ps=4100), INVALID), (dict(ts=-256), INVALID), (dict(hs=4), INVALID),
    (dict(seqs=-1), INVALID), (dict(v_s=3), INVALID), (dict(kc=BAD), INVALID), (dict(tables=BAD), INVALID),
    (dict(rows=BAD), INVALID), (dict(T=0, q=None, k=None, pos=None, freq=None), gl.OK)])
def test_rope_refuses(kw, status):
    assert _rope(**kw) == status


def _rope_grad(**kw):
    a = dict(T=4, Hq=4, Hkv=2, D=128, dtype=gl.BF16, dq_out=GOOD, dk_out=GOOD, q=GOOD, q_s=1024, k=GOOD, k_s=1024,
             wq=GOOD, wk=GOOD, eps=1e-6, pos=GOOD, freq=GOOD, rot=128, inter=0, t_len=0.0, t_exp=0.0, dq=GOOD, dk=GOOD,
             dwq=GOOD, dwk=GOOD, ws=GOOD, n=1 << 30)
    a.update(kw)
    return gl.lib().beam_moe_qk_norm_rope_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", ROPE_SHAPES + [
    (dict(dq_out=None), INVALID), (dict(dk_out=BAD), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dwq=None), INVALID), (dict(dwk=None), INVALID), (dict(ws=None), gl.ERR_WORKSPACE), (dict(n=64), gl.ERR_WORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10010)), INVALID)])
def test_rope_gradient_refuses(kw, status):
    assert _rope_grad(**kw) == status


def _attend(**kw):
    a = dict(seqs=2, Hq=4, Hkv=2, D=128, dtype=gl.BF16, q=GOOD, gate=GOOD, kc=GOOD, vc=GOOD, ps=4096, ts=256, hs=128,
             pages=8, size=16, tables=GOOD, cols=4, lengths=GOOD, scale=0.1, window=0, out=GOOD, lse=GOOD, ws=GOOD,
             n=1 << 30)
    a.update(kw)
    return gl.lib().beam_moe_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(seqs=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hq=5), INVALID), (dict(D=12), UNSUPPORTED),
    (dict(D=512), UNSUPPORTED), (dict(dtype=3), INVALID), (dict(q=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(lengths=None), INVALID), (dict(out=None), INVALID), (dict(tables=None), INVALID),
    (dict(q=BAD), INVALID), (dict(gate=BAD), INVALID), (dict(vc=BAD), INVALID), (dict(out=BAD), INVALID),
    (dict(lse=BAD), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID),
    (dict(window=-1), INVALID), (dict(size=12), UNSUPPORTED), (dict(pages=0), INVALID), (dict(cols=1 << 27), UNSUPPORTED),
    (dict(ps=4), INVALID), (dict(ts=-8), INVALID), (dict(hs=129), INVALID), (dict(ws=None), gl.ERR_WORKSPACE),
    (dict(n=1000), gl.ERR_WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), INVALID), (dict(seqs=1 << 22), UNSUPPORTED),
    (dict(seqs=0, q=None, lengths=None, out=None, ws=None, n=0), gl.OK)])
def test_attention_refuses(kw, status):
    assert _attend(**kw) == status


def _pool(count=1, layers=2, base=0x10000, size=256, layer=4096, page=256):
    p = gl.Pools()
    p.count, p.layers = count, layers
    for i in range(min(max(count, 0), 8)):
        p.base[i], p.bytes[i], p.layer_stride[i], p.page_stride[i] = base, size, layer, page
    return p


POOLS = [(dict(count=9), INVALID), (dict(count=-1), INVALID), (dict(layers=-1), INVALID), (dict(base=0), INVALID),
         (dict(base=0x10004), INVALID), (dict(size=100), INVALID), (dict(size=-16), INVALID), (dict(layer=8), INVALID),
         (dict(page=24), INVALID)]


def _update(pool=None, **kw):
    a = dict(old=4, rows=4, cols=8, pages=64, size=16, tables=GOOD, lengths=GOOD, refs=GOOD, parents=GOOD, grow=GOOD,
             t_out=ctypes.c_void_p(0x20000), l_out=ctypes.c_void_p(0x20000), r_out=ctypes.c_void_p(0x20000),
             missing=ctypes.c_void_p(0x20000))
    ws = dict(ws=GOOD, n=1 << 30)
    for k in list(kw):
        (ws if k in ws else a)[k] = kw.pop(k)
    p = pool if pool is not None else _pool()
    return gl.lib().beam_moe_pages_update(*a.values(), ctypes.byref(p), *ws.values(), None)


TABLES = [(dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(pages=-1), INVALID), (dict(rows=65537), UNSUPPORTED),
          (dict(pages=1 << 24), UNSUPPORTED), (dict(size=3), UNSUPPORTED), (dict(cols=1 << 28), UNSUPPORTED),
          (dict(rows=65536, cols=1 << 16, size=1), UNSUPPORTED), (dict(tables=None), INVALID), (dict(lengths=None), INVALID),
          (dict(refs=None), INVALID), (dict(tables=BAD), INVALID), (dict(ws=None), gl.ERR_WORKSPACE),
          (dict(n=256), gl.ERR_WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), INVALID), (dict(r_out=GOOD), INVALID),
          (dict(t_out=None), INVALID), (dict(r_out=None), INVALID)]


@pytest.mark.parametrize("kw,status", TABLES + [
    (dict(old=-1), INVALID), (dict(old=65537), UNSUPPORTED), (dict(parents=None, rows=3), INVALID),
    (dict(l_out=None), INVALID), (dict(missing=None), INVALID), (dict(t_out=GOOD), INVALID), (dict(l_out=GOOD), INVALID),
    (dict(parents=BAD), INVALID), (dict(grow=BAD), INVALID)])
def test_update_refuses(kw, status):
    assert _update(**kw) == status


def _compact(pool=None, **kw):
    a = dict(rows=4, cols=8, pages=64, size=16, tables=GOOD, lengths=GOOD, refs=GOOD, t_out=GOOD,
             r_out=ctypes.c_void_p(0x20000), new_id=GOOD, live=GOOD)
    ws = dict(ws=GOOD, n=1 << 30)
    for k in list(kw):
        (ws if k in ws else a)[k] = kw.pop(k)
    p = pool if pool is not None else _pool()
    return gl.lib().beam_moe_pages_compact(*a.values(), ctypes.byref(p), *ws.values(), None)


@pytest.mark.parametrize("kw,status", TABLES + [(dict(new_id=None), INVALID), (dict(live=None), INVALID),
                                                (dict(new_id=BAD), INVALID)])
def test_compact_refuses(kw, status):
    assert _compact(**kw) == status


@pytest.mark.parametrize("kw,status", POOLS)
def test_pools_refused(kw, status):
    p = _pool(**kw)
    assert _update(pool=p) == status and _compact(pool=p) == status
    assert gl.lib().beam_moe_pages_copy(ctypes.byref(p), 64, 2, GOOD, GOOD, None) == status


def test_copy_refuses():
    fn, p = gl.lib().beam_moe_pages_copy, _pool()
    assert fn(None, 64, 2, GOOD, GOOD, None) == INVALID
    assert fn(ctypes.byref(p), -1, 2, GOOD, GOOD, None) == INVALID
    assert fn(ctypes.byref(p), 64, -2, GOOD, GOOD, None) == INVALID
    assert fn(ctypes.byref(p), 64, 2, None, GOOD, None) == INVALID
    assert fn(ctypes.byref(p), 64, 2, GOOD, BAD, None) == INVALID
    assert fn(ctypes.byref(p), 1 << 31, 2, GOOD, GOOD, None) == UNSUPPORTED
    assert fn(ctypes.byref(p), 64, 0, None, None, None) == gl.OK


def _score(**kw):
    a = dict(T=4, V=100, dtype=gl.BF16, logits=GOOD, stride=100, targets=GOOD, cap=30.0, scale=1.0, top=2, lp=GOOD,
             entropy=GOOD, lse=GOOD, ids=GOOD, tl=GOOD, ws=GOOD, n=1 << 30)
    a.update(kw)
    return gl.lib().beam_moe_token_logprobs(*a.values(), None)


SCORES = [(dict(T=-1), INVALID), (dict(V=0), INVALID), (dict(dtype=2), INVALID), (dict(stride=99), INVALID),
          (dict(cap=-1.0), INVALID), (dict(cap=NAN), INVALID), (dict(cap=INF), INVALID), (dict(scale=0.0), INVALID),
          (dict(scale=INF), INVALID), (dict(V=(1 << 24) + 1, stride=1 << 25), UNSUPPORTED), (dict(T=1 << 23), UNSUPPORTED),
          (dict(T=1 << 22, V=1 << 20, stride=1 << 20), UNSUPPORTED), (dict(logits=None), INVALID), (dict(logits=BAD), INVALID),
          (dict(entropy=None), INVALID), (dict(lse=None), INVALID), (dict(targets=None), INVALID), (dict(targets=BAD), INVALID)]


@pytest.mark.parametrize("kw,status", SCORES + [
    (dict(lp=None), INVALID), (dict(top=-1), INVALID), (dict(top=17), UNSUPPORTED), (dict(V=5, top=6), INVALID),
    (dict(ids=None), INVALID), (dict(tl=None), INVALID), (dict(V=5000, stride=5000, ws=None), gl.ERR_WORKSPACE),
    (dict(V=5000, stride=5000, n=16), gl.ERR_WORKSPACE), (dict(ws=ctypes.c_void_p(0x10010)), INVALID),
    (dict(T=0, logits=None, lse=None), gl.OK)])
def test_score_refuses(kw, status):
    assert _score(**kw) == status


def _score_grad(**kw):
    a = dict(T=4, V=100, dtype=gl.BF16, logits=GOOD, stride=100, targets=GOOD, cap=30.0, scale=1.0, lse=GOOD, entropy=GOOD,
             dl=GOOD, dh=GOOD, out=GOOD, d_stride=100)
    a.update(kw)
    return gl.lib().beam_moe_token_logprobs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", SCORES + [
    (dict(dl=None, dh=None), INVALID), (dict(out=None), INVALID), (dict(d_stride=99), INVALID), (dict(dl=BAD), INVALID),
    (dict(d_stride=104), INVALID), (dict(T=0, logits=None, out=None), gl.OK)])
def test_score_gradient_refuses(kw, status):
    assert _score_grad(**kw) == status


def test_binding_checks():
    f, w, i = torch.zeros(2, 2, 64), torch.ones(64), torch.zeros(2, dtype=torch.int32)
    c, t = torch.zeros(2, 16, 2, 64), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        gl.qk_norm_rope(f, f, w, w)
    with pytest.raises(ValueError, match=r"\[T, heads, D\]"):
        gl.qk_norm_rope(f[0], f, w, w)
    with pytest.raises(ValueError, match="expected torch.bfloat16"):
        gl.qk_norm_rope(f.half(), f.half(), w, w)
    with pytest.raises(ValueError, match="GPU"):
        gl.paged_attention(f, c, c, t, i)
    with pytest.raises(ValueError, match="page_size"):
        gl.paged_attention(f, c[0], c, t, i)
    with pytest.raises(ValueError, match="GPU"):
        gl.pages_update(t, i, i, 16)
    with pytest.raises(ValueError, match="rows"):
        gl.pages_update(i, i, i, 16)
    with pytest.raises(ValueError, match="GPU"):
        gl.pages_compact(t, i, i, 16)
    with pytest.raises(ValueError, match="at least one"):
        gl.pages_copy([], i, i)
    with pytest.raises(ValueError, match="GPU"):
        gl.pages_copy([c], i, i)
    with pytest.raises(ValueError, match="GPU"):
        gl.token_logprobs(torch.zeros(2, 5))
    with pytest.raises(ValueError, match=r"\[T, V\]"):
        gl.token_logprobs(torch.zeros(5))
    with pytest.raises(ValueError, match="one of"):
        gl.token_logprobs_backward(torch.zeros(2, 5), w, w)
    with pytest.raises(ValueError, match="targets"):
        gl.token_logprobs_backward(torch.zeros(2, 5), w, w, d_logprobs=w)
    with pytest.raises(ValueError, match="pairs"):
        gl.rope_frequencies(3, device="cpu")


def test_frequencies():
    f = gl.rope_frequencies(8, 1e4, "cpu")
    assert f.dtype is torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert gl.rope_frequencies(0, device="cpu").numel() == 0


def test_workspaces():
    n = ctypes.c_size_t(7)
    L = gl.lib()
    assert L.beam_moe_qk_norm_rope_workspace_bytes(0, 4, 2, 128, ctypes.byref(n)) == gl.OK and n.value == 0
    assert L.beam_moe_qk_norm_rope_workspace_bytes(9, 4, 2, 128, ctypes.byref(n)) == gl.OK and n.value > 0
    assert L.beam_moe_qk_norm_rope_workspace_bytes(9, 4, 2, 128, None) == INVALID
    assert L.beam_moe_paged_attention_workspace_bytes(0, 4, 2, 128, ctypes.byref(n)) == gl.OK and n.value == 0
    assert L.beam_moe_paged_attention_workspace_bytes(3, 4, 3, 128, ctypes.byref(n)) == INVALID
    assert L.beam_moe_pages_workspace_bytes(100, 65537, ctypes.byref(n)) == UNSUPPORTED
    assert L.beam_moe_token_logprobs_workspace_bytes(3, 10, 11, ctypes.byref(n)) == INVALID
    assert L.beam_moe_token_logprobs_workspace_bytes(1, 131072, 8, ctypes.byref(n)) == gl.OK and n.value > 0

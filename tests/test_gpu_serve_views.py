"""Views that begin between 16-byte boundaries, as a shifted target or the rows of a
batch from some n on are: every index, length and scalar of the operators around a
paged cache gives what its copy gives, bit for bit."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
from gpu_util import device
from test_gpu_rope import BF16, cache, heads, make, on

pytestmark = pytest.mark.gpu


def shifted(t):
    """The same values, one element behind a 16-byte boundary."""
    flat = torch.cat([t.flatten()[:1], t.flatten()])
    v = flat[1:].view(t.shape)
    assert v.is_contiguous() and v.data_ptr() % 16
    return v


def same(fn, args, **kw):
    """fn's outputs of shifted arguments against those of plain ones."""
    def outputs(x):
        x = x.values() if isinstance(x, dict) else x if isinstance(x, tuple) else (x,)
        return [t.clone() for t in x if torch.is_tensor(t)]
    want = outputs(fn(**args, **kw))
    for name in args:
        got = outputs(fn(**{k: shifted(v) if k == name else v for k, v in args.items()}, **kw))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
    odd = {k: shifted(v) for k, v in args.items()}
    assert all(torch.equal(a, b) for a, b in zip(outputs(fn(**odd, **kw)), want))
    # on a stream of its own
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fn(**odd, **kw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(outputs(got), want))
    # captured, and replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fn(**odd, **kw)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outputs(got), want))


def test_head_norms():
    dev, T, Hq, Hkv, D = device(), 6, 4, 2, 64
    c = on(dev, make(T, Hq, Hkv, D, BF16, 64, 1, far=60))
    q, k, v = heads(c["qkv"], Hq, Hkv, D)
    args = dict(q_weight=c["q_weight"], k_weight=c["k_weight"], positions=c["positions"], inv_freq=c["inv_freq"])
    same(lambda **a: gl.qk_norm_rope(q, k, **a), args)
    same(lambda **a: gl.qk_norm_rope_backward(c["d_q"], c["d_k"], q, k, **a), args)
    args["tables"] = torch.randperm(24, device=dev)[:24].to(torch.int32).view(6, 4)
    args["rows"] = torch.arange(6, dtype=torch.int32, device=dev)

    def cached(**a):
        kc, vc = (torch.zeros(24, 16, Hkv, D, dtype=BF16, device=dev) for _ in range(2))
        side = a.get("stream")
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        return gl.qk_norm_rope(q, k, v=v, k_cache=kc, v_cache=vc, **a)[0], kc, vc
    same(cached, args)


def test_attention():
    dev, g = device(), torch.Generator().manual_seed(2)
    kc, vc = (x.to(dev) for x in cache(g, 30, 16, 2, 64, BF16, "tokens"))
    q = torch.randn(3, 6, 64, generator=g).to(BF16).to(dev)
    args = dict(tables=torch.randperm(30, generator=g).to(torch.int32).view(3, 10).to(dev),
                lengths=torch.tensor([5, 160, 77], dtype=torch.int32, device=dev))
    same(lambda **a: gl.paged_attention(q, kc, vc, with_lse=True, **a), args)


def test_pages():
    dev, i32 = device(), torch.int32
    tables = torch.tensor([[3, 1, -1], [0, 2, -1], [5, -1, -1]], dtype=i32, device=dev)
    refs = torch.tensor([1, 1, 1, 1, 0, 1, 0, 0, 0], dtype=i32, device=dev)
    args = dict(tables=tables, lengths=torch.tensor([6, 8, 1], dtype=i32, device=dev), refs=refs)
    same(lambda **a: gl.pages_compact(page_size=4, **a), args)
    args.update(parents=torch.tensor([0, 0, -1], dtype=i32, device=dev), grow=torch.tensor([1, 2, 3], dtype=i32, device=dev))
    same(lambda **a: gl.pages_update(page_size=4, **a), args)
    pool = torch.arange(2 * 9 * 8, dtype=torch.float32, device=dev).view(2, 9, 8)
    src, dst = (torch.tensor(x, dtype=i32, device=dev) for x in ([0, 2, 3], [4, 6, 7]))

    def copy(**a):
        p = pool.clone()
        if a.get("stream") is not None:
            a["stream"].wait_stream(torch.cuda.current_stream())
        gl.pages_copy([p], **a)
        return p
    same(copy, dict(src=src, dst=dst))


def test_scores():
    dev, g, T, V = device(), torch.Generator().manual_seed(3), 7, 1003
    x = (torch.randn(T, V, generator=g) * 4).to(dev)
    t = torch.randint(0, V, (T,), generator=g).to(dev)
    same(lambda **a: gl.token_logprobs(x, softcap=30.0, top=3, **a), dict(targets=t))
    r = gl.token_logprobs(x, t, softcap=30.0)
    args = dict(lse=r["lse"], entropy=r["entropy"], targets=t, d_logprobs=torch.randn(T, generator=g).to(dev),
                d_entropy=torch.randn(T, generator=g).to(dev))
    same(lambda **a: gl.token_logprobs_backward(x, softcap=30.0, **a), args)


def test_the_shift_of_a_language_model():
    # every word's score is of the word after it
    dev, g = device(), torch.Generator().manual_seed(4)
    x, tokens = torch.randn(9, 100, generator=g).to(dev), torch.randint(0, 100, (10,), generator=g).to(dev)
    got = gl.token_logprobs(x, tokens[1:])["logprobs"]
    assert torch.equal(got, gl.token_logprobs(x, tokens[1:].clone())["logprobs"])


def test_data_read_in_sixteen_bytes_is_refused():
    dev = device()
    x = torch.zeros(5, 7, dtype=BF16, device=dev)
    with pytest.raises(gl.BeamError):
        gl.token_logprobs(x[1:])
    flat = torch.zeros(2 * 64 + 1, dtype=BF16, device=dev)
    with pytest.raises(gl.BeamError):
        gl.qk_norm_rope(flat[1:].view(2, 1, 64), flat[:-1].view(2, 1, 64), torch.ones(64, device=dev), torch.ones(64, device=dev))

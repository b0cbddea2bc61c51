"""Limits of the operators around a paged cache at their edges: sizes and scalars
whose arithmetic would leave its type are refused before any GPU work."""
import pytest

import group_limited_routing_sigmoid_amd as gl
from test_serve_refusals import UNSUPPORTED, _attend, _pool, _score, _score_grad, _update

EMPTY = dict(seqs=0, q=None, lengths=None, out=None, ws=None, n=0)


@pytest.mark.parametrize("size", [1, 16, 1 << 10, 1 << 15])
def test_attention_holds_the_last_tokens_in_32_bits(size):
    # a wave looks 64 steps of at most 256 tokens ahead of a sequence's end
    most = ((1 << 31) - (1 << 16)) // size
    assert _attend(size=size, cols=most, **EMPTY) == gl.OK
    assert _attend(size=size, cols=most + 1, **EMPTY) == UNSUPPORTED


def test_pools_have_few_layers():
    # arrays times layers are counted in 32 bits
    assert _update(pool=_pool(count=8, layers=(1 << 16) + 1)) == UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(cap=1e38), gl.OK), (dict(cap=1.3e38), UNSUPPORTED), (dict(cap=30.0, scale=1e37), UNSUPPORTED),
    (dict(cap=1e-38), gl.OK), (dict(cap=5e-39), UNSUPPORTED), (dict(cap=0.0, scale=2e38), gl.OK),
    (dict(cap=0.0, scale=3e38), UNSUPPORTED)])
def test_scores_have_finite_factors(kw, status):
    # 2 log2(e) scale cap, 2 log2(e) / cap and log2(e) scale are binary32 numbers
    assert _score(T=0, **kw) == _score_grad(T=0, **kw) == status


def test_attention_has_a_finite_scale():
    assert _attend(scale=2e38, **EMPTY) == gl.OK  # times log2(e)
    assert _attend(scale=3e38, **EMPTY) == UNSUPPORTED

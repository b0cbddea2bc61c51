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

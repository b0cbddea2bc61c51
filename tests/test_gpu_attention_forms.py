"""Attention over a paged cache with every number of query heads to a key-value
head that the forms of whole sequences hold, up to their largest share of LDS.
Tolerances are test_gpu_attention's."""
import pytest
import torch

from gpu_util import device
from test_gpu_attention import BF16, F32, call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hkv,cols,window", [
    (3, 2, 16, 0), (2, 1, 24, 0),               # tables of four and six units, in one launch
    (70, 2, 40, 0), (65, 2, 60, 200)])          # 128 sequences' heads and more
@pytest.mark.parametrize("group", [1, 6, 8, 15, 16, 17])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_of_whole_sequences(B, Hkv, cols, window, group, D, dtype):
    lengths = [(i * 97) % (cols * 16 + 1) for i in range(1, B + 1)]
    lengths[0] = cols * 16
    c = make(lengths, group * Hkv, Hkv, D, 16, dtype, B + group, cols=cols)
    check(c, *call(c, device(), window, True), window, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hkv,cols", [(3, 2, 8), (4, 1, 60), (300, 2, 20)])
@pytest.mark.parametrize("group", [16, 19])
def test_heads_of_256(B, Hkv, cols, group, dtype):
    # whole and in slices
    lengths = [(i * 97) % (cols * 16 + 1) for i in range(1, B + 1)]
    c = make(lengths, group * Hkv, Hkv, 256, 16, dtype, B + group, cols=cols)
    check(c, *call(c, device(), 0, True), 0, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_heads_of_a_long_sequence(dtype):
    # the model's 48 query heads on one key-value head, in slices, again and again
    c = make([5000, 7, 901], 48, 1, 128, 16, dtype, 3)
    dev = device()
    out, lse = call(c, dev, 0, True)
    check(c, out, lse, 0, True)
    for _ in range(3):
        again, l2 = call(c, dev, 0, True)
        assert torch.equal(out, again) and torch.equal(lse, l2)

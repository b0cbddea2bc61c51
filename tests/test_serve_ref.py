"""The 64-bit gradients that the GPU tests compare against, against central
differences of the 64-bit forward functions, and the page tables' plain steps on
a case worked by hand."""
import math

import pytest
import torch

import serve_ref as ref

F64 = torch.float64


def difference(f, x, dy, h=1e-6):
    """Gradient of sum(dy * f(x)) by central differences, element by element."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view(x.shape)
        g.view(-1)[i] = ((f(x + d) - f(x - d)) * dy).sum() / (2 * h)
    return g


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,temp", [(0, None), (0, (2048.0, 0.1)), (4, None), (8, (3.0, 1.5))])
def test_rope_gradient(rot, temp, interleaved):
    g = torch.Generator().manual_seed(rot)
    x, dy = (torch.randn(3, 2, 8, generator=g, dtype=F64) for _ in range(2))
    w, pos = 1 + torch.randn(8, generator=g, dtype=F64) / 10, torch.tensor([0, 5, 1000])
    f = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=F64)[:rot // 2] if rot else None
    y = lambda a, b: ref.rope(a, b, pos, f, interleaved, 1e-6, temp)[0]
    dx, dw = ref.rope_grad(dy, x, w, pos, f, interleaved, 1e-6, temp)
    assert torch.allclose(dx, difference(lambda a: y(a, w), x, dy), rtol=1e-7, atol=1e-8)
    assert torch.allclose(dw, difference(lambda b: y(x, b), w, dy), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("softcap,scale", [(0.0, 1.0), (30.0, 1.0), (2.0, 1.7)])
def test_score_gradient(softcap, scale):
    g = torch.Generator().manual_seed(7)
    x = torch.randn(3, 6, generator=g, dtype=F64) * 2
    t, dl, dh = torch.tensor([2, -1, 5]), torch.randn(3, generator=g, dtype=F64), torch.randn(3, generator=g, dtype=F64)

    def f(a):
        r = ref.score(a, t, softcap, scale)
        return torch.stack([r["logprobs"], r["entropy"]])
    want = difference(f, x, torch.stack([dl, dh]))
    assert torch.allclose(ref.score_grad(x, t, dl, dh, softcap, scale), want, rtol=1e-6, atol=1e-8)
    x[:, 1] = -math.inf                     # a masked word takes no part
    keep = [0, 2, 3, 4, 5]
    t2 = torch.tensor([1, -1, 4])
    got = ref.score_grad(x, t, dl, dh, softcap, scale)
    assert torch.allclose(got[:, keep], ref.score_grad(x[:, keep], t2, dl, dh, softcap, scale))
    assert (got[:, 1] == 0).all()


def test_page_steps_by_hand():
    # pages of 4 tokens; row 0 holds 6 tokens (pages 3, 1), row 1 four (page 5)
    tables, lengths = [[3, 1, -1], [5, -1, -1]], [6, 4]
    refs = [0, 1, 0, 1, 2, 1, 0]
    # three go on from row 0, each with one token; row 1 ends; one starts anew
    t, n, r, missing, copies = ref.pages_update(tables, lengths, refs, 4, [0, 0, 7, 0], [1, 1, 2, 0])
    # the page 1 is shared with row 3, which does not write: both writers copy
    assert t == [[3, 0, -1], [3, 2, -1], [5, -1, -1], [3, 1, -1]] and n == [7, 7, 2, 6]
    assert r == [1, 1, 1, 3, 2, 1, 0] and missing == 0 and copies == [(1, 0), (1, 2)]
    # without the reader the lowest writer keeps it
    t, n, r, missing, copies = ref.pages_update(tables, lengths, refs, 4, [0, 0], [1, 7])
    assert t == [[3, 1, -1], [3, 0, 2]] and r == [1, 1, 1, 2, 2, 0, 0] and copies == [(1, 0)]
    assert n == [7, 12] and missing == 1          # 13 tokens: a page more than the columns


def test_packing_by_hand():
    t, r, new_id, live, moves = ref.pages_compact([[6, 1, 9], [4, 6, 0]], [12, 4], [0, 1, 0, 0, 2, 0, 3], 4)
    assert live == 3 and moves == [(4, 0), (6, 2)] and r == [2, 1, 3, 0, 0, 0, 0]
    assert new_id == [-1, 1, -1, -1, 0, -1, 2] and t == [[2, 1, -1], [0, -1, -1]]

"""Page tables and page copies (beam_moe_pages_update, _compact, _copy) on the GPU
against plain steps over lists: whole numbers, equal in every place."""
import random

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
from gpu_util import device

pytestmark = pytest.mark.gpu

I32 = torch.int32


def make(rng, rows, cols, page, pages, shared=0.3, outside=0.1):
    """A batch whose rows share their first pages now and then, counted."""
    free = list(range(pages))
    rng.shuffle(free)
    tables, lengths, refs = [], [], [0] * pages
    for i in range(rows):
        n = rng.randint(0, cols * page)
        have = ref.ceil_div(n, page)
        t = []
        if tables and rng.random() < shared:
            j = rng.randrange(i)
            t = tables[j][:min(have, ref.ceil_div(lengths[j], page))]
            if len(t) == ref.ceil_div(lengths[j], page):     # with the unfilled page, the same tokens of it
                n = lengths[j] if len(t) == have and t else n
                have = ref.ceil_div(n, page)
        while len(t) < have:
            if not free:
                n, have = len(t) * page, len(t)
                break
            t.append(free.pop())
        for p in t:
            refs[p] += 1
        tables.append(t + [-1 - rng.randrange(3)] * (cols - len(t)))
        lengths.append(n)
    for p in range(pages):
        if rng.random() < outside:
            refs[p] += 1
    return tables, lengths, refs


def to_dev(x, dev, shape=None):
    t = torch.tensor(x, dtype=I32, device=dev)
    return t if shape is None else t.reshape(shape)


def pools_of(dev, layers, pages, sizes, dtype=torch.int16):
    g = torch.Generator(device=dev).manual_seed(1)
    return [torch.randint(-30000, 30000, (layers, pages, *s), generator=g, device=dev, dtype=dtype) for s in sizes]


def check_update(tables, lengths, refs, page, parents, grow, dev, cols, layers=2, sizes=((8,), (3, 8)), **kw):
    pages, rows = len(refs), len(tables) if parents is None else len(parents)
    want = ref.pages_update(tables, lengths, refs, page, parents, grow)
    pools = pools_of(dev, layers, pages, sizes)
    kept = [p.clone() for p in pools]
    inputs = (to_dev(tables, dev, (len(tables), cols)), to_dev(lengths, dev), to_dev(refs, dev))
    before = [t.clone() for t in inputs]
    got = gl.pages_update(*inputs, page, parents=None if parents is None else to_dev(parents, dev),
                          grow=None if grow is None else to_dev(grow, dev), pools=pools, **kw)
    assert all(torch.equal(a, b) for a, b in zip(inputs, before))
    assert got["tables"].tolist() == want[0] if rows and cols else got["tables"].shape == (rows, cols)
    assert got["lengths"].tolist() == want[1]
    assert got["refs"].tolist() == want[2]
    assert got["missing"].tolist() == [want[3]]
    for p, k in zip(pools, kept):
        for a, b in want[4]:
            k[:, b] = k[:, a]
        assert torch.equal(p, k)
    return got, want


@pytest.mark.parametrize("seed", range(12))
def test_steps(seed):
    rng = random.Random(seed)
    rows, cols = rng.choice([1, 2, 7, 40, 130]), rng.choice([1, 3, 20, 70])
    page, pages = rng.choice([1, 4, 16]), rng.choice([5, 100, 2500, 6000])
    tables, lengths, refs = make(rng, rows, cols, page, pages)
    n = rng.choice([1, rows, 3 * rows])
    parents = [rng.randint(-2, rows + 1) for _ in range(n)]
    grow = [rng.choice([0, 1, 1, page, 3 * page + 1, -4]) for _ in range(n)]
    check_update(tables, lengths, refs, page, parents, grow, device(), cols)


def test_more_rows_than_a_workgroup_counts():
    rng = random.Random(5)
    tables, lengths, refs = make(rng, 60, 6, 4, 9000)
    parents = [rng.randint(-1, 59) for _ in range(2500)]
    check_update(tables, lengths, refs, 4, parents, [1] * 2500, device(), 6)


@pytest.mark.parametrize("parents,grow", [(None, None), (None, [1, 5, 0, 9]), ([1, 1, 1, 1], None), ([], [])])
def test_defaults(parents, grow):
    rng = random.Random(9)
    tables, lengths, refs = make(rng, 4, 5, 4, 60)
    check_update(tables, lengths, refs, 4, parents, grow, device(), 5)


def test_no_free_pages_and_no_columns():
    dev = device()
    # two free pages for five wants, in the rows' order
    tables, lengths, refs = [[0, 1], [2, -1], [3, 4]], [8, 2, 6], [1, 1, 1, 1, 1, 0, 0]
    got, want = check_update(tables, lengths, refs, 4, [0, 1, 1, 2, 2], [1, 1, 1, 0, 7], dev, 2)
    assert want[3] > 0
    # none at all
    check_update([[0]], [3], [2], 4, [0, 0], [1, 1], dev, 1)
    # a pool without pages, a table without columns
    check_update([[-1, -1]], [0], [], 4, [0, -1], [3, 3], dev, 2, sizes=())
    check_update([[], []], [0, 5], [0, 0], 4, [0, 1], [3, 0], dev, 0)


def test_ids_that_name_no_page():
    # carried along, not counted, not copied
    check_update([[-1, 9], [1 << 30, 2]], [7, 7], [0, 0, 1, 0, 0, 0], 4, [0, 1, 1], [1, 1, 1], device(), 2)


def test_lengths_beyond_bounds():
    check_update([[0, 1], [2, -1]], [1000, -3], [1, 1, 0, 0], 4, [0, 1], [1, 5], device(), 2)
    check_update([[0, 1]], [8], [1, 1, 0, 0], 4, [0], [(1 << 31) - 1], device(), 2)


def test_pools_of_strides_and_types():
    dev, rng = device(), random.Random(3)
    tables, lengths, refs = make(rng, 6, 4, 4, 40, outside=0.3)
    parents, grow = [0, 0, 1, 2, 3, 3, 4, 5], [1] * 8
    want = ref.pages_update(tables, lengths, refs, 4, parents, grow)
    base = torch.randn(40, 3, 2, 4, 64, device=dev)                       # [pages, layers, k or v, page, width]
    pools = [base[:, :, 0].transpose(0, 1), base[:, :, 1].transpose(0, 1)]
    big = torch.randn(3, 40, 5, 1000, device=dev, dtype=torch.float64)    # 40 KB a page
    keep, keep_big = base.clone(), big.clone()
    gl.pages_update(to_dev(tables, dev), to_dev(lengths, dev), to_dev(refs, dev), 4, to_dev(parents, dev),
                    to_dev(grow, dev), pools=pools + [big])
    assert want[4]
    for a, b in want[4]:
        keep[b], keep_big[:, b] = keep[a], keep_big[:, a]
    assert torch.equal(base, keep) and torch.equal(big, keep_big)


@pytest.mark.parametrize("seed", range(8))
def test_packing(seed):
    dev, rng = device(), random.Random(seed)
    rows, cols = rng.choice([1, 30, 200]), rng.choice([1, 8, 50])
    page, pages = rng.choice([1, 16]), rng.choice([1, 100, 2048, 7000])
    tables, lengths, refs = make(rng, rows, cols, page, pages)
    refs = [r if rng.random() < 0.9 else 0 for r in refs]      # some of them of no page now
    want = ref.pages_compact(tables, lengths, refs, page)
    pools = pools_of(dev, 2, pages, ((8,), (16, 8)))
    kept = [p.clone() for p in pools]
    got = gl.pages_compact(to_dev(tables, dev), to_dev(lengths, dev), to_dev(refs, dev), page, pools)
    assert [got[k].tolist() for k in ("tables", "refs", "new_id")] == list(want[:3])
    assert got["live"].tolist() == [want[3]]
    for p, k in zip(pools, kept):
        for a, b in want[4]:
            k[:, b] = k[:, a]
        assert torch.equal(p, k)


def test_packing_of_nothing():
    dev = device()
    e = torch.zeros(0, dtype=I32, device=dev)
    got = gl.pages_compact(torch.zeros(0, 3, dtype=I32, device=dev), e, e, 16)
    assert got["live"].tolist() == [0] and got["refs"].numel() == 0
    # all pages used, none used
    for r in ([1, 1, 2], [0, 0, 0]):
        got = gl.pages_compact(to_dev([[0, 2]], dev), to_dev([5], dev), to_dev(r, dev), 4)
        assert got["refs"].tolist() == r and got["live"].tolist() == [3 if r[0] else 0]


def test_copies():
    dev = device()
    pools = pools_of(dev, 3, 50, ((8,), (33, 8), (2, 4096)))
    kept = [p.clone() for p in pools]
    src, dst = [3, 9, -1, 7, 50, 12], [40, 41, 42, -2, 43, 1 << 30]
    gl.pages_copy(pools, to_dev(src, dev), to_dev(dst, dev))
    for k in kept:
        k[:, 40], k[:, 41] = k[:, 3], k[:, 9]
    assert all(torch.equal(a, b) for a, b in zip(pools, kept))
    gl.pages_copy(pools, to_dev([], dev), to_dev([], dev))


def test_the_largest_batch_of_one_workgroup():
    rng = random.Random(8)
    for rows, cols, pages in ((1024, 64, 8192), (1024, 64, 8193), (1025, 63, 8192), (1000, 66, 8000)):
        tables, lengths, refs = make(rng, rows, cols, 16, pages, shared=0.8)
        parents = [rng.randint(-1, rows) for _ in range(rows)]
        check_update(tables, lengths, refs, 16, parents, [rng.choice([0, 1, 40]) for _ in range(rows)], device(), cols)


@pytest.mark.parametrize("rows", [3, 1500])
def test_growth_of_every_size(rows):
    # tokens past 2^31, more missing pages than an int32 holds
    most = (1 << 31) - 1
    tables, lengths, refs = [[4, 2, 7]] * 2, [3, 2], [0, 0, 2, 0, 2, 0, 0, 1] + [0] * 40
    for grow in (most, most - 2, 1 << 30, 5):
        want = ref.pages_update(tables, lengths, refs, 1, [i % 3 for i in range(rows)], [grow] * rows)
        dev = device()
        got = gl.pages_update(to_dev(tables, dev), to_dev(lengths, dev), to_dev(refs, dev), 1,
                              to_dev([i % 3 for i in range(rows)], dev), to_dev([grow] * rows, dev))
        assert [got[k].tolist() for k in ("tables", "lengths", "refs")] == list(want[:3])
        assert got["missing"].tolist() == [min(want[3], most)]

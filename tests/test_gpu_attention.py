"""Attention of one new token over a paged cache (beam_moe_paged_attention) on
the GPU against the 64-bit formula.

Tolerances count roundings of u = 2^-24 (matrix instructions' sums: 2 u an
addition, however they round).  A score's sum of D products is off by 2 D + 4 u
of its terms' absolute values, its scaling and its distance to the maximum by 8 u
of the largest score and 8 binary orders, its exponential by 2: together the
relative error dp of a probability.  A sum over n tokens adds n / 4 of them in a
lane's chain, 2 u each, and the joining of lanes, waves and workgroups at most 400
more.  The gate's sigmoid is off by (|g| + 8) u.  The output is rounded once to
its type (half its eps)."""
import math

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
from gpu_util import device
from test_gpu_rope import cache, half_step, move

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(lengths, Hq, Hkv, D, page, dtype, seed, layout="tokens", extra=3, cols=None):
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lengths]
    cols = max(need + [1]) + 1 if cols is None else cols
    pages = sum(need) + extra
    ids = torch.randperm(pages, generator=g).tolist()
    tables = torch.full((len(lengths), cols), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(min(n, cols)):
            tables[b, i] = ids.pop()
    kc, vc = cache(g, pages, page, Hkv, D, dtype, layout)
    B = len(lengths)
    return dict(q=torch.randn(B, Hq, D, generator=g).to(dtype), gate=(torch.randn(B, Hq, D, generator=g) * 2).to(dtype),
                k_cache=kc, v_cache=vc, tables=tables, lengths=torch.tensor(lengths, dtype=torch.int32))


def call(c, dev, window=0, gate=False, scale=None, **kw):
    return gl.paged_attention(c["q"].to(dev), move(dev, c["k_cache"]), move(dev, c["v_cache"]), c["tables"].to(dev),
                              c["lengths"].to(dev), scale=scale, window=window,
                              gate=c["gate"].to(dev) if gate else None, with_lse=True, **kw)


def check(c, out, lse, window=0, gate=False, scale=None):
    D, dtype = c["q"].shape[2], c["q"].dtype
    scale = 1 / math.sqrt(D) if scale is None else scale
    want = ref.attend(c["q"], c["k_cache"], c["v_cache"], c["tables"], c["lengths"], scale, window,
                      c["gate"] if gate else None)
    out, lse = out.cpu().double(), lse.cpu().double()
    for b, w in enumerate(want):
        if w["n"] == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all(), b
            continue
        dp = ref.U * ((2 * D + 4) * w["dots"] + 8 * (w["smax"] + 8) + 2)
        chain = (w["n"] / 2 + 400) * ref.U
        rel = (2 * dp + 2 * chain + 8 * ref.U)[:, None]
        if gate:
            rel = rel + (c["gate"][b].double().abs() + 8) * ref.U
        tol = rel * w["size"]
        tol = tol + half_step(dtype) * (w["out"].abs() + tol)
        err = (out[b] - w["out"]).abs()
        assert (err <= tol).all(), f"sequence {b}: {(err - tol).max():.3e} over, at most {err.max():.3e} off"
        tol = dp + chain + 8 * ref.U * (w["lse"].abs() + 8)
        assert ((lse[b] - w["lse"]).abs() <= tol).all(), b


LENGTHS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 700, 1025]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D,page,window,gate,layout", [
    (48, 8, 128, 16, 0, True, "tokens"), (48, 8, 128, 16, 512, True, "tokens"), (6, 1, 64, 1, 0, False, "heads"),
    (4, 4, 128, 8, 100, False, "both"), (8, 2, 256, 64, 0, True, "tokens"), (17, 1, 128, 32, 0, False, "tokens"),
    (40, 1, 64, 4, 33, True, "heads"), (2, 1, 80, 16, 0, False, "tokens"), (3, 3, 8, 2, 7, True, "tokens"),
    (10, 2, 200, 256, 0, False, "heads"), (32, 2, 96, 16, 1, False, "both"), (5, 1, 128, 128, 2000, False, "tokens")])
def test_lengths(Hq, Hkv, D, page, window, gate, layout, dtype):
    c = make(LENGTHS, Hq, Hkv, D, page, dtype, Hq + D, layout)
    dev = device()
    out, lse = call(c, dev, window, gate)
    check(c, out, lse, window, gate)
    again, _ = call(c, dev, window, gate)
    assert torch.equal(out, again)
    # each sequence alone: another division of the work
    for b in (1, 6, 9, 11):
        one = {k: v[b:b + 1] if k in ("q", "gate", "tables", "lengths") else v for k, v in c.items()}
        check(one, *call(one, dev, window, gate), window, gate)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [4, 16])
def test_ids_that_name_no_page(page, dtype):
    c = make([100, 65, 40, 16], 12, 2, 128, page, dtype, 1)
    c["tables"][0, 1], c["tables"][0, 3], c["tables"][2, :] = -1, 1 << 30, -7
    c["tables"][1, 0] = c["k_cache"].shape[0]
    for window in (0, 50):
        out, lse = call(c, device(), window)
        check(c, out, lse, window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [4, 16, 64])
def test_what_is_behind_a_length_is_not_read(page, dtype):
    # NaN and infinities in the pages' rest, before a window, and in other pages
    c = make([33, 61, 130, 1], 6, 2, 64, page, dtype, 2)
    dev = device()
    for window in (0, 19):
        want, _ = call(c, dev, window)
        d = dict(c, k_cache=c["k_cache"].clone(), v_cache=c["v_cache"].clone())
        seen = torch.zeros(d["k_cache"].shape[:2], dtype=torch.bool)
        for b, n in enumerate(c["lengths"].tolist()):
            for i in range(max(0, n - window) if window else 0, n):
                seen[int(c["tables"][b, i // page]), i % page] = True
        for bad in (math.nan, math.inf, -math.inf):
            d["k_cache"][~seen], d["v_cache"][~seen] = bad, bad
            out, lse = call(d, dev, window)
            assert torch.equal(out, want) and torch.isfinite(lse).all()


def test_lengths_past_the_table_and_below_zero():
    c = make([64, 64, 10], 6, 2, 128, 16, BF16, 3, cols=4)
    c["lengths"] = torch.tensor([1000, (1 << 31) - 1, -5], dtype=torch.int32)
    check(c, *call(c, device()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [0.0, 30.0])
def test_sizes_of_scores(size, dtype):
    # all scores alike; scores hundreds apart, the largest one last or first
    for sign in (1, -1):
        c = make([200, 77], 4, 2, 64, 16, dtype, 4)
        c["q"] = (c["q"] * size).to(dtype)
        order = torch.linspace(-1, 1, c["k_cache"].shape[0])[:, None, None, None] * sign
        c["k_cache"] = (c["k_cache"] + order).to(dtype)
        check(c, *call(c, device()))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_sequences_and_a_long_one(dtype):
    # the units' division over more sequences than a wave counts at once
    lengths = [(37 * i) % 90 for i in range(150)] + [5000]
    c = make(lengths, 4, 2, 64, 16, dtype, 5)
    check(c, *call(c, device(), gate=True), gate=True)


def test_scale_and_given_output():
    c = make([50, 9], 4, 1, 64, 16, BF16, 6)
    dev = device()
    out = torch.full((2, 4, 64), 7.0, dtype=BF16, device=dev)
    got, lse = call(c, dev, scale=0.3, out=out)
    assert got is out
    check(c, got, lse, scale=0.3)


def test_cache_of_more_than_two_to_the_31():
    # 2^21 + 3 tokens of 1,024 values: element offsets past 31 bits, byte offsets
    # past 32; the weights are alike, so the result is the values' mean
    dev, P, page, Hkv, D = device(), (1 << 15) + 1, 64, 8, 128
    n = (P - 1) * page + 3
    k = torch.zeros(P, page, Hkv, D, dtype=BF16, device=dev)
    v = torch.zeros(P, page, Hkv, D, dtype=BF16, device=dev)
    assert v.numel() > 1 << 31
    v[P - 1, 2] = 8.0            # the last token
    v[0, 5] = -4.0
    q = torch.ones(1, 8, D, dtype=BF16, device=dev)
    tables = torch.arange(P, dtype=torch.int32, device=dev)[None]
    lengths = torch.tensor([n], dtype=torch.int32, device=dev)
    out, lse = gl.paged_attention(q, k, v, tables, lengths, with_lse=True)
    # exact terms; their sum over n, the division and the rounding to bf16
    assert ((out.double().cpu() - 4.0 / n).abs() <= 4.0 / n * 2.0 ** -8 * 1.01).all()
    assert ((lse.double().cpu() - math.log(n)).abs() <= 1e-5).all()
    # the last token alone, through the window
    out, lse = gl.paged_attention(q, k, v, tables, lengths, window=1, with_lse=True)
    assert (out == 8.0).all() and (lse == 0.0).all()


def test_empty_batch():
    dev = device()
    q = torch.empty(0, 4, 64, dtype=BF16, device=dev)
    k = torch.zeros(2, 16, 2, 64, dtype=BF16, device=dev)
    i = torch.zeros(0, 3, dtype=torch.int32, device=dev)
    out, lse = gl.paged_attention(q, k, k, i, i[:, 0].contiguous(), with_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [8, 16])
def test_nan_stays_where_it_is_read(page, dtype):
    # in a query: that head alone; in a cached token: the heads that read it
    c = make([300, 40, 900, 0], 6, 2, 64, page, dtype, 12)
    dev = device()
    for what in ("q", "k_cache", "v_cache"):
        d = {k: v.clone() for k, v in c.items()}
        if what == "q":
            d["q"][2, 4, 9] = math.nan
            hit = [(2, 4)]
        else:
            d[what][int(c["tables"][2, 100 // page]), 100 % page, 1, 3] = math.nan
            hit = [(2, h) for h in (3, 4, 5)]
        out, lse = call(d, dev)
        for b, h in hit:
            assert torch.isnan(out[b, h]).any()
            out[b, h], lse[b, h] = 0.0, 0.0
        assert torch.isfinite(out.float()).all()
        want, wl = call(c, dev)
        for b, h in hit:
            out[b, h], lse[b, h] = want[b, h], wl[b, h]
        check(c, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,Hkv,cols,window", [
    (3, 2, 14, 0), (5, 1, 16, 0), (2, 2, 17, 0),            # tables of a few units
    (70, 2, 68, 0), (70, 2, 150, 512), (130, 1, 17, 100),   # 128 to 511 heads of sequences
    (300, 2, 60, 0), (300, 2, 90, 300)])                    # more
@pytest.mark.parametrize("D", [64, 128])
def test_whole_sequences(B, Hkv, cols, window, D, dtype):
    lengths = [(i * 97) % (cols * 16 + 1) for i in range(1, B + 1)]
    c = make(lengths, 3 * Hkv, Hkv, D, 16, dtype, B + cols, cols=cols)
    check(c, *call(c, device(), window, True), window, True)


def test_graph_of_every_form():
    # captured calls of each way of dividing the work, replayed with other contents
    dev = device()
    cs = [make(n, 6, 2, 128, 16, BF16, i) for i, n in enumerate(([30, 9], [250], [900, 3000], [500] * 70, [40] * 300))]
    want = [[t.clone() for t in call(c, dev)] for c in cs]
    held = [(c["q"].to(dev), c["k_cache"].to(dev), c["v_cache"].to(dev), c["tables"].to(dev), c["lengths"].to(dev))
            for c in cs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [gl.paged_attention(*h, with_lse=True) for h in held]
    for _ in range(3):
        for o, l in got:
            o.zero_(), l.zero_()
        g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1])
    # a length that changes between replays is the one that counts
    held[2][4][1] = 17
    g.replay()
    torch.cuda.synchronize()
    check(dict(cs[2], lengths=held[2][4].cpu()), *got[2])

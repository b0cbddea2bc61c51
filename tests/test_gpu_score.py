"""Scores of tokens (beam_moe_token_logprobs and its gradient) on the GPU against
the 64-bit formulas.

Tolerances count roundings of u = 2^-24, in nats.  With a cap c and a scale s a
capped logit is off by dz = 16 s c u (the exponent's argument by 3 u, its
exponential by 2 more, the reciprocal by 3, at most 0.25 of the argument's error
and 5 u reaching r = 1 / (1 + e^x), which counts 2 s c times); without by 4 u of
the largest.  A probability is off by dz, by 8 u of the largest |z| (two
differences) and by 2; a row's sums add 300 u for the thread's 64 logits and the
joining.  The entropy's second sum has terms p (m - z).  The output of the
gradient is rounded once to its type (half its eps)."""
import math

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
from gpu_util import device
from test_gpu_rope import half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = ref.U


def make(T, V, dtype, seed, std=4.0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, V, generator=g) * std).to(dtype)
    if masked:
        x[torch.rand(T, V, generator=g) < masked] = -math.inf
    t = torch.randint(0, V, (T,), generator=g)
    t[::5] = -100
    if T > 3:
        t[3] = V
    return dict(logits=x, targets=t, d_l=torch.randn(T, generator=g), d_h=torch.randn(T, generator=g))


def bounds(r, softcap, scale):
    """Per row: errors of a z, a relative probability and lse."""
    z = torch.where(r["z"] > -math.inf, r["z"], 0.0).abs().amax(1)
    dz = 16 * softcap * scale * U + 0 * z if softcap else 4 * U * z
    dp = dz + 8 * U * z + 2 * U
    lse = torch.where(r["lse"] > -math.inf, r["lse"], 0.0).abs()
    return dz, dp, dp + 300 * U + 4 * U * lse, lse


def near(got, want, tol, what):
    got, tol = got.cpu().double(), tol + 0 * want
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), what
    err = (got - want).abs()[fin]
    assert (err <= tol[fin]).all(), f"{what}: {(err - tol[fin]).max():.3e} over, at most {err.max():.3e} off"


def check(c, got, softcap, scale, top):
    r = ref.score(c["logits"], c["targets"], softcap, scale, top)
    dz, dp, dl, lse = bounds(r, softcap, scale)
    near(got["lse"], r["lse"], dl, "lse")
    p = torch.exp(r["logp"])
    m = torch.where(torch.isfinite(r["z"].amax(1)), r["z"].amax(1), 0.0)
    spread = torch.where(p > 0, p * (m[:, None] - r["z"]), 0.0).sum(1)
    near(got["entropy"], r["entropy"], (1 + spread) * (2 * dp + 600 * U) + 4 * U * lse, "entropy")
    room = dz + dl + 8 * U * (lse + torch.where(r["z"] > -math.inf, r["z"], 0.0).abs().amax(1))
    near(got["logprobs"], r["logprobs"], room, "logprobs")
    if top:
        assert torch.equal(got["top_ids"].cpu().long(), r["top_ids"])
        near(got["top_logprobs"], r["top_logprobs"], room[:, None], "top")
    return r


def check_gradient(c, got, use_l, use_h, softcap, scale):
    args = (c["logits"], c["targets"], c["d_l"] if use_l else None, c["d_h"] if use_h else None, softcap, scale)
    want, size = ref.score_grad(*args), ref.score_grad(*args, absolute=True)
    r = ref.score(c["logits"], None, softcap, scale)
    _, dp, dl, _ = bounds(r, softcap, scale)
    rel = (4 * dp + 2 * dl + 1200 * U)[:, None]
    tol = rel * size
    if softcap:      # r (1 - r), each off by 12 u, counts 4 times
        d = torch.where(c["logits"] > -math.inf, 1 - torch.tanh(c["logits"].double() / softcap) ** 2, 1.0)
        tol = tol + 100 * U * size / d
    if use_h:        # the entropy's own error, and a small log probability's
        p = torch.exp(r["logp"])
        tol = tol + (scale * c["d_h"].abs().double()[:, None] * p) * ((dl + 1e-4 * 0)[:, None] * 2 + rel * (1 + r["entropy"][:, None]))
    near(got, want, tol + half_step(c["logits"].dtype) * (want.abs() + tol), "d_logits")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,softcap,scale,top,masked", [
    (1, 131072, 30.0, 1.0, 8, 0.0), (1, 1, 0.0, 1.0, 1, 0.0), (3, 7, 0.0, 2.0, 7, 0.3), (5, 8, 30.0, 1.0, 0, 0.3),
    (2, 100003, 30.0, 0.7, 16, 0.02), (40, 257, 5.0, 1.0, 16, 0.5), (7, 2048, 0.0, 1.0, 3, 0.0),
    (7, 2049, 0.0, 1.3, 5, 0.1), (4, 20000, 1.0, 10.0, 2, 0.0), (300, 5001, 0.0, 1.0, 1, 0.0),
    (1100, 2050, 30.0, 1.0, 4, 0.05), (70, 40001, 0.0, 1.0, 0, 0.0), (130, 33000, 30.0, 1.0, 5, 0.01)])
def test_scores_and_gradient(T, V, softcap, scale, top, masked, dtype):
    c = make(T, V, dtype, T + V, masked=masked)
    dev = device()
    x, t = c["logits"].to(dev), c["targets"].to(dev)
    got = gl.token_logprobs(x, t, softcap=softcap, scale=scale, top=top)
    check(c, got, softcap, scale, top)
    for use_l, use_h in ((True, True), (True, False), (False, True)):
        d = gl.token_logprobs_backward(x, got["lse"], got["entropy"], t, c["d_l"].to(dev) if use_l else None,
                                       c["d_h"].to(dev) if use_h else None, softcap=softcap, scale=scale)
        check_gradient(c, d, use_l, use_h, softcap, scale)
    # in the logits' place
    y = x.clone()
    assert gl.token_logprobs_backward(y, got["lse"], got["entropy"], None, None, c["d_h"].to(dev), softcap=softcap,
                                      scale=scale, out=y) is y
    assert torch.equal(y, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [5, 3000, 50000])
def test_equal_logits_rank_by_index(V, dtype):
    dev, g = device(), torch.Generator().manual_seed(V)
    x = torch.stack([torch.zeros(V), -torch.zeros(V), torch.randint(0, 3, (V,), generator=g).float(),
                     torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0), torch.full((V,), -math.inf),
                     torch.where(torch.arange(V) % 7 == 3, 1.0, -math.inf), torch.full((V,), 100.0),
                     50.0 + torch.randint(0, 40, (V,), generator=g)]).to(dtype)
    c = dict(logits=x, targets=torch.zeros(8, dtype=torch.int64))
    top = min(16, V)
    for softcap in (0.0, 30.0):
        got = gl.token_logprobs(x.to(dev), c["targets"].to(dev), softcap=softcap, top=top)
        check(c, got, softcap, 1.0, top)


def test_rows_that_are_masked_whole():
    dev = device()
    x = torch.full((3, 500), -math.inf)
    x[1, 7] = 2.0
    t = torch.tensor([3, 7, -1])
    for softcap in (0.0, 30.0):
        got = gl.token_logprobs(x.to(dev), t.to(dev), softcap=softcap, top=2)
        check(dict(logits=x, targets=t), got, softcap, 1.0, 2)
        d = gl.token_logprobs_backward(x.to(dev), got["lse"], got["entropy"], t.to(dev), torch.ones(3, device=dev),
                                       torch.ones(3, device=dev), softcap=softcap)
        # the only word there is has probability 1 (lse and entropy off by their bounds)
        assert (d[[0, 2]] == 0).all() and d[1].abs().max() <= 1e-4 and torch.isfinite(d).all()


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_and_infinity_stay_in_their_row(softcap, dtype):
    dev = device()
    c = make(6, 3001, dtype, 4)
    x, t = c["logits"].to(dev), c["targets"].abs().clamp(max=3000).to(dev)
    want = gl.token_logprobs(x, t, softcap=softcap, top=4)
    x[1, 5], x[4, 2999] = math.nan, math.inf
    got = gl.token_logprobs(x, t, softcap=softcap, top=4)
    bad = [1] if softcap else [1, 4]
    ok = [i for i in range(6) if i not in (1, 4)]
    for k in want:
        assert torch.equal(got[k][ok], want[k][ok]), k
        if k != "top_ids":
            assert torch.isnan(got[k][bad]).all(), k
    assert all(len(set(r)) == 4 and 0 <= min(r) and max(r) < 3001 for r in got["top_ids"].tolist())
    assert got["top_ids"][4, 0] == 2999
    d = gl.token_logprobs_backward(x, got["lse"], got["entropy"], t, c["d_l"].to(dev), c["d_h"].to(dev), softcap=softcap)
    assert torch.isnan(d[bad]).all() and torch.isfinite(d[ok]).all()


def test_rows_of_any_stride():
    dev = device()
    c = make(5, 1000, BF16, 9)
    wide = torch.full((5, 1235), 50.0, dtype=BF16, device=dev)
    wide[:, :1000] = c["logits"].to(dev)
    got = gl.token_logprobs(wide[:, :1000], c["targets"].to(dev), top=3)
    check(c, got, 0.0, 1.0, 3)
    out = torch.full((5, 1111), 9.0, dtype=BF16, device=dev)
    gl.token_logprobs_backward(wide[:, :1000], got["lse"], got["entropy"], c["targets"].to(dev), c["d_l"].to(dev),
                               out=out[:, :1000])
    check_gradient(c, out[:, :1000], True, False, 0.0, 1.0)
    assert (out[:, 1000:] == 9.0).all() and (wide[:, 1000:] == 50.0).all()


def test_far_logits():
    # sizes at which exponentials leave binary32 many times over
    dev = device()
    x = torch.tensor([[3e4, 0.0, -3e4, 2.9999e4], [-1e30, -1e30, -2e30, -1e30], [0.0, -500.0, -88.0, -120.0]])
    c = dict(logits=x, targets=torch.tensor([1, 0, 3]))
    check(c, gl.token_logprobs(x.to(dev), c["targets"].to(dev), top=4), 0.0, 1.0, 4)


def test_empty_batch_and_no_targets():
    dev = device()
    got = gl.token_logprobs(torch.empty(0, 50, device=dev), top=2)
    assert got["lse"].shape == (0,) and got["top_ids"].shape == (0, 2)
    x = make(3, 50, F32, 1)["logits"].to(dev)
    got = gl.token_logprobs(x)
    assert set(got) == {"lse", "entropy"}
    assert gl.token_logprobs_backward(torch.empty(0, 50, device=dev), *[torch.empty(0, device=dev)] * 2,
                                      d_entropy=torch.empty(0, device=dev)).shape == (0, 50)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 5000, 40000])
def test_masks_of_the_lowest_value(V, dtype):
    dev, low = device(), torch.finfo(dtype).min
    c = make(4, V, dtype, V)
    c["targets"] = torch.tensor([5, 3, 0, -1])
    c["logits"][0, ::2], c["logits"][1, 4:], c["logits"][2, :] = low, low, low
    for softcap in (0.0, 30.0, 500.0):
        for top in (0, 3):
            got = gl.token_logprobs(c["logits"].to(dev), c["targets"].to(dev), softcap=softcap, top=top)
            # (the bound grows with the largest |z|: the rows of ordinary ones alone, too)
            check(c, got, softcap, 1.0, top)
            keep = dict(logits=c["logits"][:1, 1::2].contiguous(), targets=torch.tensor([2]))
            if not softcap:
                check(keep, {k: got[k][:1] for k in ("lse", "entropy", "logprobs")}, 0.0, 1.0, 0)
            # a row of the lowest value only is uniform
            assert abs(got["logprobs"][2].item() + math.log(V)) <= 2e-5 * math.log(V)
            assert abs(got["entropy"][2].item() - math.log(V)) <= 2e-5 * math.log(V)


@pytest.mark.parametrize("softcap", [0.0, 30.0, 500.0])
def test_infinity_makes_its_row_nan(softcap):
    dev = device()
    x = make(3, 700, F32, 11)["logits"]
    x[1, 650] = math.inf
    for top in (0, 2):
        got = gl.token_logprobs(x.to(dev), torch.zeros(3, dtype=torch.int64, device=dev), softcap=softcap, top=top)
        for k in got:
            if k != "top_ids":
                assert torch.isnan(got[k][1]).all() and torch.isfinite(got[k][[0, 2]]).all(), k


@pytest.mark.parametrize("softcap,scale", [(30.0, 1.0), (300.0, 1.0), (30.0, 20.0), (0.0, 1.0)])
@pytest.mark.parametrize("T,V,top", [(1, 300000, 16), (2, 600001, 3), (1500, 9000, 16), (600, 17000, 2)])
def test_pieces_of_every_length(T, V, top, softcap, scale):
    # every number of steps a piece, joins of more pieces than threads, caps whose
    # exponentials need a maximum
    c = make(T, V, BF16, T, masked=0.01)
    dev = device()
    x, t = c["logits"].to(dev), c["targets"].to(dev)
    for k in (0, top):
        check(c, gl.token_logprobs(x, t, softcap=softcap, scale=scale, top=k), softcap, scale, k)

"""Scores of tokens and their gradient where z is large: rows of the type's
lowest value under a scale, logits with a common offset, and caps far above the
logits.

Tolerances count roundings of u = 2^-24, in nats.  Without a cap a word's
distance to its row's largest logit is one difference and two products (3 u of
it; past 104 nats a probability is 0), its exponential 4 u; a capped z past a cap
of 66 is off by 20 u of itself.  A thread adds V / 256 terms one by one, and the
joining of threads and pieces 64 more, u each, all of one sign.  The logarithm of
a sum adds 4 u of itself."""
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
MOST = torch.finfo(F32).max


def parts(r, softcap, scale):
    """Per row: the errors of a relative probability, of ln S and of the entropy."""
    V = r["z"].shape[1]
    z = torch.where(r["z"] > -math.inf, r["z"], 0.0)
    dist = (z.amax(1, keepdim=True) - z).clamp(max=104.0)
    dp = 2 * 20 * U * z.abs().amax(1) if softcap else 0 * z[:, 0]
    dp = dp + (3 * 104 + 4) * U
    p = torch.exp(r["logp"])
    ls = dp + (V / 256 + 64) * U + 4 * U * math.log(V + 1)
    return dp, ls, (1 + (p * dist).sum(1)) * (2 * dp + 2 * ls) + 4 * U * math.log(V + 1)


def level(x):
    """Each row less its largest logit, in 64 bits, which would lose ln S beside the
    logits themselves; without a cap everything but lse stays as it is."""
    return x.double() - x.double().amax(1, keepdim=True)


def check_gradient(x, t, d_l, d_h, got, softcap, scale):
    dtype, x = x.dtype, x if softcap else level(x)
    want, size = (ref.score_grad(x, t, d_l, d_h, softcap, scale, absolute=a) for a in (False, True))
    r = ref.score(x, None, softcap, scale)
    dp, ls, dh = parts(r, softcap, scale)
    rel = (2 * (dp + ls) + 8 * U)[:, None]
    tol = rel * size
    if softcap:      # z' = scale (1 - tanh^2), off by 100 u of scale
        tol = tol + 100 * U * size / (1 - torch.tanh(x.double() / softcap) ** 2).clamp(min=1e-30)
    if d_h is not None:   # a log probability's error, and the entropy's own
        tol = tol + scale * d_h.abs().double()[:, None] * torch.exp(r["logp"]) * 2 * (dp + ls + dh)[:, None]
    tol = tol + half_step(dtype) * (want.abs() + tol)
    least = sum(k * d.abs().double() for k, d in ((1, d_l), (104 + math.log(x.shape[1]), d_h)) if d is not None)
    tol = tol + 2.0 ** -126 * (1 + scale * least)[:, None]
    got = got.cpu().double()
    assert torch.isfinite(got).all()
    err = (got - want).abs()
    assert (err <= tol).all(), f"{(err - tol).max():.3e} over, at most {err.max():.3e} off, rows {(err > tol).any(1).nonzero()[:, 0].tolist()}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.5, 1.0, 1.25, 3.0])
@pytest.mark.parametrize("V", [5, 5000, 40000])
def test_rows_of_one_value_are_uniform(V, scale, dtype):
    info, dev = torch.finfo(dtype), device()
    values = [info.min, info.max, -1e30, 1e20, 0.0]
    x = torch.tensor(values, dtype=dtype)[:, None].repeat(1, V)
    t = torch.tensor([0, V - 1, 2, 3, -1])
    # a sum of V ones is exact; its logarithm, and a product
    tol, want = 8 * U * math.log(V), -math.log(V)
    for top in (0, 3):
        got = {k: v.cpu().double() for k, v in gl.token_logprobs(x.to(dev), t.to(dev), scale=scale, top=top).items()}
        assert ((got["logprobs"][:4] - want).abs() <= tol).all() and got["logprobs"][4] == 0
        assert ((got["entropy"] + want).abs() <= tol).all()
        lse = (x[:, 0].double() * scale - want).clamp(-MOST, MOST)
        assert ((got["lse"] - lse).abs() <= 4 * U * lse.abs() + tol).all()
        if top:
            assert (got["top_ids"] == torch.arange(3)).all() and ((got["top_logprobs"] - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1.0, 1.25])
@pytest.mark.parametrize("V", [40, 5000, 40000])
def test_masks_of_the_lowest_value_under_a_scale(V, scale, dtype):
    dev, low = device(), torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(3, V, generator=g) * 4).to(dtype)
    x[0, ::2], x[1, 4:], x[2, :] = low, low, low
    t = torch.tensor([5, 0, 7])
    got = gl.token_logprobs(x.to(dev), t.to(dev), scale=scale, top=4)
    kept = [x[0, 1::2], x[1, :4], x[2]]
    for i, row in enumerate(kept):
        r = ref.score(level(row[None]), torch.tensor([(2, 0, 7)[i]]), 0.0, scale)
        dp, ls, dh = parts(r, 0.0, scale)
        one = lambda k: got[k][i].cpu().double()
        assert (one("logprobs") - r["logprobs"][0]).abs() <= 2 * (dp + ls) + 4 * U * 40
        assert (one("entropy") - r["entropy"][0]).abs() <= dh
        assert torch.isfinite(got["top_logprobs"][i]).all()
    # a masked word's log probability: its distance, past binary32's range -infinity
    got = gl.token_logprobs(x.to(dev), torch.tensor([0, 4, 0], device=dev), scale=scale)["logprobs"].cpu().double()
    far = low * scale if abs(low * scale) <= MOST else -math.inf
    assert all(v == far or abs(v - far) <= 4 * U * abs(far) for v in got[:2].tolist())


# the sums of rows of 3 words or fewer pieces, of pieces, and of one piece a row
SIZES = [(6, 7), (5, 40003), (1100, 517)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1.0, 1.25])
@pytest.mark.parametrize("T,V", SIZES)
def test_gradient_of_rows_of_one_value(T, V, scale, dtype):
    info, dev = torch.finfo(dtype), device()
    g = torch.Generator().manual_seed(T)
    x = (torch.randn(T, V, generator=g) * 4).to(dtype)
    x[0], x[1], x[2, :] = info.min, info.max, -1e30
    x[3, ::2] = info.min
    t = torch.randint(-1, V, (T,), generator=g)
    t[:3] = torch.tensor([1, V - 1, 0])
    d_l, d_h = torch.randn(T, generator=g), torch.randn(T, generator=g)
    got = gl.token_logprobs(x.to(dev), t.to(dev), scale=scale)
    for a, b in ((d_l, None), (None, d_h), (d_l, d_h)):
        d = gl.token_logprobs_backward(x.to(dev), got["lse"], got["entropy"], t.to(dev), None if a is None else a.to(dev),
                                       None if b is None else b.to(dev), scale=scale)
        check_gradient(x, t, a, b, d, 0.0, scale)


@pytest.mark.parametrize("scale", [1.0, 0.7])
@pytest.mark.parametrize("offset", [300.0, 1e4, -1e4, 1e6])
@pytest.mark.parametrize("T,V", SIZES)
def test_gradient_of_logits_with_an_offset(T, V, offset, scale):
    dev, g = device(), torch.Generator().manual_seed(V)
    x = torch.randn(T, V, generator=g) * 4
    x[::3] += offset               # beside rows without one
    t = torch.randint(0, V, (T,), generator=g)
    d_l, d_h = torch.randn(T, generator=g), torch.randn(T, generator=g)
    dx, dt, da, db = x.to(dev), t.to(dev), d_l.to(dev), d_h.to(dev)
    got = gl.token_logprobs(dx, dt, scale=scale)
    d = gl.token_logprobs_backward(dx, got["lse"], got["entropy"], dt, da, db, scale=scale)
    check_gradient(x, t, d_l, d_h, d, 0.0, scale)
    # in the logits' place, and into rows that start elsewhere
    wide = torch.full((T, V + 5), 9.0, device=dev)
    gl.token_logprobs_backward(dx, got["lse"], got["entropy"], dt, da, db, scale=scale, out=wide[:, :V])
    assert torch.equal(wide[:, :V], d) and (wide[:, V:] == 9.0).all()
    gl.token_logprobs_backward(dx, got["lse"], got["entropy"], dt, da, db, scale=scale, out=dx)
    assert torch.equal(dx, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", SIZES)
def test_gradient_under_a_cap_past_every_sum(T, V, dtype):
    # words that lie further apart than any sum reaches, beside ordinary ones
    dev, g = device(), torch.Generator().manual_seed(V)
    x = (torch.randn(T, V, generator=g) * 4).to(dtype)
    x[2] = (torch.randn(V, generator=g) * 3e29).clamp(max=1.5e30).to(dtype)
    x[2, 5] = 2e30        # (the next one's tanh is 0.06 less: far from a tie in binary32)
    t = torch.randint(0, V, (T,), generator=g)
    t[2] = 5
    d_l, d_h = torch.randn(T, generator=g), torch.randn(T, generator=g)
    got = gl.token_logprobs(x.to(dev), t.to(dev), softcap=1e30)
    d = gl.token_logprobs_backward(x.to(dev), got["lse"], got["entropy"], t.to(dev), d_l.to(dev), d_h.to(dev), softcap=1e30)
    keep = torch.arange(T) != 2
    check_gradient(x[keep], t[keep], d_l[keep], d_h[keep], d[keep.to(dev)], 1e30, 1.0)
    # p is 1 for the largest word, and the gradient 0 but for a product's rounding
    assert got["logprobs"][2] == 0 and got["entropy"][2] == 0 and (d[2].abs() <= 4 * U * d_l[2].abs().item()).all()


def test_far_rows_in_a_graph():
    # captured once, replayed over rows that are near and far in turn
    dev, g = device(), torch.Generator().manual_seed(8)
    T, V = 5, 40003
    x = torch.randn(T, V, generator=g).to(dev) * 4
    t, d_l, d_h = (v.to(dev) for v in (torch.randint(0, V, (T,), generator=g), torch.randn(T, generator=g),
                                       torch.randn(T, generator=g)))

    def step(y):
        got = gl.token_logprobs(y, t)
        return gl.token_logprobs_backward(y, got["lse"], got["entropy"], t, d_l, d_h)

    held, graph = x.clone(), torch.cuda.CUDAGraph()
    step(held)
    with torch.cuda.graph(graph):
        out = step(held)
    for offsets in ([0] * 5, [1e4, 0, -1e5, 0, 300], [0, 1e6, 0, 0, 0], [0] * 5):
        held.copy_(x + torch.tensor(offsets, device=dev)[:, None])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(held))


@pytest.mark.parametrize("offset", [0.0, 300.0, -2000.0])
def test_entropy_gradient_of_a_shard(offset):
    # half of a vocabulary each, with the whole's lse and entropy (a target outside the
    # half has no gradient of its logprob, so that the entropy's is what can be cut)
    dev, g = device(), torch.Generator().manual_seed(9)
    T, V = 40, 9000
    x = torch.randn(T, V, generator=g) * 4 + offset
    d_h = torch.randn(T, generator=g)
    whole = gl.token_logprobs(x.to(dev))
    got = torch.cat([gl.token_logprobs_backward(h.contiguous().to(dev), whole["lse"], whole["entropy"], d_entropy=d_h.to(dev))
                     for h in x.split(V // 2, 1)], 1).cpu().double()
    want, size = (ref.score_grad(level(x), None, None, d_h, absolute=a) for a in (False, True))
    r = ref.score(level(x))
    dp, ls, dh = parts(r, 0.0, 1.0)
    dp = dp + U * ref.score(x)["lse"].abs()          # lse's own rounding
    tol = (2 * (dp + ls) + 8 * U)[:, None] * size
    tol = tol + d_h.abs().double()[:, None] * torch.exp(r["logp"]) * 2 * (dp + ls + dh)[:, None]
    assert ((got - want).abs() <= tol + U * want.abs() + 2.0 ** -120).all()

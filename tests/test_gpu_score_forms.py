"""The loops of the score kernels at the lengths at which they do their work: whole
steps four and two at a time, many of them a thread, pieces of four steps, rows of
every start.  The tolerances are test_gpu_score's; of its 300 u for a row's sums
64 are the logits of a thread, and longer chains add theirs (`chain`)."""
import math

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
import test_gpu_score as ts
from gpu_util import device

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(T, V, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(T, V, device="cuda").normal_(0, 4, generator=g)
    x[torch.rand(T, V, device="cuda", generator=g) < 0.02] = -math.inf
    t = torch.randint(0, V, (T,), device="cuda", generator=g)
    d = [torch.empty(T, device="cuda").normal_(generator=g) for _ in range(2)]
    return dict(logits=x.to(dtype), targets=t, d_l=d[0], d_h=d[1])


def rows_of(c, rows):
    return {k: v[rows].cpu() for k, v in c.items()}


def sample(T):
    """Rows that start at every place of 16 bytes (of an odd length), first and last."""
    return sorted(set(range(9)) | set(range(T // 2, T // 2 + 8)) | {T - 2, T - 1})


def check(c, got, softcap, scale, top, chain):
    """As test_gpu_score's, with a thread's chain of additions: u each, twice in
    the entropy, whose terms are p (m - z)."""
    r = ref.score(c["logits"], c["targets"], softcap, scale, top)
    dz, dp, dl, lse = ts.bounds(r, softcap, scale)
    dl = dl + chain * ref.U
    ts.near(got["lse"], r["lse"], dl, "lse")
    p = torch.exp(r["logp"])
    spread = torch.where(p > 0, p * (r["z"].amax(1)[:, None] - r["z"]), 0.0).sum(1)
    z = torch.where(r["z"] > -math.inf, r["z"], 0.0).abs().amax(1)
    # (under a small cap the second sum is one of p r, times 2 cap, beside the first
    # times cap)
    spread = spread + (3 * softcap * scale if 0 < softcap * scale <= 35 else 0.0)
    ts.near(got["entropy"], r["entropy"], (1 + spread) * (2 * dp + (600 + 2 * chain) * ref.U) + 4 * ref.U * lse, "entropy")
    ts.near(got["logprobs"], r["logprobs"], dz + dl + 8 * ref.U * (lse + z), "logprobs")
    if top:
        assert torch.equal(got["top_ids"].cpu().long(), r["top_ids"])
        ts.near(got["top_logprobs"], r["top_logprobs"], (dz + dl + 8 * ref.U * (lse + z))[:, None], "top")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softcap,scale", [(0.0, 1.0), (30.0, 1.0), (300.0, 1.0)])
@pytest.mark.parametrize("T,V", [(1100, 20001), (1100, 100003), (300, 30001)])
def test_long_rows(T, V, softcap, scale, dtype):
    c = make(T, V, dtype, V)
    rows = sample(T)
    few, at = rows_of(c, rows), torch.tensor(rows, device="cuda")
    for top in (0, 2):
        got = gl.token_logprobs(c["logits"], c["targets"], softcap=softcap, scale=scale, top=top)
        check(few, {k: v[at] for k, v in got.items()}, softcap, scale, top, V / 256)
    args = (got["lse"], got["entropy"], c["targets"], c["d_l"], c["d_h"])
    d = gl.token_logprobs_backward(c["logits"], *args, softcap=softcap, scale=scale)
    ts.check_gradient(few, d[at], True, True, softcap, scale)
    # targets at every place of an unrolled step, and at a row's first and last word
    few["targets"] = torch.tensor([(0, 1, V - 1, V - 2, 2048, 4095, 4096, 8191)[i % 8] for i in range(len(rows))])
    t = c["targets"].clone()
    t[at] = few["targets"].cuda()
    e = gl.token_logprobs_backward(c["logits"], *args[:2], t, c["d_l"], None, softcap=softcap, scale=scale)
    ts.check_gradient(few, e[at], True, False, softcap, scale)
    # rows of the output that start elsewhere, and the logits' own place: the same bits
    wide = torch.full((T, V + 3), 9.0, dtype=dtype, device="cuda")
    gl.token_logprobs_backward(c["logits"], *args, softcap=softcap, scale=scale, out=wide[:, :V])
    assert torch.equal(wide[:, :V], d) and (wide[:, V:] == 9.0).all()
    assert gl.token_logprobs_backward(c["logits"], *args, softcap=softcap, scale=scale, out=c["logits"]) is c["logits"]
    assert torch.equal(c["logits"], d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softcap", [0.0, 30.0, 300.0])
@pytest.mark.parametrize("T,V,top", [(300, 30001, 16), (300, 30001, 1), (150, 60003, 5), (2100, 20001, 16)])
def test_alternatives_of_pieces_of_four_and_eight_steps(T, V, top, softcap, dtype):
    c = make(T, V, dtype, T + V)
    rows = sample(T)
    got = gl.token_logprobs(c["logits"], c["targets"], softcap=softcap, top=top)
    check(rows_of(c, rows), {k: v[rows] for k, v in got.items()}, softcap, 1.0, top, 0)


@pytest.mark.parametrize("softcap", [0.0, 30.0, 300.0])
def test_maximum_that_rises_along_a_row(softcap):
    # the largest logit last: every step raises the maximum
    T, V = 1030, 50021
    x = (torch.linspace(-20, 20, V, device="cuda")[None] + torch.arange(T, device="cuda")[:, None] / T).to(BF16)
    c = dict(logits=x, targets=torch.arange(T, device="cuda"), d_l=torch.ones(T, device="cuda"), d_h=torch.ones(T, device="cuda"))
    rows = sample(T)
    got = gl.token_logprobs(x, c["targets"], softcap=softcap)
    check(rows_of(c, rows), {k: v[rows] for k, v in got.items()}, softcap, 1.0, 0, V / 256)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("words", [1, 3, 15, 16, 50, 700])
def test_alternatives_of_rows_with_few_words(words, dtype):
    # scattered words that a grammar leaves
    T, V = 30, 50001
    g = torch.Generator().manual_seed(words)
    x = torch.full((T, V), -math.inf)
    for i in range(T):
        x[i, torch.randperm(V, generator=g)[:words]] = torch.randn(words, generator=g) * 4
    c = dict(logits=x.to(dtype), targets=torch.randint(0, V, (T,), generator=g))
    for softcap in (0.0, 30.0):
        got = gl.token_logprobs(c["logits"].to(device()), c["targets"].to(device()), softcap=softcap, top=16)
        check(c, got, softcap, 1.0, 16, 0)

"""Norms and rotation of attention heads (beam_moe_qk_norm_rope and its
gradients) on the GPU against the 64-bit formulas.

Tolerances count roundings of u = 2^-24.  A head's sum of squares is off by at
most 14 u (8 in its lane, 5 between lanes, the square), so its inverse root by
10; two products make 12.  An angle is off by 0.4 u (what is left of a quarter
turn, rounded) plus its position's part of binary64, its sine and cosine by 4
more, and a turned value adds three operations: 20 u of the terms' absolute
values.  The temperature's power is off by its exponent times 3 u and 4 more.
KAPPA = 48 covers these.  A gradient passes through the turn, the temperature
and the norm's mean (another 14 u and what its terms carry): 4 KAPPA.  Weights'
gradients add their terms one by one: a lane's tokens and heads, then the lanes
and workgroups.  Every output is rounded once more to its type (half its eps)."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
from gpu_util import device

pytestmark = pytest.mark.gpu

KAPPA = 48
EPS = 1e-6
BF16, F32 = torch.bfloat16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, tol, what):
    assert got.shape == want.shape, what
    assert torch.isfinite(got.float()).all(), what
    err = (got.cpu().double() - want).abs()
    assert (err <= tol).all(), f"{what}: {(err - tol).max():.3e} over, at most {err.max():.3e} off"


def make(T, Hq, Hkv, D, dtype, rot, seed, far=4096):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(dtype)
    c = dict(qkv=qkv, q_weight=1 + torch.randn(D, generator=g) / 10, k_weight=1 + torch.randn(D, generator=g) / 10,
             positions=torch.randint(0, far, (T,), generator=g, dtype=torch.int32),
             d_q=torch.randn(T, Hq, D, generator=g).to(dtype), d_k=torch.randn(T, Hkv, D, generator=g).to(dtype))
    c["inv_freq"] = gl.rope_frequencies(rot, 1e4, "cpu") if rot else None
    return c


def heads(qkv, Hq, Hkv, D):
    T = qkv.shape[0]
    return (qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
            qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))


def on(dev, c):
    return {k: v.to(dev) if torch.is_tensor(v) else v for k, v in c.items()}


def check_forward(c, x, w, got, interleaved, temp, dtype, what, eps=EPS):
    y, size = ref.rope(x, w, c["positions"], c["inv_freq"], interleaved, eps, temp)
    # the angle's part of binary64
    far = c["positions"].abs().max().double() * 2.0 ** -52 if c["inv_freq"] is not None else 0.0
    tol = (KAPPA * ref.U + far) * size
    within(got, y, tol + half_step(dtype) * (y.abs() + tol), what)


def check_backward(c, x, w, dy, got, got_w, interleaved, temp, dtype, what, eps=EPS):
    args = (dy, x, w, c["positions"], c["inv_freq"], interleaved, eps, temp)
    (dx, dw), (sx, sw) = ref.rope_grad(*args), ref.rope_grad(*args, absolute=True)
    far = c["positions"].abs().max().double() * 2.0 ** -52 if c["inv_freq"] is not None else 0.0
    tol = (4 * KAPPA * ref.U + far) * sx
    within(got, dx, tol + half_step(dtype) * (dx.abs() + tol), "d_" + what)
    T, H, D = x.shape
    adds = -(-T // min(1024 * 4, 4 * -(-T // 4))) * H + 4 * 64 + 64 + 16
    within(got_w, dw, (4 * KAPPA + adds) * ref.U * sw, f"d_{what}_weight")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,temp", [
    (1, 48, 8, 128, 128, False, None), (5, 48, 8, 128, 0, False, (2048.0, 0.1)), (3, 4, 2, 64, 32, True, None),
    (7, 3, 1, 256, 256, False, None), (2, 1, 1, 8, 0, False, None), (33, 6, 3, 16, 16, False, (100.0, -1.5)),
    (4, 5, 5, 80, 64, True, (7.5, 2.0)), (9, 2, 1, 96, 32, False, None), (70, 7, 2, 128, 64, False, None),
    (2, 9, 9, 24, 16, True, None), (300, 2, 1, 32, 32, False, None), (2, 16, 1, 200, 192, False, None)])
def test_forward_and_gradients(T, Hq, Hkv, D, rot, interleaved, temp, dtype):
    c = make(T, Hq, Hkv, D, dtype, rot, T + D)
    dc = on(device(), c)
    args = dict(positions=dc["positions"], inv_freq=dc["inv_freq"], interleaved=interleaved, eps=EPS, temperature=temp)
    dq, dk, _ = heads(dc["qkv"], Hq, Hkv, D)
    q, k, _ = heads(c["qkv"], Hq, Hkv, D)
    yq, yk = gl.qk_norm_rope(dq, dk, dc["q_weight"], dc["k_weight"], **args)
    check_forward(c, q, c["q_weight"], yq, interleaved, temp, dtype, "q")
    check_forward(c, k, c["k_weight"], yk, interleaved, None, dtype, "k")
    got = gl.qk_norm_rope_backward(dc["d_q"], dc["d_k"], dq, dk, dc["q_weight"], dc["k_weight"], **args)
    check_backward(c, q, c["q_weight"], c["d_q"], got["d_q"], got["d_q_weight"], interleaved, temp, dtype, "q")
    check_backward(c, k, c["k_weight"], c["d_k"], got["d_k"], got["d_k_weight"], interleaved, None, dtype, "k")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_tokens(dtype):
    # more tokens than the gradients' workgroups take at once
    T, Hq, Hkv, D = 4500, 3, 1, 64
    c = make(T, Hq, Hkv, D, dtype, 64, 3)
    dc = on(device(), c)
    args = dict(positions=dc["positions"], inv_freq=dc["inv_freq"], eps=EPS)
    q, k, _ = heads(c["qkv"], Hq, Hkv, D)
    dq, dk, _ = heads(dc["qkv"], Hq, Hkv, D)
    yq, _ = gl.qk_norm_rope(dq, dk, dc["q_weight"], dc["k_weight"], **args)
    check_forward(c, q, c["q_weight"], yq, False, None, dtype, "q")
    got = gl.qk_norm_rope_backward(dc["d_q"], dc["d_k"], dq, dk, dc["q_weight"], dc["k_weight"], **args)
    again = gl.qk_norm_rope_backward(dc["d_q"], dc["d_k"], dq, dk, dc["q_weight"], dc["k_weight"], **args)
    assert all(torch.equal(got[n], again[n]) for n in got)
    check_backward(c, q, c["q_weight"], c["d_q"], got["d_q"], got["d_q_weight"], False, None, dtype, "q")
    check_backward(c, k, c["k_weight"], c["d_k"], got["d_k"], got["d_k_weight"], False, None, dtype, "k")


def test_far_positions():
    # angles near 2^30 radians, and positions on both sides of 0
    c = make(6, 2, 1, 128, F32, 128, 4)
    c["positions"] = torch.tensor([0, 1, (1 << 20) + 1, (1 << 30) + 3, (1 << 31) - 1, -5], dtype=torch.int32)
    dc = on(device(), c)
    q, k, _ = heads(c["qkv"], 2, 1, 128)
    dq, dk, _ = heads(dc["qkv"], 2, 1, 128)
    y, _ = gl.qk_norm_rope(dq, dk, dc["q_weight"], dc["k_weight"], dc["positions"], dc["inv_freq"], eps=EPS)
    for i in range(6):
        one = dict(c, positions=c["positions"][i:i + 1])
        check_forward(one, q[i:i + 1], c["q_weight"], y[i:i + 1], False, None, F32, f"token {i}")


@pytest.mark.parametrize("scale", [0.0, 1e-18, 1e18])
def test_sizes_of_values(scale):
    # rows of zeros, and squares at the ends of binary32
    c = make(4, 2, 1, 64, F32, 64, 5)
    c["qkv"] = c["qkv"] * scale
    dc = on(device(), c)
    q, k, _ = heads(c["qkv"], 2, 1, 64)
    dq, dk, _ = heads(dc["qkv"], 2, 1, 64)
    y, _ = gl.qk_norm_rope(dq, dk, dc["q_weight"], dc["k_weight"], dc["positions"], dc["inv_freq"], eps=EPS)
    check_forward(c, q, c["q_weight"], y, False, None, F32, "q")


def test_nan_stays_in_its_head():
    c = on(device(), make(3, 4, 2, 64, BF16, 64, 6))
    args = (c["q_weight"], c["k_weight"], c["positions"], c["inv_freq"])
    q, k, _ = heads(c["qkv"], 4, 2, 64)
    want, _ = gl.qk_norm_rope(q, k, *args)
    for bad in (float("nan"), float("inf")):
        x = c["qkv"].clone()
        q2, k2, _ = heads(x, 4, 2, 64)
        q2[1, 2, 7] = bad
        y, _ = gl.qk_norm_rope(q2, k2, *args)
        assert not torch.isfinite(y[1, 2].float()).all()
        y[1, 2] = want[1, 2]
        assert torch.equal(y, want)


def cache(g, pages, page, Hkv, D, dtype, layout):
    """(k_cache, v_cache) [pages, page, Hkv, D] of a layout of memory."""
    n = lambda *s: torch.randn(*s, generator=g).to(dtype)
    if layout == "tokens":
        return n(pages, page, Hkv, D), n(pages, page, Hkv, D)
    if layout == "heads":               # a head's tokens together
        return n(pages, Hkv, page, D).transpose(1, 2), n(pages, Hkv, page, D).transpose(1, 2)
    both = n(pages, page, 2, Hkv, D)    # keys and values of a token together
    return both[:, :, 0], both[:, :, 1]


def move(dev, x):
    """To the GPU with its strides."""
    base = x._base if x._base is not None else x
    return base.to(dev).as_strided(x.shape, x.stride(), x.storage_offset())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
@pytest.mark.parametrize("T,page,D,rot", [(1, 16, 128, 128), (40, 1, 64, 0), (129, 32, 80, 16), (6, 8, 256, 256)])
def test_into_the_cache(T, page, D, rot, layout, dtype):
    Hq, Hkv, seqs, cols, pages = 4, 2, 5, 6, 40
    g = torch.Generator().manual_seed(T)
    c = make(T, Hq, Hkv, D, dtype, rot, T)
    tables = torch.randperm(pages, generator=g)[:seqs * cols].to(torch.int32).view(seqs, cols)
    tables[1, 2], tables[2, 0], tables[3, 1] = -1, pages, 1 << 30      # no pages
    # different places; some without a page, past the table, of no sequence
    spots = torch.randperm(seqs * (cols + 1) * page, generator=g)[:T]
    T = len(spots)
    c = {k: v[:T] if k in ("qkv", "d_q", "d_k") else v for k, v in c.items()}
    c["positions"] = (spots % ((cols + 1) * page)).to(torch.int32)
    rows = (spots // ((cols + 1) * page)).to(torch.int32)
    if T > 4:
        c["positions"][0], rows[1], rows[2], rows[3] = -1, -1, seqs, 1 << 30
    kc, vc = cache(g, pages, page, Hkv, D, dtype, layout)
    dev, dc = device(), on(device(), c)
    dkc, dvc = (move(dev, kc), move(dev, vc))
    before_k, before_v = dkc.clone(), dvc.clone()
    q, k, v = heads(dc["qkv"], Hq, Hkv, D)
    args = (dc["q_weight"], dc["k_weight"], dc["positions"], dc["inv_freq"])
    wq, wk = gl.qk_norm_rope(q, k, *args)
    yq, yk = gl.qk_norm_rope(q, k, *args, v=v, k_cache=dkc, v_cache=dvc, tables=tables.to(dev), rows=rows.to(dev),
                             with_k=True)
    assert torch.equal(yq, wq) and torch.equal(yk, wk)
    for t in range(T):
        r, p = int(rows[t]), int(c["positions"][t])
        if not (0 <= r < seqs and 0 <= p < cols * page and 0 <= int(tables[r, p // page]) < pages):
            continue
        before_k[int(tables[r, p // page]), p % page] = wk[t]
        before_v[int(tables[r, p // page]), p % page] = v[t]
    assert torch.equal(dkc, before_k) and torch.equal(dvc, before_v)
    # without with_k the same, and tokens in the rows' own order
    kc2, vc2 = before_k.clone(), before_v.clone()
    y2, none = gl.qk_norm_rope(q, k, *args, v=v, k_cache=kc2, v_cache=vc2, tables=tables.to(dev), rows=rows.to(dev))
    assert none is None and torch.equal(y2, wq) and torch.equal(kc2, before_k) and torch.equal(vc2, before_v)


def test_a_token_of_each_sequence():
    c = on(device(), make(3, 2, 1, 64, BF16, 64, 8, far=8))
    q, k, v = heads(c["qkv"], 2, 1, 64)
    dev = device()
    kc, vc = torch.zeros(6, 4, 1, 64, dtype=BF16, device=dev), torch.zeros(6, 4, 1, 64, dtype=BF16, device=dev)
    tables = torch.tensor([[5, 0], [1, 2], [3, 4]], dtype=torch.int32, device=dev)
    args = dict(positions=c["positions"], inv_freq=c["inv_freq"], v=v, tables=tables)
    gl.qk_norm_rope(q, k, c["q_weight"], c["k_weight"], k_cache=kc, v_cache=vc, **args)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    gl.qk_norm_rope(q, k, c["q_weight"], c["k_weight"], k_cache=kc2, v_cache=vc2,
                    rows=torch.arange(3, dtype=torch.int32, device=dev), **args)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2) and (kc != 0).any()


def test_empty_batch():
    dev = device()
    e = torch.empty(0, 2, 64, dtype=BF16, device=dev)
    w = torch.ones(64, device=dev)
    q, k = gl.qk_norm_rope(e, e, w, w)
    assert q.shape == k.shape == (0, 2, 64)
    got = gl.qk_norm_rope_backward(e, e, e, e, w, w)
    assert (got["d_q_weight"] == 0).all() and (got["d_k_weight"] == 0).all()

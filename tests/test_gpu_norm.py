"""The step between two blocks (beam_moe_norm_residual and its gradients) on
the GPU against the 64-bit formulas.

Tolerances count roundings of u = 2^-24.  A row's sum of squares (all terms
positive) is off by at most n u with n the additions on a value's way to the
total: at most 16 in its thread, 6 in its wave, 16 over the waves; its inverse
root by half of that and three more.  The gate's sigmoid is off by (|g| + 8) u.
With KAPPA = 16 + 6 + 16 + 30 covering one chain of these and the products
around it, every term of a result is off by at most (KAPPA + |g|) u of its
absolute value, or twice that where it passes through both norms, and the
output is rounded once more to its type (half its eps)."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import layer_ref as ref
from gpu_util import device

pytestmark = pytest.mark.gpu

KAPPA = 68
EPS = 1e-6
ALPHA, BETA = 0.98828125, 0.1640625          # exact in binary32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make(T, H, dtype, gate, after, seed):
    g = torch.Generator().manual_seed(seed)
    c = {"residual": torch.randn(T, H, generator=g), "pre": 1 + torch.randn(H, generator=g) / 10,
         "o": None, "post": None, "gate": None}
    if after:
        c["o"] = (torch.randn(T, H, generator=g) * 0.5).to(dtype)
        c["post"] = 1 + torch.randn(H, generator=g) / 10
        if gate:
            c["gate"] = (torch.randn(T, H if gate == "channel" else 1, generator=g) * 2).to(dtype)
    c["d_r"], c["d_x"] = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g).to(dtype)
    return c


def on(dev, c):
    return {k: None if v is None else v.to(dev) for k, v in c.items()}


def kw(c, pre=True, eps=EPS):
    return dict(o=c["o"], post_weight=c["post"], gate=c["gate"], pre_weight=c["pre"] if pre else None,
                eps=eps, alpha=ALPHA, beta=BETA)


def within(got, want, tol, what):
    err = (got.cpu().double() - want).abs()
    assert torch.isfinite(got.float()).all(), what
    assert (err <= tol).all(), f"{what}: {(err - tol).max():.3e} over, at most {err.max():.3e} off"


def check_forward(c, dtype, r, x, eps=EPS):
    rp, xx, y, g = ref.norm_step(c["residual"], c["o"], c["post"], c["gate"], c["pre"], eps, ALPHA, BETA)
    gmax = 0.0 if c["gate"] is None else c["gate"].double().abs().amax().item()
    term = torch.zeros_like(rp) if y is None else (BETA * g * y).abs()
    d_r = ref.U * (rp.abs() + (KAPPA + gmax) * term)
    if y is None:
        d_r.zero_()
    within(r, rp, d_r, "residual")
    if x is not None:
        inv = 1 / torch.sqrt((rp * rp).mean(1, keepdim=True) + eps)
        hat = (rp * inv).abs()
        # the stream's own error, directly and through the norm
        d_x = c["pre"].double().abs() * inv * (d_r + hat * (hat * d_r).mean(1, keepdim=True))
        d_x = d_x + KAPPA * ref.U * xx.abs()
        within(x, xx, d_x + half_step(dtype) * (xx.abs() + d_x), "x")
    return rp, xx


def check_backward(c, dtype, r, got, use_r=True, use_x=True, eps=EPS):
    args = (r.cpu(), c["d_r"] if use_r else None, c["d_x"] if use_x else None, c["o"], c["post"], c["gate"],
            c["pre"], eps, ALPHA, BETA)
    want = ref.norm_step_grad(*args)
    size = ref.norm_step_grad(*args, absolute=True)
    gmax = 0.0 if c["gate"] is None else c["gate"].double().abs().amax().item()
    T = c["residual"].shape[0]
    assert set(got) == set(want)
    for k, w in want.items():
        kappa = 2 * (KAPPA + 2 * gmax)
        if k in ("d_pre_weight", "d_post_weight"):
            kappa += -(-T // 512) + 512 / 4 + 4      # additions over the tokens
        if k == "d_gate" and c["gate"].shape[1] == 1:
            kappa += 40                              # and over the row
        tol = kappa * ref.U * size[k]
        if k in ("d_o", "d_gate"):
            tol = tol + half_step(dtype) * (w.abs() + tol)
        within(got[k], w, tol, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("T,H", [(1, 5120), (3, 8), (5, 1), (2, 7), (33, 128), (1000, 264), (7, 1001), (4, 4099),
                                 (2, 8200), (3, 16384), (2, 16383), (1, 64)])
def test_step_and_gradients(T, H, gate, dtype):
    c = make(T, H, dtype, gate, True, 10 * T + H)
    dc = on(device(), c)
    # a row of one channel is its own norm: with eps 1e-6 the gradient of o is
    # a difference of near-equal terms, which the bound's absolute values hold
    r, x = gl.norm_residual(dc["residual"], **kw(dc))
    check_forward(c, dtype, r, x)
    got = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    check_backward(c, dtype, r, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 5120), (600, 96), (3, 51)])
def test_first_norm_alone(T, H, dtype):
    c = make(T, H, dtype, None, False, T + H)
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], pre_weight=dc["pre"], eps=EPS, dtype=dtype)
    assert r.data_ptr() == dc["residual"].data_ptr()
    check_forward(c, dtype, r, x)
    for use_r in (True, False):
        got = gl.norm_residual_backward(r, dc["d_r"] if use_r else None, dc["d_x"], pre_weight=dc["pre"],
                                        eps=EPS)
        check_backward(c, dtype, r, got, use_r=use_r)


@pytest.mark.parametrize("H", [512, 513])
def test_last_norm_alone(H):
    c = make(20, H, torch.bfloat16, "channel", True, 77)
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], **kw(dc, pre=False))
    assert x is None
    check_forward(c, torch.bfloat16, r, None)
    got = gl.norm_residual_backward(r, dc["d_r"], None, **kw(dc, pre=False))
    check_backward(c, torch.bfloat16, r, got, use_x=False)
    got = gl.norm_residual_backward(r, None, dc["d_x"], **kw(dc))
    check_backward(c, torch.bfloat16, r, got, use_r=False)


def test_agrees_with_the_blocks_own_epilogue():
    # forward_residual's norm and stream on the same block output (bf16 here,
    # fp32 inside its combine: half a bf16 step of o, through the norm)
    import synth
    from gpu_util import desc_for
    sh = synth.small_shape()
    w = synth.WORKLOADS["prefill4k"]
    inp = synth.make_inputs(w, device=device(), tokens=50, shape=sh, seed=9)
    d = desc_for(w, sh)
    weight = torch.rand(sh.hidden, device=inp.x.device) + 0.5
    r0 = torch.randn(50, sh.hidden, device=inp.x.device)
    fused = r0.clone()
    out = torch.empty_like(inp.x)
    gl.forward_residual(d, inp.x, inp.w_router, inp.bias, inp.w_gate_up, inp.w_down, weight, EPS, 7, fused,
                        out=out)
    alpha, beta = gl.residual_scale(7)
    r, _ = gl.norm_residual(r0, o=out, post_weight=weight, eps=EPS, alpha=alpha, beta=beta)
    y = ref.norm_step(r0.cpu(), out.cpu(), weight.cpu(), None, None, EPS, alpha, beta)[2].abs()
    tol = beta * (2.0 ** -8 * 2 * y + 2.0 ** -8 * y.mean()) + 1e-5
    assert ((r - fused).abs().cpu().double() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("after", [True, False])
@pytest.mark.parametrize("T,H", [(1, 128), (37, 5120), (5, 8320)])
def test_codes(T, H, after, dtype):
    c = make(T, H, dtype, "channel", after, 3 * T + H)
    c["residual"][0, :128] = 0.0
    if after:
        c["o"][0, :128] = 0.0                         # an all-zero block: scale 1
    dc = on(device(), c)
    args = kw(dc) if after else dict(pre_weight=dc["pre"], eps=EPS, dtype=dtype)
    r, q, s, x = gl.norm_residual_e4m3(dc["residual"], with_x=True, **args)
    r2, q2, s2 = gl.norm_residual_e4m3(dc["residual"], **args)
    assert torch.equal(r, r2) and torch.equal(q, q2) and torch.equal(s, s2)
    _, x2 = gl.norm_residual(dc["residual"], **args)
    assert torch.equal(x, x2)
    check_forward(c, dtype, r, x)
    if dtype == torch.float32:                        # x unrounded: the recipe bit for bit
        q3, s3 = gl.quant_e4m3(x)
        assert torch.equal(q, q3) and torch.equal(s, s3)
    # the codes stand for x within half an e4m3 step and the smallest code's
    xf = x.float().view(T, -1, 128)
    back = q.view(torch.float8_e4m3fn).float().view(T, -1, 128) * s[..., None]
    assert ((back - xf).abs() <= xf.abs() * (2.0 ** -4 + 2.0 ** -7) + s[..., None] * 2.0 ** -10).all()
    assert s[0, 0] == 1.0 and (q[0, :128] == 0).all()


def test_zero_rows_and_large_values():
    # a row of zeros, one of values whose squares underflow, and large ones
    c = make(4, 256, torch.bfloat16, "token", True, 5)
    for k in ("residual", "o"):
        c[k][0] = 0.0
        c[k][1] *= 1e-30
        c[k][2] *= 1e16
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], **kw(dc))
    check_forward(c, torch.bfloat16, r, x)
    got = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    check_backward(c, torch.bfloat16, r, got)
    # gates far out: sigmoid 0 and 1
    c["gate"] = torch.tensor([[-1e4], [1e4], [-90.0], [90.0]]).to(torch.bfloat16)
    for k in ("residual", "o"):
        c[k] = torch.randn(4, 256).to(c[k].dtype)
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], **kw(dc))
    got = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    assert all(torch.isfinite(v).all() for v in got.values())
    assert torch.equal(r[0], ALPHA * dc["residual"][0])
    assert got["d_gate"][0] == 0 and got["d_gate"][1] == 0


def test_in_place_and_deterministic():
    c = make(700, 640, torch.bfloat16, "channel", True, 21)
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], **kw(dc))
    a = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    b = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc), workspace=gl.Workspace(device()))
    assert all(torch.equal(a[k], b[k]) for k in a)
    stream = dc["residual"].clone()
    r2, x2 = gl.norm_residual(stream, residual_out=stream, **kw(dc))
    assert r2.data_ptr() == stream.data_ptr() and torch.equal(r2, r) and torch.equal(x2, x)
    # rows are independent: a slice of the batch gives the same bits
    # (batches of 1,024 tokens on split a row over fewer threads)
    r3, x3 = gl.norm_residual(dc["residual"][40:57].contiguous(), o=dc["o"][40:57].contiguous(),
                              post_weight=dc["post"], gate=dc["gate"][40:57].contiguous(),
                              pre_weight=dc["pre"], eps=EPS, alpha=ALPHA, beta=BETA)
    assert torch.equal(r3, r[40:57]) and torch.equal(x3, x[40:57])


def test_empty_batch():
    c = make(0, 256, torch.bfloat16, "channel", True, 1)
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], **kw(dc))
    assert r.shape == (0, 256) and x.shape == (0, 256)
    got = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    assert got["d_o"].shape == (0, 256)
    assert (got["d_pre_weight"] == 0).all() and (got["d_post_weight"] == 0).all()


def test_long_stream_offsets():
    # element offsets past 2^31: the last rows equal the same rows alone
    T, H = 140000, 16384
    dev = device()
    res = torch.zeros(T, H, device=dev)
    last = torch.randn(5, H, device=dev)
    res[-5:] = last
    pre = torch.ones(H, device=dev)
    _, q, s = gl.norm_residual_e4m3(res, pre_weight=pre, eps=EPS)
    _, q2, s2 = gl.norm_residual_e4m3(last, pre_weight=pre, eps=EPS)
    assert torch.equal(q[-5:], q2) and torch.equal(s[-5:], s2)


def test_captured_with_work_between_replays():
    dev = device()
    c = on(dev, make(300, 1024, torch.bfloat16, "token", True, 31))
    other = on(dev, make(300, 1024, torch.bfloat16, "token", True, 32))
    ws = gl.Workspace(dev)

    def step(v):
        r, x = gl.norm_residual(v["residual"], **kw(v))
        return dict(gl.norm_residual_backward(r, v["d_r"], v["d_x"], **kw(v), workspace=ws), r=r, x=x)

    want, want_other = step(c), step(other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step(c)
    side.synchronize()
    assert all(torch.equal(on_side[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(c)
    for _ in range(3):
        for v in got.values():
            v.fill_(float("nan"))
        between = step(other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert all(torch.equal(between[k], want_other[k]) for k in want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("T,H", [(9, 9), (9, 10), (9, 11), (8, 12), (9, 13), (9, 14), (9, 15), (5, 17), (3, 5119),
                                 (2, 8191), (2, 8193), (1500, 31), (2100, 70)])
def test_rows_that_end_inside_a_chunk(T, H, gate, dtype):
    # every odd start of a row and every length of its last chunk of 8
    c = make(T, H, dtype, gate, True, 3 * T + H)
    dc = on(device(), c)
    buf = torch.full((T + 1, H), 7.0, device=device())
    r, x = gl.norm_residual(dc["residual"], residual_out=buf[:T], **kw(dc))
    assert r.data_ptr() == buf.data_ptr() and (buf[T] == 7.0).all()
    check_forward(c, dtype, r, x)
    got = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    check_backward(c, dtype, r, got)
    for use in (dict(d_x=dc["d_x"]), dict(d_residual_out=dc["d_r"])):
        part = gl.norm_residual_backward(r, **use, **kw(dc))
        check_backward(c, dtype, r, part, use_r="d_residual_out" in use, use_x="d_x" in use)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(4000, 31), (3000, 519), (2000, 5119), (600, 12345)])
def test_odd_rows_in_place(T, H, dtype):
    # threads of two waves share columns at a row's end: each has to have read
    # them before the other writes
    c = make(T, H, dtype, "token", True, H)
    dc = on(device(), c)
    r, x = gl.norm_residual(dc["residual"], **kw(dc))
    want = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **kw(dc))
    for _ in range(3):
        stream = dc["residual"].clone()
        _, x2 = gl.norm_residual(stream, residual_out=stream, **kw(dc))
        assert torch.equal(stream, r) and torch.equal(x2, x)
        d = dc["d_r"].clone()
        got = backward_in_place(r, d, dc)
        assert torch.equal(d, want["d_residual"])
        assert all(torch.equal(v, want[k]) for k, v in got.items())


def backward_in_place(r, d, dc):
    """norm_residual_backward through the C ABI with d_residual = d_residual_out."""
    import ctypes
    T, H = r.shape
    out = {k: torch.empty_like(v) for k, v in (("d_o", dc["o"]), ("d_gate", dc["gate"]), ("d_pre_weight", dc["pre"]),
                                               ("d_post_weight", dc["post"]))}
    n = ctypes.c_size_t()
    assert gl.lib().beam_moe_norm_residual_workspace_bytes(T, H, ctypes.byref(n)) == gl.OK
    ws = torch.empty(n.value, dtype=torch.uint8, device=r.device)
    st = gl.lib().beam_moe_norm_residual_backward(
        T, H, gl.BF16 if dc["o"].dtype == torch.bfloat16 else gl.F32, dc["o"].data_ptr(), dc["post"].data_ptr(),
        dc["gate"].data_ptr(), 1, dc["pre"].data_ptr(), EPS, ALPHA, BETA, r.data_ptr(), d.data_ptr(),
        dc["d_x"].data_ptr(), d.data_ptr(), out["d_o"].data_ptr(), out["d_gate"].data_ptr(),
        out["d_pre_weight"].data_ptr(), out["d_post_weight"].data_ptr(), ws.data_ptr(), n.value,
        torch.cuda.current_stream().cuda_stream)
    assert st == gl.OK
    torch.cuda.synchronize()
    return out


def test_very_many_rows():
    # the last of five million rows equal the same rows alone
    T, H = 5_000_003, 9
    g = torch.Generator(device=device()).manual_seed(1)
    res = torch.randn(T, H, generator=g, device=device())
    o = torch.randn(T, H, generator=g, device=device())
    post, pre = torch.ones(H, device=device()), torch.ones(H, device=device())
    r, x = gl.norm_residual(res, o, post, pre_weight=pre, alpha=ALPHA, beta=BETA)
    n = slice(T - 7, T)
    r2, x2 = gl.norm_residual(res[n].contiguous(), o[n].contiguous(), post, pre_weight=pre, alpha=ALPHA, beta=BETA)
    assert torch.equal(r[n], r2) and torch.equal(x[n], x2)
    got = gl.norm_residual_backward(r, res, x, o, post, pre_weight=pre, alpha=ALPHA, beta=BETA)
    alone = gl.norm_residual_backward(r2, res[n].contiguous(), x2, o[n].contiguous(), post, pre_weight=pre,
                                      alpha=ALPHA, beta=BETA)
    assert torch.equal(got["d_o"][n], alone["d_o"]) and torch.equal(got["d_residual"][n], alone["d_residual"])

"""A layer's operators one after another, as a layer stack calls them: norm to
e4m3 codes, dense product, norm step, softmax routing and the expert block,
norm step, and the way back.  Every operator is checked against the 64-bit
formula of its own inputs, which are the outputs of the one before it, with
the tolerances of its own tests; the whole run is repeated on another stream
and from captured graphs, bit for bit."""
import numpy as np
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import layer_ref as ref
import oracle
import test_gpu_matmul as mm
import test_gpu_norm as nm
import test_gpu_route_scores as rs
from gpu_util import device, max_rel_err
from synth import WORKLOADS, make_inputs, small_shape

pytestmark = pytest.mark.gpu

FLAGS = gl.ROUTE_SOFTMAX | gl.ROUTE_UNNORMED
ALPHA, BETA, EPS = nm.ALPHA, nm.BETA, nm.EPS


def make(T, seed):
    dev, sh = device(), small_shape()
    H, g = sh.hidden, torch.Generator(device=device()).manual_seed(seed)
    inp = make_inputs(WORKLOADS["prefill4k"], device=dev, tokens=T, shape=sh, seed=seed)
    n = lambda *s: torch.randn(*s, generator=g, device=dev)
    c = dict(sh=sh, inp=inp, d=gl.make_desc(sh, gl.BF16, gl.BF16, FLAGS), residual=n(T, H), gate=n(T, 1).bfloat16(),
             w=(n(H, H) / H ** 0.5).bfloat16(), d_r=n(T, H), d_x=n(T, H).bfloat16(), d_w=n(T, sh.top_k))
    for k in ("pre1", "post1", "pre2", "post2", "pre3"):
        c[k] = 1 + n(H) / 10
    c["wq"], c["ws"], c["wt"], c["wts"] = gl.quant_e4m3_2d(c["w"], block=True)
    return c


def run(c, stream=None, workspace=None):
    """The layer forward and back; every intermediate."""
    kw, inp, d, v = dict(stream=stream), c["inp"], c["d"], {}
    ws = dict(kw, workspace=workspace)
    step1 = dict(post_weight=c["post1"], gate=c["gate"], pre_weight=c["pre2"], eps=EPS, alpha=ALPHA, beta=BETA)
    step2 = dict(post_weight=c["post2"], pre_weight=c["pre3"], eps=EPS, alpha=ALPHA, beta=BETA)
    _, v["q"], v["s"] = gl.norm_residual_e4m3(c["residual"], pre_weight=c["pre1"], eps=EPS, **kw)
    v["y"] = gl.matmul_e4m3(v["q"], v["s"], c["wq"], c["ws"], **kw)
    v["r1"], v["x1"] = gl.norm_residual(c["residual"], v["y"], **step1, **kw)
    v["o"], v["idx"], v["w"], v["lg"] = gl.forward(d, v["x1"], inp.w_router, inp.bias, inp.w_gate_up, inp.w_down,
                                                   return_routing=True, **ws)
    v["r2"], v["x2"] = gl.norm_residual(v["r1"], v["o"], **step2, **kw)
    b2 = gl.norm_residual_backward(v["r2"], c["d_r"], c["d_x"], v["o"], **step2, **ws)
    v.update({"b2_" + k: t for k, t in b2.items()})
    v["d_lg"] = gl.route_backward(d, v["lg"], v["idx"], c["d_w"], **kw)
    b1 = gl.norm_residual_backward(v["r1"], b2["d_residual"], b2["d_o"], v["y"], **step1, **ws)
    v.update({"b1_" + k: t for k, t in b1.items()})
    v["gq"], v["gs"], v["gt"], v["gts"] = gl.quant_e4m3_2d(b1["d_o"], **kw)
    v["dx"] = gl.matmul_e4m3(v["gq"], v["gs"], c["wt"], c["wts"], **kw)
    return v


@pytest.mark.parametrize("T", [1, 60, 257])
def test_layer(T):
    c = make(T, 40 + T)
    v, sh, inp = run(c), c["sh"], c["inp"]
    cpu = lambda t: None if t is None else t.cpu()
    bf = torch.bfloat16
    # the codes are those of the exact x but where its rounding decides one
    # way or the other: within a code's half step and x's own tolerance
    x0 = ref.norm_step(cpu(c["residual"]), None, None, None, cpu(c["pre1"]), EPS, 1.0, 1.0)[1]
    back = v["q"].view(torch.float8_e4m3fn).cpu().double() * cpu(v["s"]).double().repeat_interleave(128, 1)
    tol = 2.0 ** -4 * x0.abs() * (1 + 2.0 ** -15) + cpu(v["s"]).double().repeat_interleave(128, 1) * 2.0 ** -10
    assert ((back - x0).abs() <= tol + 2 * nm.KAPPA * ref.U * x0.abs()).all()
    mm.check(v["y"], v["q"], v["s"], c["wq"], c["ws"], False)
    n1 = dict(residual=c["residual"], o=v["y"], post=c["post1"], gate=c["gate"], pre=c["pre2"])
    n2 = dict(residual=v["r1"], o=v["o"], post=c["post2"], gate=None, pre=c["pre3"])
    nm.check_forward({k: cpu(t) for k, t in n1.items()}, bf, v["r1"], v["x1"], eps=EPS)
    nm.check_forward({k: cpu(t) for k, t in n2.items()}, bf, v["r2"], v["x2"], eps=EPS)
    idx, lg = cpu(v["idx"]), cpu(v["lg"])
    assert torch.equal(idx, ref.select(lg, cpu(inp.bias), sh.n_groups, sh.topk_groups, sh.top_k,
                                       sh.group_score_topn, True))
    want = oracle.forward_tokens(sh, np.arange(T), v["x1"].cpu(), idx.numpy(), v["w"].cpu().numpy(),
                                 inp.w_gate_up.cpu(), inp.w_down.cpu())
    assert max_rel_err(v["o"].float().cpu().numpy(), want) <= 2e-2      # the bf16 block's bar
    b2 = {k[3:]: t for k, t in v.items() if k.startswith("b2_")}
    b1 = {k[3:]: t for k, t in v.items() if k.startswith("b1_")}
    n2.update(d_r=c["d_r"], d_x=c["d_x"])
    n1.update(d_r=b2["d_residual"], d_x=b2["d_o"])
    nm.check_backward({k: cpu(t) for k, t in n2.items()}, bf, v["r2"], b2, eps=EPS)
    nm.check_backward({k: cpu(t) for k, t in n1.items()}, bf, v["r1"], b1, eps=EPS)
    d_lg = ref.route_grad(lg, idx, cpu(c["d_w"]), sh.routed_scale, True, False)
    bound = rs.grad_bound(lg, idx, cpu(c["d_w"]), True, False, sh.routed_scale)
    assert ((v["d_lg"].cpu().double() - d_lg).abs() <= bound).all()
    mm.check(v["dx"], v["gq"], v["gs"], c["wt"], c["wts"], False)


def same(a, b):
    return [k for k in a if not torch.equal(a[k], b[k])]


def test_two_streams_at_once():
    # default workspaces: one a stream
    cs = [make(130, 1), make(33, 2)]
    want = [run(c) for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        got = [run(c, stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        assert [same(w, g) for w, g in zip(want, got)] == [[], []]


def test_two_graphs_on_two_streams():
    # captured without a workspace: each graph has scratch memory of its own,
    # so the two may run at once, beside eager calls with a third
    cs = [make(70, 3), make(70, 4), make(90, 5)]
    want = [run(c) for c in cs]
    torch.cuda.synchronize()
    before = set(gl._default_ws)
    graphs, got = [], []
    for c in cs[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(run(c))
    assert set(gl._default_ws) == before      # nothing of the graphs' memory is kept
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for v in got:
            for t in v.values():
                t.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = run(cs[2])
        torch.cuda.synchronize()
        assert [same(w, g) for w, g in zip(want, got + [eager])] == [[], [], []]


def test_one_workspace_for_every_operator():
    c, ws = make(50, 6), gl.Workspace(device())
    assert same(run(c), run(c, workspace=ws)) == []


def test_nan_stays_in_its_row():
    # a NaN or an infinity in one token reaches that token's outputs only, and
    # does reach them
    c = make(40, 7)
    want = run(c)
    for bad in (float("nan"), float("inf")):
        x = want["x1"].clone()
        x[13, 5] = bad
        q, s, _, _ = gl.quant_e4m3_2d(x, transposed=False)
        good = gl.quant_e4m3_2d(want["x1"], transposed=False)
        for dtype in (torch.bfloat16, torch.float32):
            y = gl.matmul_e4m3(q, s, c["wq"], c["ws"], dtype=dtype)
            clean = gl.matmul_e4m3(good[0], good[1], c["wq"], c["ws"], dtype=dtype)
            assert not torch.isfinite(y[13].float()).any()
            y[13] = clean[13]
            assert torch.equal(y, clean)
        r = c["residual"].clone()
        r[13, 5] = bad
        _, q, s = gl.norm_residual_e4m3(r, pre_weight=c["pre1"], eps=EPS)
        y = gl.matmul_e4m3(q, s, c["wq"], c["ws"])
        assert not torch.isfinite(y[13].float()).any()
        y[13] = want["y"][13]
        assert torch.equal(y, want["y"])


def test_routing_refuses_what_it_cannot_read():
    c = make(4, 8)
    d = gl.with_flags(c["d"], FLAGS | gl.ROUTE_LOGITS_IN)
    E = c["sh"].n_experts
    lg = torch.zeros(4, E, device=device())
    for bad in (lg.double(), lg[:, :E // 2].contiguous(), lg.cpu(), torch.zeros(E, 4, device=device()).t()):
        with pytest.raises(ValueError):
            gl.route(d, None, None, None, bad)
    with pytest.raises(ValueError, match="bias"):
        gl.route(d, None, None, torch.zeros(E + 1, device=device()), lg)


def test_routing_of_nan_rows_stays_distinct():
    # every bit pattern of a NaN: still K different experts, nothing out of range
    c = make(4, 9)
    E, K = c["sh"].n_experts, c["sh"].top_k
    bits = torch.tensor([-1, 0x7FC00000, -4194304, 0x7F800001], dtype=torch.int32, device=device())
    lg = bits.view(torch.float32)[:, None].expand(4, E).contiguous()
    for flags in (0, gl.ROUTE_SOFTMAX):
        idx, _, _ = gl.route(gl.with_flags(c["d"], flags | gl.ROUTE_LOGITS_IN), None, None, None, lg)
        idx = idx.cpu()
        assert ((idx >= 0) & (idx < E)).all()
        assert all(len(set(r.tolist())) == K for r in idx)


@pytest.mark.parametrize("flags", [gl.ROUTE_SOFTMAX, gl.ROUTE_SOFTMAX | gl.ROUTE_UNNORMED])
def test_nan_and_infinite_logits_make_their_row_nan(flags):
    c = make(6, 10)
    d = gl.with_flags(c["d"], flags | gl.ROUTE_LOGITS_IN)
    lg = torch.randn(6, c["sh"].n_experts, device=device())
    clean = gl.route(d, None, None, None, lg)
    g = gl.route_backward(d, lg, clean[0], c["d_w"])
    lg[1, 3], lg[4, 50] = float("nan"), float("inf")
    idx, w, _ = gl.route(d, None, None, None, lg)
    got = gl.route_backward(d, lg, idx, c["d_w"])
    ok = [0, 2, 3, 5]
    assert torch.isnan(w[[1, 4]]).all() and torch.equal(w[ok], clean[1][ok]) and torch.equal(idx[ok], clean[0][ok])
    chosen = torch.gather(got, 1, idx.long())
    assert torch.isnan(chosen[[1, 4]]).all() and torch.equal(got[ok], g[ok])
    assert all(len(set(r)) == c["sh"].top_k for r in idx.tolist())


def test_residual_out_needs_a_block_output():
    c = make(3, 11)
    with pytest.raises(ValueError, match="belongs to o"):
        gl.norm_residual(c["residual"], pre_weight=c["pre1"], residual_out=torch.empty_like(c["residual"]))

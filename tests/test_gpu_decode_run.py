"""The operators around a paged cache one after another, as a server calls them:
a prompt's keys into the cache, samples that fork its pages, decode steps of
norms, rotation, attention and scores whose best alternatives are the next
step's parents, the pool packed in between; and a training step of the same
heads and logits.  Every operator is checked against the 64-bit formula of its
own inputs with the tolerances of its own tests; the whole run is repeated on
another stream and from captured graphs, bit for bit."""
import math

import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import serve_ref as ref
import test_gpu_attention as ta
import test_gpu_rope as tr
import test_gpu_score as ts
from gpu_util import device

pytestmark = pytest.mark.gpu

Hq, Hkv, D, PAGE, POOL, COLS, V, BEAMS = 12, 2, 64, 8, 60, 8, 1003, 3
LAYERS = ((0, (2048.0, 0.1), 0), (64, None, 20))         # rotated channels, temperature, window
I32, BF16, F32 = torch.int32, torch.bfloat16, torch.float32


def make(prompts, steps, seed):
    """Weights, and each step's projections as drawn once: the run's inputs."""
    dev, g = device(), torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    T, B = sum(prompts), BEAMS * len(prompts)
    width = (Hq + 2 * Hkv) * D
    c = dict(prompts=prompts, steps=steps, w=[[1 + n(D) / 10, 1 + n(D) / 10] for _ in LAYERS],
             prompt=[n(T, width).to(BF16) for _ in LAYERS],
             step=[[n(B, width).to(BF16) for _ in LAYERS] for _ in range(steps)],
             gate=[n(B, Hq, D).to(BF16) for _ in LAYERS], head=(n(Hq * D, V) / (Hq * D) ** 0.5 * 8).to(BF16),
             d_q=n(T, Hq, D).to(BF16), d_k=n(T, Hkv, D).to(BF16), d_l=n(T), d_h=n(T), logits=n(T, V).to(BF16) * 3,
             targets=torch.randint(-1, V, (T,), generator=g))
    rows = torch.cat([torch.full((p,), i, dtype=I32) for i, p in enumerate(prompts)])
    pos = torch.cat([torch.arange(p, dtype=I32) for p in prompts])
    c.update(rows=rows, pos=pos, grow=torch.tensor(prompts, dtype=I32))

    def move(x):
        return x.to(dev) if torch.is_tensor(x) else [move(y) for y in x] if isinstance(x, list) else x
    c = {k: move(v) if k not in ("prompts", "steps") else v for k, v in c.items()}
    c["freq"] = gl.rope_frequencies(LAYERS[1][0], 1e4, dev)
    # allocated once, so that a captured run finds them again
    c["k"], c["v"] = (torch.zeros(len(LAYERS), POOL, PAGE, Hkv, D, dtype=BF16, device=dev) for _ in range(2))
    c["empty"] = dict(tables=torch.full((len(prompts), COLS), -1, dtype=I32, device=dev),
                      lengths=torch.zeros(len(prompts), dtype=I32, device=dev), refs=torch.zeros(POOL, dtype=I32, device=dev))
    # pages that something else holds until the pool is packed
    c["held"] = (torch.arange(POOL, device=dev) % 3 == 0).to(I32) * (torch.arange(POOL, device=dev) < 24)
    c["empty"]["refs"] += c["held"]
    c["first"] = torch.tensor([i for i in range(len(prompts)) for _ in range(BEAMS)], dtype=I32, device=dev)
    c["one"] = torch.ones(BEAMS * len(prompts), dtype=I32, device=dev)
    # every prompt's samples go on from two of them in turn
    c["next"] = torch.tensor([BEAMS * i + (0, 0, 2)[j % 3] for i in range(len(prompts)) for j in range(BEAMS)],
                             dtype=I32, device=dev)
    return c


def heads(x):
    return tr.heads(x, Hq, Hkv, D)


def run(c, see=None, **kw):
    """The run; see(what, inputs, outputs) looks on.  Returns every output."""
    out, ws = [], dict(kw)
    kw = {k: v for k, v in kw.items() if k == "stream"}
    see = see or (lambda *a: None)

    def keep(what, inputs, outputs):
        see(what, inputs, outputs)
        out.extend(t for t in outputs.values() if torch.is_tensor(t))

    def pages(t, parents, grow, what):
        got = gl.pages_update(t["tables"], t["lengths"], t["refs"], PAGE, parents, grow, pools=[c["k"], c["v"]], **ws)
        keep(what, dict(t, parents=parents, grow=grow), got)
        return got

    def norms(layer, x, pos, rows, t):
        rot, temp, _ = LAYERS[layer]
        q, k, v = heads(x)
        args = dict(positions=pos, inv_freq=c["freq"] if rot else None, temperature=temp)
        y, kk = gl.qk_norm_rope(q, k, *c["w"][layer], **args, v=v, k_cache=c["k"][layer], v_cache=c["v"][layer],
                                tables=t["tables"], rows=rows, with_k=True, **kw)
        keep("norms", dict(layer=layer, x=x, pos=pos, rows=rows, tables=t["tables"]), dict(q=y, k=kk))
        return y

    t = pages(c["empty"], None, c["grow"], "prompt pages")
    for i in range(len(LAYERS)):
        norms(i, c["prompt"][i], c["pos"], c["rows"], t)
    parents = c["first"]
    for s in range(c["steps"]):
        t = pages(t, parents, c["one"], "step")
        pos = t["lengths"] - 1
        x = None
        for i, (_, _, window) in enumerate(LAYERS):
            q = norms(i, c["step"][s][i], pos, None, t)
            o, lse = gl.paged_attention(q, c["k"][i], c["v"][i], t["tables"], t["lengths"], window=window,
                                        gate=c["gate"][i], with_lse=True, **ws)
            keep("attention", dict(q=q, layer=i, window=window, tables=t["tables"], lengths=t["lengths"]),
                 dict(out=o, lse=lse))
            x = o if x is None else (x + o)
        logits = x.view(len(x), -1) @ c["head"]
        sc = gl.token_logprobs(logits, torch.zeros_like(c["one"], dtype=torch.int64), softcap=30.0, top=4, **ws)
        keep("scores", dict(logits=logits), sc)
        parents = c["next"]
        if s == 1:
            old = dict(t, refs=t["refs"] - c["held"])
            got = gl.pages_compact(t["tables"], t["lengths"], old["refs"], PAGE, pools=[c["k"], c["v"]], **ws)
            keep("packing", old, got)
            t = dict(t, tables=got["tables"], refs=got["refs"])
    # a training step of the rotated layer's heads and of the logits
    q, k, _ = heads(c["prompt"][1])
    b = gl.qk_norm_rope_backward(c["d_q"], c["d_k"], q, k, *c["w"][1], positions=c["pos"], inv_freq=c["freq"], **ws)
    keep("gradients", {}, b)
    sc = gl.token_logprobs(c["logits"], c["targets"], softcap=30.0, **ws)
    d = gl.token_logprobs_backward(c["logits"], sc["lse"], sc["entropy"], c["targets"], c["d_l"], c["d_h"], softcap=30.0, **kw)
    keep("score gradients", {}, dict(sc, d=d))
    out.extend((c["k"], c["v"]))
    return out


def cpu(x):
    return {k: v.cpu() if torch.is_tensor(v) else v for k, v in x.items()}


def test_server():
    c = make([5, 16, 23], 5, 1)
    seen = []
    state = {}

    def see(what, i, o):
        seen.append(what)
        i, o = cpu(i), cpu(o)
        k, v = c["k"].cpu(), c["v"].cpu()
        if what in ("prompt pages", "step"):
            par = None if i["parents"] is None else i["parents"].tolist()
            w = ref.pages_update(i["tables"].tolist(), i["lengths"].tolist(), i["refs"].tolist(), PAGE, par,
                                 i["grow"].tolist())
            assert [o["tables"].tolist(), o["lengths"].tolist(), o["refs"].tolist(), o["missing"].tolist()] == \
                [*w[:3], [w[3]]] and w[3] == 0
            for a, b in w[4]:
                state["k"][:, b], state["v"][:, b] = state["k"][:, a], state["v"][:, a]
        elif what == "packing":
            w = ref.pages_compact(i["tables"].tolist(), i["lengths"].tolist(), i["refs"].tolist(), PAGE)
            assert [o["tables"].tolist(), o["refs"].tolist(), o["new_id"].tolist(), o["live"].tolist()] == [*w[:3], [w[3]]]
            assert w[4]
            for a, b in w[4]:
                state["k"][:, b], state["v"][:, b] = state["k"][:, a], state["v"][:, a]
        elif what == "norms":
            rot, temp, _ = LAYERS[i["layer"]]
            q, kk, vv = heads(i["x"])
            w = [x.cpu() for x in c["w"][i["layer"]]]
            case = dict(positions=i["pos"], inv_freq=c["freq"].cpu() if rot else None)
            tr.check_forward(case, q, w[0], o["q"], False, temp, BF16, "q")
            tr.check_forward(case, kk, w[1], o["k"], False, None, BF16, "k")
            rows = range(len(q)) if i["rows"] is None else i["rows"].tolist()
            for t, (r, p) in enumerate(zip(rows, i["pos"].tolist())):
                page = int(i["tables"][r, p // PAGE])
                state["k"][i["layer"], page, p % PAGE] = o["k"][t]
                state["v"][i["layer"], page, p % PAGE] = vv[t]
        elif what == "attention":
            case = dict(q=i["q"], gate=c["gate"][i["layer"]].cpu(), k_cache=k[i["layer"]], v_cache=v[i["layer"]],
                        tables=i["tables"], lengths=i["lengths"])
            ta.check(case, o["out"], o["lse"], i["window"], True)
        elif what == "scores":
            ts.check(dict(logits=i["logits"], targets=torch.zeros(len(i["logits"]), dtype=torch.int64)), o, 30.0, 1.0, 4)
        elif what == "gradients":
            case = dict(positions=c["pos"].cpu(), inv_freq=c["freq"].cpu())
            q, kk, _ = heads(c["prompt"][1].cpu())
            w = [x.cpu() for x in c["w"][1]]
            tr.check_backward(case, q, w[0], c["d_q"].cpu(), o["d_q"], o["d_q_weight"], False, None, BF16, "q")
            tr.check_backward(case, kk, w[1], c["d_k"].cpu(), o["d_k"], o["d_k_weight"], False, None, BF16, "k")
        else:
            case = dict(logits=c["logits"].cpu(), targets=c["targets"].cpu(), d_l=c["d_l"].cpu(), d_h=c["d_h"].cpu())
            ts.check(case, o, 30.0, 1.0, 0)
            ts.check_gradient(case, o["d"], True, True, 30.0, 1.0)
        # the cache holds what was put there and nothing else moved
        assert torch.equal(k, state["k"]) and torch.equal(v, state["v"]), what

    state["k"], state["v"] = c["k"].cpu(), c["v"].cpu()
    run(c, see)
    assert {"prompt pages", "step", "norms", "attention", "scores", "packing", "gradients", "score gradients"} <= set(seen)


def clean(c):
    c["k"].zero_()
    c["v"].zero_()


def same(a, b):
    return [i for i, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y)]


def test_two_streams_at_once():
    cs = [make([5, 16, 23], 3, 2), make([9, 1], 3, 3)]
    want = [[t.clone() for t in run(c)] for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        for c in cs:
            clean(c)
        torch.cuda.synchronize()
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(run(c))
        torch.cuda.synchronize()
        assert [same(w, g) for w, g in zip(want, got)] == [[], []]


def test_a_stream_given_to_the_calls():
    # every operator alone on a stream that is not the current one
    c = make([5, 16], 1, 4)
    s = torch.cuda.Stream()
    want = run(c)
    want = [t.clone() for t in want]
    clean(c)
    torch.cuda.synchronize()
    # (the run's torch steps between the operators need the same order)
    t = gl.pages_update(**c["empty"], page_size=PAGE, grow=c["grow"], pools=[c["k"], c["v"]], stream=s)
    q, k, v = heads(c["prompt"][0])
    y, _ = gl.qk_norm_rope(q, k, *c["w"][0], positions=c["pos"], temperature=LAYERS[0][1], v=v, k_cache=c["k"][0],
                           v_cache=c["v"][0], tables=t["tables"], rows=c["rows"], stream=s)
    o = gl.paged_attention(y[:2].contiguous(), c["k"][0], c["v"][0], t["tables"], t["lengths"], stream=s)
    sc = gl.token_logprobs(c["logits"], c["targets"], top=2, stream=s)
    b = gl.token_logprobs_backward(c["logits"], sc["lse"], sc["entropy"], c["targets"], c["d_l"], stream=s)
    gl.pages_copy([c["k"]], c["first"][:1], c["first"][:1] + POOL, stream=s)       # (no page: nothing moves)
    s.synchronize()
    assert torch.equal(t["tables"], want[0]) and torch.isfinite(o.float()).all() and torch.isfinite(b.float()).all()


def test_two_graphs_on_two_streams():
    # captured without a workspace: each graph has scratch memory of its own; every
    # replay is checked, with eager work between
    cs = [make([5, 16, 23], 3, 5), make([20, 7], 3, 6), make([6, 6], 2, 7)]
    want = [[t.clone() for t in run(c)] for c in cs]
    torch.cuda.synchronize()
    before = set(gl._default_ws)
    graphs, got = [], []
    for c in cs[:2]:
        clean(c)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(run(c))
    assert set(gl._default_ws) == before
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for v in got:
            for t in v:
                t.zero_()
        clean(cs[2])
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = run(cs[2])
        torch.cuda.synchronize()
        assert [same(w, g) for w, g in zip(want, got + [eager])] == [[], [], []]


def test_one_workspace_for_every_operator():
    c, ws = make([5, 16, 23], 3, 8), gl.Workspace(device())
    want = [t.clone() for t in run(c)]
    clean(c)
    assert same(want, run(c, workspace=ws)) == []


def test_tensors_that_do_not_fit_are_refused():
    dev = device()
    q, w = torch.zeros(2, 4, 64, dtype=BF16, device=dev), torch.ones(64, device=dev)
    k = torch.zeros(2, 2, 64, dtype=BF16, device=dev)
    kc = torch.zeros(4, 8, 2, 64, dtype=BF16, device=dev)
    tb, ln = torch.zeros(2, 3, dtype=I32, device=dev), torch.ones(2, dtype=I32, device=dev)
    pos = torch.zeros(2, dtype=I32, device=dev)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:1]), dict(positions=pos, inv_freq=torch.ones(8, device=dev)),
                dict(inv_freq=gl.rope_frequencies(16)), dict(temperature=(0.0, 1.0), positions=pos),
                dict(v=k), dict(k_cache=kc, v_cache=kc, v=k, tables=tb), dict(k_cache=kc, v_cache=kc, positions=pos, tables=tb),
                dict(k_cache=kc, v_cache=kc.float(), v=k, positions=pos, tables=tb),
                dict(k_cache=kc, v_cache=kc, v=k, positions=pos, tables=tb[:1]),
                dict(k_cache=kc, v_cache=kc, v=k, positions=pos, tables=tb.long()),
                dict(k_cache=kc, v_cache=kc.transpose(1, 2).contiguous().transpose(1, 2), v=k, positions=pos, tables=tb),
                dict(k_cache=kc[..., ::2], v_cache=kc[..., ::2], v=k, positions=pos, tables=tb), dict(with_k=False)):
        with pytest.raises(ValueError):
            gl.qk_norm_rope(q, k, w, w, **bad)
    for args in ((q, k[:1], w, w), (q, k.float(), w, w), (q[..., ::2], k[..., ::2], w[:32], w[:32]), (q, k, w[:32], w),
                 (q.transpose(0, 1), k, w, w)):
        with pytest.raises(ValueError):
            gl.qk_norm_rope(*args)
    with pytest.raises(gl.BeamError):       # a row that does not start on 16 bytes
        x = torch.zeros(2, 2 * 4 * 64 + 2, dtype=BF16, device=dev)[:, :256].view(2, 4, 64)
        gl.qk_norm_rope(x, k, w, w)
    for args in ((q, kc, kc, tb[:1], ln), (q, kc, kc, tb, ln.long()), (q, kc, kc.float(), tb, ln), (q[:, :3], kc, kc, tb, ln),
                 (q.float(), kc, kc, tb, ln)):
        with pytest.raises((ValueError, gl.BeamError)):
            gl.paged_attention(*args)
    with pytest.raises(ValueError):
        gl.paged_attention(q, kc, kc, tb, ln, gate=q[:1])
    refs = torch.zeros(4, dtype=I32, device=dev)
    pool = torch.zeros(2, 4, 64, device=dev)
    for bad in (dict(parents=ln.long()), dict(grow=ln[:1]), dict(pools=[pool[:, :3]]), dict(pools=[pool, pool[:1]]),
                dict(pools=[pool.transpose(1, 2)]), dict(pools=[pool] * 9), dict(pools=[pool.cpu()])):
        with pytest.raises(ValueError):
            gl.pages_update(tb, ln, refs, 8, **bad)
    with pytest.raises(gl.BeamError):       # 12 bytes a page
        gl.pages_update(tb, ln, refs, 8, pools=[pool[:, :, :3].contiguous()])
    with pytest.raises(gl.BeamError):
        gl.pages_update(tb, ln, refs, 12)
    lg = torch.zeros(2, 10, device=dev)
    for bad in (dict(targets=ln), dict(targets=ln.long()[:1])):
        with pytest.raises(ValueError):
            gl.token_logprobs(lg, **bad)
    with pytest.raises(ValueError):
        gl.token_logprobs(lg.t())
    with pytest.raises(gl.BeamError):
        gl.token_logprobs(lg, top=11)
    with pytest.raises(ValueError):
        gl.token_logprobs_backward(lg, lg[:, 0].contiguous(), lg[:1, 0], d_entropy=lg[:, 0].contiguous())

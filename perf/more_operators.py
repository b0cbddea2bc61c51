"""What is measured of the operators around a paged key-value cache, and how.

Four operators, each in its plain form (elementary torch operations in 32
bits, angles of positions in 64, rounded once at the end) and as a user calls
the library:

qk       the norm of every query and key head with the rotation by position (or
         the query's temperature) in the same pass; in serving the keys and
         values go to their places in a paged cache; in training also the
         gradients of the projections and of both norms' weights.
attend   attention of one new token of every sequence over its pages, whole or
         over a sliding window, with a gate for each channel or without.
pages    the step of a batch's page tables: rows that go on from a parent's
         tokens, shared pages copied before they are written, new pages, pages
         of rows that went away; and the moving of used pages to the pool's
         front.
score    log probabilities of given tokens under capped logits, the entropy and
         the best alternatives; in training also the gradient of the logits.

48 query and 8 key-value heads of 128, the window of 512 tokens, the query's
temperature (1 + (pos + 1) / 2048)^0.1 and the cap of 30 are the framework's
own model; the other sizes are generic.
"""
import math

import torch

own = False

Q_HEADS, KV_HEADS, HEAD, WINDOW = 48, 8, 128, 512
TEMPERATURE = (2048.0, 0.1)
CAP, EPS, BASE = 30.0, 1e-6, 1e6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
I32 = torch.int32


# ---- the cases -----------------------------------------------------------

def _qk(name, tokens, seqs, heads, kv_heads, head, dtype, rot, pairs, page, train):
    """rot: the channels that turn; 0: none, and the query has a temperature.
    pairs: neighbouring channels turn together, else those half of rot apart.
    seqs: the sequences that the tokens belong to."""
    return {"name": name, "op": "qk", "tokens": tokens, "seqs": seqs, "heads": heads, "kv_heads": kv_heads,
            "head": head, "dtype": dtype, "rot": rot, "pairs": pairs, "page": page, "train": train}


def _attend(name, seqs, shortest, longest, heads, kv_heads, head, dtype, page, window, gate):
    """Lengths spread over their logarithm from shortest to longest."""
    return {"name": name, "op": "attend", "seqs": seqs, "shortest": shortest, "longest": longest, "heads": heads,
            "kv_heads": kv_heads, "head": head, "dtype": dtype, "page": page, "window": window, "gate": gate}


def _pages(name, what, rows, longest, page, layers, width, share):
    """width: values of a page's token in one layer; share: rows of the batch
    to a row that they go on from."""
    return {"name": name, "op": "pages", "what": what, "rows": rows, "longest": longest, "page": page,
            "layers": layers, "width": width, "share": share}


def _score(name, rows, vocab, dtype, cap, top, train):
    return {"name": name, "op": "score", "rows": rows, "vocab": vocab, "dtype": dtype, "cap": cap, "top": top,
            "train": train}


def listed():
    return [
        # the new tokens of a decode batch in a sliding-window layer
        _qk("qk decode 64", 64, 64, Q_HEADS, KV_HEADS, HEAD, "bf16", HEAD, False, 16, False),
        # a prefill of three prompts of unlike lengths in a global layer
        _qk("qk prefill 16381 global", 16381, 3, Q_HEADS, KV_HEADS, HEAD, "bf16", 0, False, 64, False),
        # a training step on a ragged batch, with the gradients
        _qk("qk train 8191", 8191, 5, Q_HEADS, KV_HEADS, HEAD, "bf16", HEAD, False, 0, True),
        # one request at the start of its answer
        _attend("attend 1 of 900", 1, 900, 900, Q_HEADS, KV_HEADS, HEAD, "bf16", 16, 0, True),
        # a decode batch of unlike lengths in a global layer
        _attend("attend 64 ragged", 64, 100, 32000, Q_HEADS, KV_HEADS, HEAD, "bf16", 16, 0, True),
        # the same batch's size in a sliding-window layer
        _attend("attend 256 window", 256, 200, 20000, Q_HEADS, KV_HEADS, HEAD, "bf16", 16, WINDOW, True),
        # one request at the end of the longest context
        _attend("attend 1 of 1000003", 1, 1000003, 1000003, Q_HEADS, KV_HEADS, HEAD, "bf16", 64, 0, False),
        # samples of four prompts, the next step of each: tables and copies
        _pages("pages step 32", "step", 32, 3000, 16, 4, KV_HEADS * HEAD, 8),
        # a full decode batch, two rows to a parent
        _pages("pages step 512", "step", 512, 3000, 16, 4, KV_HEADS * HEAD, 2),
        # a pool that emptied in places is packed to its front
        _pages("pages pack", "pack", 200, 4000, 16, 4, KV_HEADS * HEAD, 1),
        # one request's logits: the token's log probability, eight alternatives
        _score("score 1 of 131072", 1, 131072, "f32", True, 8, False),
        # a training step of a policy with its entropy, an odd vocabulary
        _score("score train 4096 of 100003", 4096, 100003, "bf16", True, 0, True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk", "attend", "pages", "score"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    head = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "dtype": dtype, "head": head, "kv_heads": kv, "heads": kv * rng.randint(1, 8),
         "page": rng.choice([8, 16, 32, 64, 256])}
    if op == "qk":
        most = 16381 * Q_HEADS * HEAD // (c["heads"] * head * (2 if dtype == "f32" else 1))
        c.update(tokens=min(_spread(rng, 1, 16381), most), rot=rng.choice([0, head // 2, head]),
                 pairs=rng.random() < 0.3, train=rng.random() < 0.4)
        c["seqs"] = rng.randint(1, min(c["tokens"], 64))
        if c["train"]:
            c["tokens"] = max(c["seqs"], c["tokens"] // 2)
    elif op == "attend":
        c["seqs"] = _spread(rng, 1, 256)
        most = 500000 * 2 * KV_HEADS * HEAD // (kv * head * (2 if dtype == "f32" else 1) * c["seqs"])
        c["longest"] = _spread(rng, 1, max(2, min(300000, most)))
        c["shortest"] = _spread(rng, 1, c["longest"])
        c.update(window=rng.choice([0, 0, _spread(rng, 1, 4096)]), gate=rng.random() < 0.5)
    elif op == "pages":
        c = {"op": op, "what": rng.choice(["step", "step", "pack"]), "rows": _spread(rng, 1, 500),
             "page": rng.choice([1, 8, 16, 32, 64]), "layers": rng.randint(1, 9), "width": 8 * _spread(rng, 8, 128),
             "share": rng.randint(1, 8)}
        most = 256 * 3000 * 4 * KV_HEADS * HEAD // (-(-c["rows"] // c["share"]) * c["layers"] * c["width"])
        c["longest"] = _spread(rng, 1, max(2, min(6000, most)))
    else:
        vocab, train = _spread(rng, 100, 200000), rng.random() < 0.5
        c = {"op": op, "dtype": dtype, "vocab": vocab, "train": train, "cap": rng.random() < 0.5,
             "rows": max(1, min(_spread(rng, 1, 4096), 4096 * 100003 // vocab // (2 if dtype == "f32" else 1))),
             "top": rng.choice([0, 1, 5, 16])}
    return c


# ---- inputs --------------------------------------------------------------

def _type(c):
    return BF16 if c["dtype"] == "bf16" else F32


def _normal(g, *shape, dtype=F32, std=1.0):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=I32)


def _lengths(g, n, lo, hi):
    """Evenly over the logarithm, in any order."""
    u = (torch.randperm(n, generator=g, device="cuda").to(F64) + 0.5) / n
    return (lo * (hi / lo) ** u).round().clamp(lo, hi).to(I32)


def _prepare_qk(c, g):
    t, h, kv, d, dt = c["tokens"], c["heads"], c["kv_heads"], c["head"], _type(c)
    # what one projection leaves: queries, keys and values side by side
    qkv = _normal(g, t, (h + 2 * kv) * d, dtype=dt)
    c["q"] = qkv[:, :h * d].view(t, h, d)
    c["k"] = qkv[:, h * d:(h + kv) * d].view(t, kv, d)
    c["v"] = qkv[:, (h + kv) * d:].view(t, kv, d)
    c["q_weight"], c["k_weight"] = (1 + _normal(g, d, std=0.1) for _ in range(2))
    c["inv_freq"] = None
    if c["rot"]:
        c["inv_freq"] = BASE ** (-torch.arange(0, c["rot"], 2, dtype=F64, device="cuda") / c["rot"])
    # sequences of unlike lengths, each going on at a place of its own
    n = c["seqs"]
    cuts = torch.sort(torch.randperm(t - 1, generator=g, device="cuda")[:n - 1] + 1).values
    begin = torch.cat([cuts.new_zeros(1), cuts])
    row = torch.zeros(t, dtype=torch.int64, device="cuda")
    row[cuts] = 1
    row = row.cumsum(0)
    first = _ints(g, 0, 100000, n)
    c["positions"] = (first[row] + torch.arange(t, device="cuda") - begin[row]).to(I32)
    c["rows"] = row.to(I32)
    if c["train"]:
        c["d_q"], c["d_k"] = _normal(g, t, h, d, dtype=dt), _normal(g, t, kv, d, dtype=dt)
        return
    # only the pages that are written are there, in any order
    page = c["page"]
    lo, hi = first.long() // page, c["positions"].new_zeros(n, dtype=torch.int64)
    hi.scatter_reduce_(0, row, c["positions"].long() // page, "amax")
    many = hi - lo + 1
    start = many.cumsum(0) - many
    total = t // page + 2 * n
    ids = torch.randperm(total, generator=g, device="cuda")
    at = torch.arange((100000 + t) // page + 1, device="cuda")[None, :]
    inside = (at >= lo[:, None]) & (at <= hi[:, None])
    c["tables"] = torch.where(inside, ids[(start[:, None] + at - lo[:, None]).clamp(0, total - 1)], -1).to(I32)
    c["k_cache"], c["v_cache"] = (_normal(g, total, page, kv, d, dtype=dt) for _ in range(2))


def _prepare_attend(c, g):
    n, h, kv, d, dt, page = c["seqs"], c["heads"], c["kv_heads"], c["head"], _type(c), c["page"]
    c["lengths"] = _lengths(g, n, c["shortest"], c["longest"])
    many = (c["lengths"].long() + page - 1) // page
    start, total = many.cumsum(0) - many, int(many.sum())
    at = torch.arange(int(many.max()), device="cuda")[None, :]
    ids = torch.randperm(total, generator=g, device="cuda")
    c["tables"] = torch.where(at < many[:, None], ids[(start[:, None] + at).clamp(0, total - 1)], -1).to(I32)
    c["k_cache"], c["v_cache"] = (_normal(g, total, page, kv, d, dtype=dt) for _ in range(2))
    c["q"] = _normal(g, n, h, d, dtype=dt)
    c["gates"] = _normal(g, n, h, d, dtype=dt) if c["gate"] else None
    c["host_lengths"] = c["lengths"].tolist()


def _prepare_pages(c, g):
    n, page, share = c["rows"], c["page"], c["share"]
    old = -(-n // share)
    lengths = _lengths(g, old, max(1, c["longest"] // 8), c["longest"])
    many = (lengths.long() + page - 1) // page
    start, held = many.cumsum(0) - many, int(many.sum())
    c["width_pages"] = c["longest"] // page + 2
    at = torch.arange(c["width_pages"], device="cuda")[None, :]
    pool = held + held // 3 + 2 * n + 8
    ids = torch.randperm(pool, generator=g, device="cuda")[:held]
    c["tables"] = torch.where(at < many[:, None], ids[(start[:, None] + at).clamp(0, held - 1)], -1).to(I32)
    c["lengths"] = lengths
    refs = torch.zeros(pool, dtype=I32, device="cuda")
    refs[ids] = 1
    # pages that a cache of prompts holds beside the batch
    kept = torch.rand(pool, generator=g, device="cuda") < 0.05
    c["refs"] = torch.where(kept, refs + 1, refs).to(I32)
    if c["what"] == "step":
        # each row goes on from one of the old ones, some start anew, and some
        # old ones end
        parents = _ints(g, 0, old, n)
        fresh = torch.rand(n, generator=g, device="cuda") < 0.05
        c["parents"] = torch.where(fresh, -1, parents).to(I32)
        # mostly one token, now and then a drafted run of them
        c["grow"] = torch.where(torch.rand(n, generator=g, device="cuda") < 0.1, 15, 1).to(I32)
    c["pools"] = [_normal(g, c["layers"], pool, page * c["width"], dtype=BF16) for _ in range(2)]


def _prepare_score(c, g):
    t, v = c["rows"], c["vocab"]
    c["logits"] = _normal(g, t, v, dtype=_type(c), std=4.0)
    # the vocabulary's last words are ruled out, some tokens do not count
    c["logits"][:, v - v // 50:] = -math.inf
    c["targets"] = torch.randint(0, v - v // 50, (t,), generator=g, device="cuda")
    c["targets"][torch.rand(t, generator=g, device="cuda") < 0.05] = -100
    if c["train"]:
        c["d_logprobs"] = _normal(g, t, std=1.0 / t)
        c["d_entropy"] = _normal(g, t, std=0.01 / t)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    {"qk": _prepare_qk, "attend": _prepare_attend, "pages": _prepare_pages, "score": _prepare_score}[c["op"]](c, g)
    return c


# ---- the operators in their plain form -----------------------------------

def _partners(v, rot, pairs):
    """The two channels of every pair that turns."""
    if pairs:
        return v[..., 0:rot:2], v[..., 1:rot:2]
    return v[..., :rot // 2], v[..., rot // 2:rot]


def _join(a, b, v, rot, pairs):
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, v[..., rot:]], -1)


def _turn(v, cos, sin, rot, pairs):
    a, b = _partners(v, rot, pairs)
    return _join(a * cos - b * sin, a * sin + b * cos, v, rot, pairs)


def _hat(x):
    return x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS))


def _plain_qk(c):
    dt, rot = _type(c), c["rot"]
    if rot:
        # far positions' angles need 64 bits
        angle = (c["positions"].double()[:, None] * c["inv_freq"])[:, None, :]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        scale = 1.0
    else:
        scale = (1 + (c["positions"].float() + 1) / TEMPERATURE[0])[:, None, None] ** TEMPERATURE[1]
    out = {}
    for name in ("q", "k"):
        hat, w = _hat(c[name].float()), c[name + "_weight"]
        v = hat * w
        if rot:
            v = _turn(v, cos, sin, rot, c["pairs"])
        elif name == "q":
            v = v * scale
        out[name] = v.to(dt)
        if c["train"]:
            d = c["d_" + name].float()
            if rot:
                d = _turn(d, cos, -sin, rot, c["pairs"])
            elif name == "q":
                d = d * scale
            out["d_%s_weight" % name] = (d * hat).sum((0, 1))
            d = d * w
            x = c[name].float()
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            out["d_" + name] = (r * (d - hat * (d * hat).mean(-1, keepdim=True))).to(dt)
    if not c["train"]:
        pos = c["positions"].long()
        at = c["tables"][c["rows"].long(), pos // c["page"]].long()
        c["k_cache"][at, pos % c["page"]] = out.pop("k")
        c["v_cache"][at, pos % c["page"]] = c["v"]
        out["k_cache"], out["v_cache"] = c["k_cache"], c["v_cache"]
    return out


def _plain_attend(c):
    kv, d, group = c["kv_heads"], c["head"], c["heads"] // c["kv_heads"]
    out = torch.empty(c["seqs"], c["heads"], d, device="cuda")
    for i, n in enumerate(c["host_lengths"]):
        first = max(0, n - c["window"]) if c["window"] else 0
        pages = c["tables"][i, first // c["page"]:-(-n // c["page"])].long()
        skip = first % c["page"]
        k = c["k_cache"][pages].view(-1, kv, d)[skip:skip + n - first].float()
        v = c["v_cache"][pages].view(-1, kv, d)[skip:skip + n - first].float()
        q = c["q"][i].float().view(kv, group, d)
        s = q @ k.permute(1, 2, 0).contiguous() / math.sqrt(d)
        p = torch.exp(s - s.amax(-1, keepdim=True))
        out[i] = (p @ v.permute(1, 0, 2).contiguous() / p.sum(-1, keepdim=True)).view(-1, d)
    if c["gate"]:
        out = out * (1 / (1 + torch.exp(-c["gates"].float())))
    return {"out": out.to(_type(c))}


def _plain_step(c):
    tables, refs, n, page = c["tables"].long(), c["refs"].long(), c["rows"], c["page"]
    lengths, grow = c["lengths"].long(), c["grow"].long()
    wide, pool = tables.shape[1], refs.shape[0]
    at = torch.arange(wide, device="cuda")[None, :]
    old = torch.where(at < ((lengths + page - 1) // page)[:, None], tables, -1)
    go, parent = c["parents"] >= 0, c["parents"].long().clamp(min=0)
    new = torch.where(go[:, None], old[parent], -1)
    had = torch.where(go, lengths[parent], 0)
    count = torch.cat([refs, refs.new_zeros(1)])
    count.scatter_add_(0, torch.where(new >= 0, new, pool).flatten(), torch.ones_like(new).flatten())
    count.scatter_add_(0, torch.where(old >= 0, old, pool).flatten(), -torch.ones_like(old).flatten())
    # rows that write into a page that others hold too
    last = new.gather(1, (had // page).clamp(max=wide - 1)[:, None])[:, 0]
    writes = (grow > 0) & (had % page > 0) & (last >= 0)
    last = torch.where(writes, last, pool)
    order = torch.arange(n, device="cuda")
    many = torch.zeros_like(count).scatter_add_(0, last, torch.ones_like(last))
    lowest = torch.full_like(count, n).scatter_reduce_(0, last, order, "amin")
    keeps = (count[last] == 1) | ((count[last] == many[last]) & (lowest[last] == order))
    copies = writes & ~keeps
    # every row's wants in turn meet the free pages in turn
    size = had + grow
    need, have = torch.clamp((size + page - 1) // page, max=wide), (had + page - 1) // page
    want = copies.long() + need - have
    begin = want.cumsum(0) - want
    free = torch.nonzero(count[:pool] <= 0)[:, 0]
    given = torch.cat([free, free.new_full((max(0, int(want.sum()) - len(free)),), -1)])
    rank = begin[:, None] + copies.long()[:, None] + at - have[:, None]
    fresh = (at >= have[:, None]) & (at < need[:, None])
    if len(given):
        new = torch.where(fresh, given[rank.clamp(0, len(given) - 1)], new)
    src, dst = last[copies], given[begin[copies]]
    new[torch.nonzero(copies)[:, 0], (had // page)[copies]] = dst
    count.scatter_add_(0, src, -torch.ones_like(src))
    count = count[:pool]
    taken = given[:int(want.sum())]
    count[taken[taken >= 0]] = 1
    ok = dst >= 0
    for p in c["pools"]:
        p[:, dst[ok]] = p[:, src[ok]]
    missing = torch.clamp(want.sum() - len(free), min=0) + torch.clamp((size + page - 1) // page - wide, min=0).sum()
    return {"tables": new.to(I32), "lengths": torch.clamp(size, max=wide * page).to(I32), "refs": count.to(I32),
            "missing": missing.to(I32).view(1), "k": c["pools"][0], "v": c["pools"][1]}


def _plain_pack(c):
    refs, pool = c["refs"].long(), c["refs"].shape[0]
    live = refs > 0
    n = live.sum()
    ids = torch.arange(pool, device="cuda")
    # used pages behind the front's end fill its holes in order
    moves, holes = ids[live & (ids >= n)], ids[~live & (ids < n)]
    new_id = torch.where(live, ids, -1)
    new_id[moves] = holes
    out = torch.zeros_like(refs)
    out[new_id[live]] = refs[live]
    at = torch.arange(c["tables"].shape[1], device="cuda")[None, :]
    used = at < ((c["lengths"].long() + c["page"] - 1) // c["page"])[:, None]
    tables = torch.where(used & (c["tables"] >= 0), new_id[c["tables"].long().clamp(min=0)], -1)
    for p in c["pools"]:
        p[:, holes] = p[:, moves]
    return {"tables": tables.to(I32), "refs": out.to(I32), "new_id": new_id.to(I32), "live": n.to(I32).view(1),
            "k": c["pools"][0], "v": c["pools"][1]}


def _plain_score(c):
    x, t = c["logits"].float(), c["targets"]
    z = CAP * torch.tanh(x / CAP) if c["cap"] else x
    z = torch.where(x == -math.inf, x, z)     # a masked word stays masked
    e = torch.exp(z - z.amax(-1, keepdim=True))
    total = e.sum(-1, keepdim=True)
    lse = z.amax(-1, keepdim=True) + torch.log(total)
    logp, p = z - lse, e / total
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(-1)
    ok = (t >= 0) & (t < c["vocab"])
    at = torch.where(ok, t, 0)[:, None]
    out = {"logprobs": torch.where(ok, logp.gather(1, at)[:, 0], 0.0), "entropy": entropy, "lse": lse[:, 0]}
    if c["top"]:
        # the cap keeps the order: the logits themselves are compared
        out["ids"] = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]].to(I32)
        out["top"] = logp.gather(1, out["ids"].long())
    if c["train"]:
        d = -torch.where(ok, c["d_logprobs"], 0.0)[:, None] * p
        d.scatter_add_(1, at, torch.where(ok, c["d_logprobs"], 0.0)[:, None])
        d = d - torch.where(p > 0, c["d_entropy"][:, None] * p * (logp + entropy[:, None]), 0.0)
        if c["cap"]:
            d = d * (1 - torch.tanh(x / CAP) ** 2)
        out["d_logits"] = torch.where(x == -math.inf, 0.0, d).to(_type(c))
    return out


# ---- the framework's calls -----------------------------------------------

def _own_qk(c):
    import group_limited_routing_sigmoid_amd as gl
    args = dict(positions=c["positions"], inv_freq=c["inv_freq"], interleaved=c["pairs"], eps=EPS,
                temperature=None if c["rot"] else TEMPERATURE)
    if c["train"]:
        q, k = gl.qk_norm_rope(c["q"], c["k"], c["q_weight"], c["k_weight"], **args)
        got = gl.qk_norm_rope_backward(c["d_q"], c["d_k"], c["q"], c["k"], c["q_weight"], c["k_weight"], **args)
        return {"q": q, "k": k, **got}
    q, _ = gl.qk_norm_rope(c["q"], c["k"], c["q_weight"], c["k_weight"], v=c["v"], k_cache=c["k_cache"],
                           v_cache=c["v_cache"], tables=c["tables"], rows=c["rows"], **args)
    return {"q": q, "k_cache": c["k_cache"], "v_cache": c["v_cache"]}


def _own_attend(c):
    import group_limited_routing_sigmoid_amd as gl
    return {"out": gl.paged_attention(c["q"], c["k_cache"], c["v_cache"], c["tables"], c["lengths"],
                                      window=c["window"], gate=c["gates"])}


def _own_pages(c):
    import group_limited_routing_sigmoid_amd as gl
    if c["what"] == "step":
        out = gl.pages_update(c["tables"], c["lengths"], c["refs"], c["page"], parents=c["parents"], grow=c["grow"],
                              pools=c["pools"])
    else:
        out = gl.pages_compact(c["tables"], c["lengths"], c["refs"], c["page"], pools=c["pools"])
    return {**out, "k": c["pools"][0], "v": c["pools"][1]}


def _own_score(c):
    import group_limited_routing_sigmoid_amd as gl
    cap = CAP if c["cap"] else 0.0
    got = gl.token_logprobs(c["logits"], c["targets"], softcap=cap, top=c["top"])
    out = {"logprobs": got["logprobs"], "entropy": got["entropy"], "lse": got["lse"]}
    if c["top"]:
        out["ids"], out["top"] = got["top_ids"], got["top_logprobs"]
    if c["train"]:
        out["d_logits"] = gl.token_logprobs_backward(c["logits"], got["lse"], got["entropy"], c["targets"],
                                                     c["d_logprobs"], c["d_entropy"], softcap=cap)
    return out


def run(state):
    op = state["op"]
    if own:
        return {"qk": _own_qk, "attend": _own_attend, "pages": _own_pages, "score": _own_score}[op](state)
    if op == "pages":
        return _plain_step(state) if state["what"] == "step" else _plain_pack(state)
    return {"qk": _plain_qk, "attend": _plain_attend, "score": _plain_score}[op](state)


# ---- what a pass cannot do without ---------------------------------------

def _mean_length(c):
    lo, hi = c["shortest"], c["longest"]
    return lo if lo == hi else (hi - lo) / math.log(hi / lo)


def _mean_window(c):
    """Mean of the smaller of a length and the window, lengths spread evenly
    over their logarithm."""
    lo, hi, w = c["shortest"], c["longest"], c["window"]
    if not w or w >= hi:
        return _mean_length(c)
    if w <= lo:
        return w
    return ((w - lo) + w * math.log(hi / w)) / math.log(hi / lo)


def work(case):
    c = case
    size = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "qk":
        t, h, kv, d = c["tokens"], c["heads"], c["kv_heads"], c["head"]
        row = 2 * size * d * (h + kv) + 4
        if c["train"]:
            row += 2 * size * d * (h + kv)
        else:
            row += 2 * size * d * kv + 8
        return {"bytes": t * row + 16 * d, "flops": (30 if c["train"] else 10) * t * (h + kv) * d}
    if c["op"] == "attend":
        n, h, kv, d = c["seqs"], c["heads"], c["kv_heads"], c["head"]
        tokens = n * _mean_window(c)
        own_rows = (3 if c["gate"] else 2) * n * h * d * size
        return {"bytes": int(tokens * (2 * kv * d * size + 4 / c["page"]) + own_rows + 4 * n),
                "flops": int(4 * tokens * h * d)}
    if c["op"] == "pages":
        n, page, share = c["rows"], c["page"], c["share"]
        old = -(-n // share)
        lo, hi = max(1, c["longest"] // 8), c["longest"]
        mean = lo if lo == hi else (hi - lo) / math.log(hi / lo)
        held = old * (mean / page + 0.5)
        pool = held * 4 / 3 + 2 * n + 8
        one = 2 * 2 * c["layers"] * 2 * page * c["width"]      # one page read and written in both pools
        if c["what"] == "step":
            # rows that go on share a parent or not; a page in 16 begins anew
            copied = max(0.0, n - old * (1 - (1 - 1 / old) ** n)) * 0.95 * (1 - 1 / page)
            table = n * (mean / page + c["longest"] // page + 2)
        else:
            # the holes in front of the end of what is used
            share_live = held / pool + (1 - held / pool) * 0.05
            copied = pool * share_live * (1 - share_live)
            table = 2 * held
        return {"bytes": int(4 * table + 8 * pool + copied * one), "flops": int(2 * pool + table)}
    t, v = c["rows"], c["vocab"]
    b = t * v * size + 20 * t + 8 * t * c["top"]
    if c["train"]:
        b += t * v * size + 8 * t
    return {"bytes": b, "flops": (20 if c["train"] else 8) * t * v}


# ---- the definitions in 64 bits ------------------------------------------

def _exact_qk(c):
    out = {}
    pos, rot, d = c["positions"].to(F64), c["rot"], c["head"]
    mat = None
    if rot:
        turn = torch.polar(torch.ones((), dtype=F64, device="cuda"), torch.outer(pos, c["inv_freq"]))

        def mat(x):
            if c["pairs"]:
                z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous())
                z = torch.view_as_real(z * turn[:, None]).reshape(*x.shape[:2], rot)
            else:
                z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn[:, None]
                z = torch.cat((z.real, z.imag), 2)
            return torch.cat((z, x[..., rot:]), 2) if rot < d else z
    for name in ("q", "k"):
        x = c[name].to(F64).requires_grad_(c["train"])
        w = c[name + "_weight"].to(F64).requires_grad_(c["train"])
        y = x * (x.square().mean(2, keepdim=True) + EPS).rsqrt() * w
        if mat:
            y = mat(y)
        elif name == "q":
            y = y * torch.pow(1 + (pos + 1) / TEMPERATURE[0], TEMPERATURE[1]).view(-1, 1, 1)
        out[name] = y.detach()
        if c["train"]:
            out["d_" + name], out["d_%s_weight" % name] = torch.autograd.grad(y, (x, w), c["d_" + name].to(F64))
    if not c["train"]:
        place = c["tables"][c["rows"].long(), (c["positions"] // c["page"]).long()].long() * c["page"]
        place = place + c["positions"].long() % c["page"]
        for name, new in (("k_cache", out.pop("k")), ("v_cache", c["v"].to(F64))):
            full = c[name].to(F64).flatten(0, 1)
            out[name] = full.index_copy(0, place, new).view(c[name].shape)
    return out


def _exact_attend(c):
    kv, group, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["head"]
    rows = []
    for i in range(c["seqs"]):
        n = int(c["lengths"][i])
        at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
        where = c["tables"][i].long()[at // c["page"]] * c["page"] + at % c["page"]
        heads = []
        for j in range(kv):
            k = c["k_cache"].flatten(0, 1)[where, j].to(F64)
            v = c["v_cache"].flatten(0, 1)[where, j].to(F64)
            q = c["q"][i, j * group:(j + 1) * group].to(F64)
            heads.append(torch.mm(torch.softmax(torch.mm(k, q.t().contiguous()) * d ** -0.5, 0).t().contiguous(), v))
        rows.append(torch.cat(heads))
    out = torch.stack(rows)
    return {"out": out * torch.sigmoid(c["gates"].to(F64)) if c["gate"] else out}


def _exact_step(c):
    page, wide = c["page"], c["tables"].shape[1]
    old, lens, refs = c["tables"].tolist(), c["lengths"].tolist(), c["refs"].tolist()
    rows = []
    for p, g in zip(c["parents"].tolist(), c["grow"].tolist()):
        n = lens[p] if p >= 0 else 0
        rows.append((n, g, old[p][:-(-n // page)] if p >= 0 else []))
    for t, n in zip(old, lens):
        for x in t[:-(-n // page)]:
            refs[x] -= 1
    for _, _, t in rows:
        for x in t:
            refs[x] += 1
    free = iter([i for i, r in enumerate(refs) if r <= 0])
    shared, writers = list(refs), {}
    for i, (n, g, t) in enumerate(rows):
        if g > 0 and n % page:
            writers.setdefault(t[-1], []).append(i)
    tables, lengths, moved, missing = [], [], [], 0
    for i, (n, g, t) in enumerate(rows):
        t = list(t)
        if g > 0 and n % page:
            p = t[-1]
            if shared[p] > 1 and (shared[p] != len(writers[p]) or writers[p][0] != i):
                t[-1] = next(free, -1)
                refs[p] -= 1
                missing += t[-1] < 0
                if t[-1] >= 0:
                    moved.append((p, t[-1]))
        need = -(-(n + g) // page)
        missing += max(0, need - wide)
        while len(t) < min(need, wide):
            t.append(next(free, -1))
            missing += t[-1] < 0
        for x in t[len(t) - (min(need, wide) - -(-n // page)):]:
            if x >= 0:
                refs[x] = 1
        tables.append(t + [-1] * (wide - len(t)))
        lengths.append(min(n + g, wide * page))
    for _, x in moved:
        refs[x] = 1
    out = {k: torch.tensor(v, dtype=I32, device="cuda")
           for k, v in (("tables", tables), ("lengths", lengths), ("refs", refs), ("missing", [missing]))}
    for name, pool in zip("kv", c["pools"]):
        out[name] = pool.clone()
        for a, b in moved:
            out[name][:, b] = pool[:, a]
    return out


def _exact_pack(c):
    refs = c["refs"].tolist()
    live = [i for i, r in enumerate(refs) if r > 0]
    holes = [i for i, r in enumerate(refs[:len(live)]) if r <= 0]
    to = {i: i for i in live if i < len(live)}
    moved = list(zip([i for i in live if i >= len(live)], holes))
    to.update(moved)
    packed = [0] * len(refs)
    for i in live:
        packed[to[i]] = refs[i]
    tables = []
    for t, n in zip(c["tables"].tolist(), c["lengths"].tolist()):
        used = -(-n // c["page"])
        tables.append([to.get(x, -1) for x in t[:used]] + [-1] * (len(t) - used))
    new_id = [to.get(i, -1) for i in range(len(refs))]
    out = {k: torch.tensor(v, dtype=I32, device="cuda")
           for k, v in (("tables", tables), ("refs", packed), ("new_id", new_id), ("live", [len(live)]))}
    for name, pool in zip("kv", c["pools"]):
        out[name] = pool.clone()
        for a, b in moved:
            out[name][:, b] = pool[:, a]
    return out


def _exact_score(c):
    names = ["logprobs", "entropy", "lse"] + (["ids", "top"] if c["top"] else []) + (["d_logits"] if c["train"] else [])
    out = {k: [] for k in names}
    # a few rows at a time: 64 bits of a large batch do not fit
    step = max(1, (1 << 27) // c["vocab"])
    for i in range(0, c["rows"], step):
        x = c["logits"][i:i + step].to(F64).requires_grad_(c["train"])
        masked = torch.isinf(x.detach())
        z = (x.masked_fill(masked, 0.0) / CAP).tanh() * CAP if c["cap"] else x.masked_fill(masked, 0.0)
        logp = torch.log_softmax(z.masked_fill(masked, -1e9), 1)
        h = -(logp.exp() * logp).masked_fill(masked, 0.0).sum(1)
        t = c["targets"][i:i + step]
        there = (t >= 0) & (t < c["vocab"])
        lp = torch.take_along_dim(logp, t.clamp(0, c["vocab"] - 1)[:, None], 1)[:, 0] * there
        out["logprobs"].append(lp.detach())
        out["entropy"].append(h.detach())
        out["lse"].append((z - logp)[:, 0].detach())
        if c["top"]:
            ids = torch.argsort(-x.detach(), dim=1, stable=True)[:, :c["top"]]
            out["ids"].append(ids.to(I32))
            out["top"].append(torch.take_along_dim(logp.detach().masked_fill(masked, -math.inf), ids, 1))
        if c["train"]:
            s = (lp * c["d_logprobs"][i:i + step]).sum() + (h * c["d_entropy"][i:i + step]).sum()
            out["d_logits"].append(torch.autograd.grad(s, x)[0])
    return {k: torch.cat(v) for k, v in out.items()}


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "pages":
        return _exact_step(c) if c["what"] == "step" else _exact_pack(c)
    return {"qk": _exact_qk, "attend": _exact_attend, "score": _exact_score}[c["op"]](c)

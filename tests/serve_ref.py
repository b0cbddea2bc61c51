"""Plain implementations in 64 bits, on the CPU, of the operators around a paged
key-value cache: what the GPU tests compare against.  They share no code with
the library."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U = 2.0 ** -24          # half a step of binary32, relative


# ---- norms and rotation of heads ------------------------------------------

def turns(positions, inv_freq, interleaved, D, back=False):
    """[T, D, D] matrices that turn a head's values."""
    T, n = positions.shape[0], inv_freq.numel()
    m = torch.eye(D, dtype=F64).repeat(T, 1, 1)
    ang = positions.double()[:, None] * inv_freq[None, :]
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        c, s = torch.cos(ang[:, i]), torch.sin(ang[:, i])
        m[:, a, a], m[:, b, b] = c, c
        m[:, a, b], m[:, b, a] = -s, s
    return m.transpose(1, 2) if back else m


def temperature(positions, temp):
    if temp is None:
        return torch.ones(positions.shape[0], 1, 1, dtype=F64)
    return ((1 + (positions.double() + 1) / temp[0]) ** temp[1])[:, None, None]


def rope(x, w, positions, inv_freq, interleaved, eps, temp=None):
    """(y, size): the normed, turned head values, and the sums of their terms'
    absolute values."""
    x = x.double()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    t = temperature(positions, temp) if temp is not None else 1.0
    if inv_freq is None:
        return n * t, (n * t).abs()
    m = turns(positions, inv_freq, interleaved, x.shape[-1])
    return (torch.einsum("tab,thb->tha", m, n) * t, torch.einsum("tab,thb->tha", m.abs(), n.abs()) * t)


def rope_grad(dy, x, w, positions, inv_freq, interleaved, eps, temp=None, absolute=False):
    """(dx, dw) by their formulas; with absolute every term enters by its
    absolute value: the scale of the roundings."""
    A = (lambda v: v.abs()) if absolute else (lambda v: v)
    x, d = x.double(), A(dy.double())
    if temp is not None:
        d = d * temperature(positions, temp)
    if inv_freq is not None:
        m = turns(positions, inv_freq, interleaved, x.shape[-1], back=True)
        d = torch.einsum("tab,thb->tha", A(m), d)
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    hat = A(x * inv)
    dw = (d * hat).sum((0, 1))
    g = d * A(w.double())
    mean = hat * (g * hat).mean(-1, keepdim=True)
    return inv * (g + mean if absolute else g - mean), dw


# ---- attention over pages -----------------------------------------------------

def attend(q, k_cache, v_cache, tables, lengths, scale, window, gate=None):
    """A list by sequence of dicts: out [Hq, D] and lse [Hq]; size, the mean of
    |v| by the same weights; smax [Hq], the largest |score|; dots [Hq], the
    largest sum of a score's terms' absolute values; n, the tokens."""
    P, page, Hkv, D = k_cache.shape
    Hq = q.shape[1]
    res = []
    for b in range(q.shape[0]):
        n = min(max(int(lengths[b]), 0), tables.shape[1] * page)
        at = [i for i in range(max(0, n - window) if window else 0, n)
              if 0 <= int(tables[b, i // page]) < P]
        group = Hq // Hkv
        if not at:
            z = torch.zeros(Hq, D, dtype=F64)
            res.append(dict(out=z, lse=torch.full((Hq,), -math.inf, dtype=F64), size=z.clone(),
                            smax=torch.zeros(Hq, dtype=F64), dots=torch.zeros(Hq, dtype=F64), n=0))
            continue
        i = torch.tensor(at)
        pg = tables[b].long()[i // page]
        k = k_cache[pg, i % page].double().repeat_interleave(group, 1)     # [n, Hq, D]
        v = v_cache[pg, i % page].double().repeat_interleave(group, 1)
        qq = q[b].double()
        s = (k * qq).sum(-1) * scale
        lse = torch.logsumexp(s, 0)
        p = torch.exp(s - lse)[..., None]
        out = (p * v).sum(0)
        size = (p * v.abs()).sum(0)
        if gate is not None:
            g = torch.sigmoid(gate[b].double())
            out, size = out * g, size * g
        res.append(dict(out=out, lse=lse, size=size, smax=s.abs().amax(0),
                        dots=((k * qq).abs().sum(-1) * scale).amax(0), n=len(at)))
    return res


# ---- page tables ------------------------------------------------------------------

def ceil_div(a, b):
    return -(-a // b)


def pages_update(tables, lengths, refs, page, parents=None, grow=None):
    """(tables, lengths, refs, missing, copies) as lists, step by step."""
    cols, P = len(tables[0]) if tables else 0, len(refs)
    valid = lambda p: 0 <= p < P
    held = [min(max(n, 0), cols * page) for n in lengths]
    old = [list(t[:ceil_div(n, page)]) for t, n in zip(tables, held)]
    if parents is None:
        parents = list(range(len(old)))
    new = []
    for i, r in enumerate(parents):
        has = 0 <= r < len(old)
        g = max(grow[i], 0) if grow is not None else 0
        new.append(dict(t=list(old[r]) if has else [], n=held[r] if has else 0, g=g))
    refs = list(refs)
    for t in old:
        for p in t:
            if valid(p):
                refs[p] -= 1
    for r in new:
        for p in r["t"]:
            if valid(p):
                refs[p] += 1
    # who writes into a page that is filled in part
    open_rows = {}
    for i, r in enumerate(new):
        if r["g"] > 0 and r["n"] % page and valid(r["t"][-1]):
            open_rows.setdefault(r["t"][-1], []).append(i)
    copies_of = {}
    for p, who in open_rows.items():
        if refs[p] == 1:
            continue
        for i in who:
            if not (refs[p] == len(who) and i == min(who)):
                copies_of[i] = p
    free = [p for p in range(P) if refs[p] <= 0]
    missing, copies = 0, []

    def take():
        nonlocal missing
        if free:
            return free.pop(0)
        missing += 1
        return -1

    for i, r in enumerate(new):
        if i in copies_of:
            p = take()
            refs[copies_of[i]] -= 1
            r["t"][-1] = p
            if p >= 0:
                refs[p] = 1
                copies.append((copies_of[i], p))
        want = ceil_div(r["n"] + r["g"], page)
        missing += max(0, want - cols)
        while len(r["t"]) < min(want, cols):
            p = take()
            r["t"].append(p)
            if p >= 0:
                refs[p] = 1
    out = [r["t"] + [-1] * (cols - len(r["t"])) for r in new]
    return out, [min(r["n"] + r["g"], cols * page) for r in new], refs, missing, copies


def pages_compact(tables, lengths, refs, page):
    """(tables, refs, new_id, live, moves) as lists."""
    P = len(refs)
    used = [p for p in range(P) if refs[p] > 0]
    n = len(used)
    holes = [p for p in range(n) if refs[p] <= 0]
    moves = list(zip([p for p in used if p >= n], holes))
    to = {p: p for p in used if p < n}
    to.update(moves)
    new_id = [to.get(p, -1) for p in range(P)]
    packed = [0] * P
    for p in used:
        packed[to[p]] = refs[p]
    out = []
    for t, m in zip(tables, lengths):
        have = ceil_div(min(max(m, 0), len(t) * page), page)
        out.append([to.get(p, -1) if i < have else -1 for i, p in enumerate(t)])
    return out, packed, new_id, n, moves


# ---- scores of tokens ------------------------------------------------------------------

def score(logits, targets=None, softcap=0.0, scale=1.0, top=0):
    """A dict as token_logprobs gives, with z and logp [T, V] too."""
    x = logits.double()
    masked = x == -math.inf
    z = (softcap * torch.tanh(x / softcap) if softcap else x) * scale
    z = torch.where(masked, -math.inf, z)
    lse = torch.logsumexp(z, 1)
    none = masked.all(1)
    logp = torch.where(masked | none[:, None], -math.inf, z - torch.where(none, 0.0, lse)[:, None])
    p = torch.exp(logp)
    out = dict(z=z, logp=logp, lse=lse, entropy=-torch.where(p > 0, p * logp, 0.0).sum(1))
    if targets is not None:
        ok = (targets >= 0) & (targets < x.shape[1])
        lp = logp.gather(1, torch.where(ok, targets, 0)[:, None])[:, 0]
        out["logprobs"] = torch.where(ok, lp, 0.0)
    if top:
        out["top_ids"] = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        out["top_logprobs"] = logp.gather(1, out["top_ids"])
    return out


def score_grad(logits, targets, d_logprobs, d_entropy, softcap=0.0, scale=1.0, absolute=False):
    r = score(logits, targets, softcap, scale)
    x, logp = logits.double(), r["logp"]
    p = torch.exp(logp)
    A = (lambda v: v.abs()) if absolute else (lambda v: v)
    lg = torch.where(p > 0, logp, 0.0)
    d = torch.zeros_like(x)
    if d_logprobs is not None:
        ok = (targets >= 0) & (targets < x.shape[1])
        g = A(torch.where(ok, d_logprobs.double(), 0.0))[:, None]
        d = g * p if absolute else -g * p
        d = d.scatter_add(1, torch.where(ok, targets, 0)[:, None], g)
    if d_entropy is not None:
        h = A(d_entropy.double())[:, None]
        e = r["entropy"][:, None]
        d = d + h * p * (lg.abs() + e) if absolute else d - h * p * (lg + e)
    dz = scale * (1 - torch.tanh(x / softcap) ** 2) if softcap else scale
    return torch.where(x == -math.inf, 0.0, d * dz)

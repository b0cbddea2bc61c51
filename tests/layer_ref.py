"""Plain implementations in 64 bits, on the CPU, of the operators around the
expert block: what the GPU tests compare against.  They share no code with the
library or its CPU oracle."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U = 2.0 ** -24          # half a step of binary32, relative


# ---- routing -------------------------------------------------------------

def scores(logits, softmax: bool):
    x = logits.double()
    if not softmax:
        return torch.sigmoid(x)
    m = x.amax(1, keepdim=True)
    e = torch.where(x > -math.inf, torch.exp(x - torch.where(m > -math.inf, m, 0.0)), 0.0)
    tot = e.sum(1, keepdim=True)
    return torch.where(tot > 0, e / tot, 0.0)


def select(logits, bias, groups, kept, top, topn, softmax):
    """Chosen experts, by the binary32 comparison the routing specifies."""
    T, E = logits.shape
    s = scores(logits, softmax).float()
    u = s + (bias if bias is not None else torch.zeros(E))
    rows = []
    for t in range(T):
        ug = u[t].view(groups, -1)
        best = torch.sort(ug, dim=1, descending=True).values[:, :topn]
        gs = best[:, 0] if topn == 1 else best[:, 0] + best[:, 1]
        keep = sorted(range(groups), key=lambda g: (-gs[g].item(), g))[:kept]
        size = E // groups
        cand = [e for g in keep for e in range(g * size, (g + 1) * size)]
        rows.append(sorted(cand, key=lambda e: (-u[t, e].item(), e))[:top])
    return torch.tensor(rows, dtype=torch.int32).reshape(T, top)


def weights(logits, idx, scale, softmax, normed):
    s = scores(logits, softmax).gather(1, idx.long())
    if normed:
        d = s.sum(1, keepdim=True)
        s = torch.where(d > 0, s / d, 0.0)
    return s * scale


def route_grad(logits, idx, dw, scale, softmax, normed):
    """The gradient by its formula; ids outside [0, E) add nothing."""
    T, E = logits.shape
    ok = (idx >= 0) & (idx < E)
    at = torch.where(ok, idx, 0).long()
    s_all = scores(logits, softmax)
    s = torch.where(ok, s_all.gather(1, at), 0.0)
    dw = torch.where(ok, dw.double(), 0.0)
    d = torch.ones(T, 1, dtype=F64)
    if normed:
        d = s.sum(1, keepdim=True)
    q = torch.where(d > 0, s / torch.where(d > 0, d, 1.0), 0.0)
    c = (dw * q).sum(1, keepdim=True)
    if softmax:
        g = q * (dw - c) if normed else s * dw
    else:
        x = logits.double().gather(1, at)
        ds = torch.where(ok, torch.sigmoid(x) * torch.sigmoid(-x), 0.0)
        g = torch.where(d > 0, ds / torch.where(d > 0, d, 1.0), 0.0) * (dw - c if normed else dw)
    out = torch.zeros(T, E, dtype=F64)
    if softmax and not normed:
        out = -s_all * c
    return scale * out.scatter_add(1, at, torch.where(ok, g, 0.0))


# ---- the step between two blocks -------------------------------------------

def norm_step(r, o, post, gate, pre, eps, alpha, beta):
    """(r', x, y, g): the forward in 64 bits (y the normed block output, g the
    gate's sigmoid)."""
    r = r.double()
    y, g = None, torch.ones(r.shape[0], 1, dtype=F64)
    if o is not None:
        o = o.double()
        y = o / torch.sqrt((o * o).mean(1, keepdim=True) + eps) * post.double()
        if gate is not None:
            g = torch.sigmoid(gate.double())
        r = alpha * r + beta * g * y
    x = None
    if pre is not None:
        x = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * pre.double()
    return r, x, y, g


def norm_step_grad(rp, d_rp, dx, o, post, gate, pre, eps, alpha, beta, absolute=False):
    """The gradients by their formulas, from the forward's r'.  With absolute
    every term enters by its absolute value: the scale of the roundings."""
    def A(v):
        return v.abs() if absolute else v

    def minus(a, b):
        return a + b if absolute else a - b

    rp = rp.double()
    out = {}
    d = A(d_rp.double()) if d_rp is not None else torch.zeros_like(rp)
    if dx is not None:
        inv = 1 / torch.sqrt((rp * rp).mean(1, keepdim=True) + eps)
        hat, dx = A(rp * inv), A(dx.double())
        out["d_pre_weight"] = (dx * hat).sum(0)
        w = A(pre.double()) * dx
        d = d + inv * minus(w, hat * (w * hat).mean(1, keepdim=True))
    if o is None:
        out["d_residual"] = d            # r' is the residual itself: alpha plays no part
        return out
    out["d_residual"] = A(torch.tensor(alpha, dtype=F64)) * d
    d = A(torch.tensor(beta, dtype=F64)) * d
    o = o.double()
    inv = 1 / torch.sqrt((o * o).mean(1, keepdim=True) + eps)
    hat, post = A(o * inv), A(post.double())
    if gate is not None:
        s = torch.sigmoid(gate.double())
        dg = d * hat * post * s * torch.sigmoid(-gate.double())
        out["d_gate"] = dg.sum(1, keepdim=True) if gate.shape[1] == 1 and hat.shape[1] != 1 else dg
        d = d * s
    out["d_post_weight"] = (d * hat).sum(0)
    w = post * d
    out["d_o"] = inv * minus(w, hat * (w * hat).mean(1, keepdim=True))
    return out


# ---- e4m3 products ----------------------------------------------------------

def expand(s, n, k, rows):
    """Block scales [ceil(n/128) or n, k/128] as one value per element."""
    s = s.double()
    if not rows:
        s = s.repeat_interleave(128, 0)[:n]
    return s.repeat_interleave(128, 1)


def codes(q):
    return q.view(torch.float8_e4m3fn).to(F64)


def product(a, sa, b, sb, rows):
    """(y, size): the scaled product in 64 bits and the sum of its terms'
    absolute values."""
    x = codes(a) * expand(sa, a.shape[0], a.shape[1], True)
    w = codes(b) * expand(sb, b.shape[0], b.shape[1], rows)
    return x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()


def quantise(v, block_rows, block_cols):
    """(codes as values, scales) of v by blocks, the scale and the quotient
    rounded to binary32 as the recipe has them; v padded with zeros."""
    r, c = v.shape
    p = torch.nn.functional.pad(v.double(), (0, -c % block_cols, 0, -r % block_rows))
    R, C = p.shape[0] // block_rows, p.shape[1] // block_cols
    p = p.view(R, block_rows, C, block_cols)
    s = (p.abs().amax((1, 3)) / 448.0).float()
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (p / s.double()[:, None, :, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(R * block_rows, C * block_cols).view(torch.uint8), s

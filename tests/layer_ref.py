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

"""The 64-bit formulas the GPU tests of the operators around the expert block
compare with, against central differences of their forwards (h = 1e-6: the
difference is off by h^2 f''' / 6 and 1e-16 / h, so 1e-7 holds both for values
of this size)."""
import pytest
import torch

import layer_ref as ref


def numeric(f, x, h=1e-6):
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + h
        up = f()
        flat[i] = v - h
        dn = f()
        flat[i] = v
        out[i] = (up - dn) / (2 * h)
    return g


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("normed", [True, False])
def test_route_gradient_formula(softmax, normed):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 12, generator=g, dtype=torch.float64)
    dw = torch.randn(3, 4, generator=g, dtype=torch.float64)
    idx = torch.stack([torch.randperm(12, generator=g)[:4] for _ in range(3)]).int()
    got = ref.route_grad(x, idx, dw, 2.5, softmax, normed)
    want = numeric(lambda: (ref.weights(x, idx, 2.5, softmax, normed) * dw).sum().item(), x)
    assert (got - want).abs().max() < 1e-7


@pytest.mark.parametrize("gate_cols", [0, 1, 6])
@pytest.mark.parametrize("after", [True, False])
def test_norm_step_gradient_formulas(after, gate_cols):
    g = torch.Generator().manual_seed(2)
    T, H = 3, 6

    def rn(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    r, pre, c_r, c_x = rn(T, H), 1 + rn(H) / 10, rn(T, H), rn(T, H)
    o = post = gate = None
    if after:
        o, post = rn(T, H), 1 + rn(H) / 10
        gate = rn(T, gate_cols) if gate_cols else None
    elif gate_cols:
        return

    def f():
        rp, x, _, _ = ref.norm_step(r, o, post, gate, pre, 1e-3, 0.9, 0.4)
        return ((rp * c_r).sum() + (x * c_x).sum()).item()

    rp = ref.norm_step(r, o, post, gate, pre, 1e-3, 0.9, 0.4)[0]
    got = ref.norm_step_grad(rp, c_r, c_x, o, post, gate, pre, 1e-3, 0.9, 0.4)
    for name, leaf in (("d_residual", r), ("d_pre_weight", pre), ("d_o", o), ("d_post_weight", post),
                       ("d_gate", gate)):
        if leaf is not None:
            assert (got[name] - numeric(f, leaf)).abs().max() < 1e-7, name

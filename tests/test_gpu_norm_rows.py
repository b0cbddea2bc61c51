"""Tokens of the norm step's gradients do not reach one another: with a token
whose sums are not finite among them, every other token's gradients keep their
bits.  The batches have more tokens than workgroups, so that each workgroup
goes on to another token after the bad one."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import test_gpu_norm as nm
from gpu_util import device

pytestmark = pytest.mark.gpu

ROWS = ("d_residual", "d_o", "d_gate")
T, BAD = 3500, [2, 5, 11, 600]       # at most 1,536 workgroups: three tokens and more each


def spoil(dc, r, what):
    """The batch with tokens BAD made bad in one input."""
    dc, r = dict(dc), r.clone()
    if what in ("nan r'", "inf r'"):
        r[BAD, 7] = float(what.split()[0])
    elif what == "nan o":
        dc["o"] = dc["o"].clone()
        dc["o"][BAD, 7] = float("nan")
    elif what == "nan d_residual_out":
        dc["d_r"] = dc["d_r"].clone()
        dc["d_r"][BAD, 7] = float("nan")
    else:                            # "nan d_x", or finite ones whose sum of products is infinite
        dc["d_x"] = dc["d_x"].clone()
        dc["d_x"][BAD] = float("nan") if what == "nan d_x" else 3e38 * r[BAD].sign().to(dc["d_x"].dtype)
    return dc, r


# widths whose 8-column chunks fill whole waves (512), leave lanes without
# columns (64 .. 2,880; 8,200 with two chunks a thread) and odd ones
@pytest.mark.parametrize("H", [64, 128, 264, 512, 768, 1000, 2880, 8200, 9, 1001])
@pytest.mark.parametrize("gate", [None, "token", "channel"])
def test_bad_tokens_reach_no_other(H, gate):
    for dtype in (torch.bfloat16, torch.float32):
        c = nm.make(T if H < 8000 else 1100, H, dtype, gate, True, H)
        dc = nm.on(device(), c)
        r, _ = gl.norm_residual(dc["residual"], **nm.kw(dc))
        want = gl.norm_residual_backward(r, dc["d_r"], dc["d_x"], **nm.kw(dc))
        good = torch.ones(r.shape[0], dtype=torch.bool, device=r.device)
        good[BAD] = False
        for what in ("nan r'", "inf r'", "nan o", "nan d_x", "large d_x", "nan d_residual_out"):
            bad, rb = spoil(dc, r, what)
            got = gl.norm_residual_backward(rb, bad["d_r"], bad["d_x"], **nm.kw(bad))
            for k in ROWS:
                if k in want:
                    assert torch.equal(got[k][good], want[k][good]), (dtype, what, k)
            assert not torch.isfinite(got["d_o"][BAD].float()).all(1).any(), (dtype, what)

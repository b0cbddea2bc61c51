"""Every form of the dense e4m3 product: both result types, each tile, the large
tiles with and without whole rounds of them before a last round that is uncut
or cut into halves or quarters.  Tolerances are those of test_gpu_matmul.py."""
import pytest
import torch

import group_limited_routing_sigmoid_amd as gl
import matmul_forms as mf
import test_gpu_matmul as mm

FORMS, SMALL = mf.table()

# a shape with ragged ends for each case that bf16 or binary32 results reach
SHAPES = {
    torch.bfloat16: [(1, 1), (31, 4097), (8193, 1), (33, 4097), (33, 8193), (65, 8193), (65, 16385), (257, 16385),
                     (129, 16385), (577, 16384), (1025, 16385), (769, 16385), (16385, 513), (6945, 1793), (20000, 1025),
                     (20000, 513), (193, 16385), (1793, 7937), (16385, 1537), (8065, 2817), (20000, 769)],
    torch.float32: [(1, 1), (31, 4097), (8193, 1), (33, 4097), (33, 8193), (65, 8193), (65, 16385), (193, 16385),
                    (8065, 769), (20000, 513), (20000, 769), (385, 16385), (10241, 769), (673, 16384), (20000, 1025)],
}


def cases(dtype):
    return [mf.case(M, N, dtype is torch.float32, FORMS, SMALL) for M, N in SHAPES[dtype]]


@pytest.mark.parametrize("dtype", SHAPES)
def test_shapes_reach_every_form(dtype):
    heights = sorted({h * y + d for h in (128, 192, 224, 256) for y in range(1, 40) for d in (0, 1)}
                     | {1, 33, 65, 100, 10241, 16385, 20000})
    widths = sorted({256 * y + d for y in range(33) for d in (0, 1)} - {0} | {17, 33, 65, 129, 16384, 16385})
    reached = {mf.case(M, N, dtype is torch.float32, FORMS, SMALL) for M in heights for N in widths}
    assert reached <= set(cases(dtype)), sorted(reached - set(cases(dtype)))
    built = {(f[0], f[1]) for f in FORMS if f[3 if dtype is torch.float32 else 2] > 0}
    assert built == {c[1:3] for c in cases(dtype)}          # no tile that no call reaches


def run(M, N, K, rows, dtype, seed):
    from gpu_util import device
    a, sa = mm.operand(M, K, 1, seed, device())
    b, sb = mm.operand(N, K, 1 if rows else 128, seed + 1, device())
    out = torch.full((M, N), float("nan"), dtype=dtype, device=device())
    gl.matmul_e4m3(a, sa, b, sb, dtype=dtype, out=out)
    mm.check(out, a, sa, b, sb, rows)
    assert torch.equal(out, gl.matmul_e4m3(a, sa, b, sb, dtype=dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("dtype,M,N", [(d, *s) for d in SHAPES for s in SHAPES[d]])
def test_form(dtype, M, N, rows):
    for K in (128, 256, 640):                # one block, both stages, an odd number of blocks
        run(M, N, K, rows, dtype, M + N + K)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", SHAPES)
@pytest.mark.parametrize("M,N,K,rows", [(5120, 2560, 4224, True), (4099, 5120, 2560, False), (4099, 2560, 5120, False),
                                        (8192, 5120, 5120, False), (64, 5125, 2560, False), (1, 5120, 5120, False)])
def test_layer_products(M, N, K, rows, dtype):
    run(M, N, K, rows, dtype, M + K)

"""The norm and the quantisation of rows, held to bounds that do not grow with the row's length.

A thread adds at most 65 squares, its wavefront joins 64 lanes in 6 additions and the workgroup at most 16 wavefronts: every
square passes 87 additions at most, each right to u = 2^-24.  The squares: z is right to u (2 u of its square), the product is
exact within the addition.  Half of that for the root, and u each for the division by c (half), the addition of eps (half),
the root, its inverse (2 u each) and three products: (87 + 2 + 1 + 1) / 2 + 4 + 3 < 54 u.  TOP = 56 u is above it.
"""
import math

import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import close, half, rand, types, U
from test_gpu_quantized import EPS, LEAST, LENGTHS, norm_ref

pytestmark = pytest.mark.gpu
TOP = 56 * U


def check_rows(q, scales, ref, off):
    step = ref.abs().amax(dim=1).clamp(min=LEAST) / 127
    assert ((scales.cpu().double() - step).abs() <= (off + 4 * U) * step).all()
    far = (q.cpu().double() - ref / step[:, None]).abs()
    assert (far <= 0.5 + 127 * (off + 4 * U)).all(), float(far.max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", LENGTHS)
def test_lengths(c, dtype):
    t = types()[dtype]
    x, r, w = rand((33, c), 1, t, 3.0), rand((33, c), 2, t), rand((c,), 3, t)
    for residual in (None, r):
        z, y = norm_ref(x, w, EPS, residual)
        got = dyra.dyra_norm(x.cuda(), w.cuda(), EPS, residual=None if residual is None else residual.cuda())
        got = got if residual is None else got[0]
        close(got, y, TOP * y.abs() + half(t) * (1 + TOP) * y.abs())
        q, scales, *_ = dyra.dyra_norm_quantize(x.cuda(), w.cuda(), EPS, residual=None if residual is None else residual.cuda())
        check_rows(q, scales, y, TOP)
    check_rows(*dyra.dyra_quantize(x.cuda()), x.double(), 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [3, 64, 1000, 4096, 9000, 65536])
def test_quantised_extremes(c, dtype):
    """dyra_quantize takes no sum: its bounds are those of a division and a product, in rows of any size."""
    import torch
    t = types()[dtype]
    x = rand((20, c), 21, t)
    big, tiny = torch.finfo(t).max, torch.finfo(t).tiny
    for row, v in {3: 0.0, 5: big, 7: tiny, 9: -big}.items():
        x[row, c // 2] = v
    x[3], x[7], x[11], x[13] = 0.0, tiny, big, -big
    x[15], x[17] = x[15].double().mul(1e30).to(t), x[17].double().mul(1e-30).to(t)
    x[19] = tiny * 100
    check_rows(*dyra.dyra_quantize(x.cuda()), x.double(), 0.0)
    x[1, 0], x[2, c - 1], x[4, c // 2] = math.inf, math.nan, -math.inf
    q, scales = dyra.dyra_quantize(x.cuda())
    assert scales[[1, 2, 4]].isnan().all() and (q[[1, 2, 4]] == 0).all()

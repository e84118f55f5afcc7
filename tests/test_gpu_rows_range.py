"""Norms of rows whose values or weights span much of float32's range: what is made on the way (z 2^-96 of rows whose
squares leave the range, z w) must not fall below it where the result does not."""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import half, rand, types
from test_gpu_quantized import check_rows, check_sum, norm_ref, relative

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [64, 1000, 4100, 40000])
def test_small_values_beside_one_whose_square_is_past_the_range(c, dtype):
    """One value of 2^70, others from 2^-48 on: results from 2^-118 on are normal numbers, right to the bound of any other."""
    import torch
    t = types()[dtype]
    g = torch.Generator().manual_seed(c)
    x = torch.ldexp(rand((12, c), 1, torch.float32).abs() + 1, torch.randint(-48, 30, (12, c), generator=g)).to(t)
    x[:, c // 3] = 2.0 ** 70
    w = (rand((c,), 2, torch.float32).abs() + 1).to(t)
    for weight in (None, w):
        y = dyra.dyra_norm(x.cuda(), None if weight is None else weight.cuda(), 1e-5)
        ref = norm_ref(x, weight, 1e-5, None)[1].abs()   # (check_norm allows 1e-30)
        assert ref[ref > 0].min() > 2.0 ** -126
        off = (y.cpu().double().abs() - ref).abs()
        assert (off <= (relative(c) + half(t) * (1 + relative(c))) * ref).all(), float((off / ref).max())
    q, scales = dyra.dyra_norm_quantize(x.cuda(), w.cuda(), 1e-5)
    check_rows(q, scales, norm_ref(x, w, 1e-5, None)[1], True)


# exponents of the values, of the weights and of eps: z w is below 2^-126 where z w / sqrt(mean z^2 + eps) is above it
SMALL = [(-84, -84, -126), (-20, -117, -40), (-63, -60, -126), (-126, -20, -126), (100, -149, -20), (-20, -125, -126)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [3, 64, 1000, 4100, 40000])
@pytest.mark.parametrize("ez,ew,ee", SMALL)
def test_small_products_of_values_and_weights(c, dtype, ez, ew, ee):
    import torch
    t = types()[dtype]
    x = torch.ldexp(rand((9, c), 3, torch.float32), torch.tensor(ez)).to(t)
    r = torch.ldexp(rand((9, c), 4, torch.float32), torch.tensor(ez)).to(t)
    w = torch.ldexp(rand((c,), 5, torch.float32), torch.tensor(ew)).to(t)
    x[4], r[4] = 0.0, 0.0
    z, y = norm_ref(x, w, 2.0 ** ee, r)
    q, scales, s = dyra.dyra_norm_quantize(x.cuda(), w.cuda(), 2.0 ** ee, residual=r.cuda())
    check_rows(q, scales, y, True)
    assert (q[4] == 0).all() and scales[4] == 2.0 ** -126
    if ez > -100:
        check_sum(s, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [3, 64, 1000, 4100, 40000])
@pytest.mark.parametrize("ez,ew", [(60, 90), (100, 120), (40, 124)])
def test_large_products_of_values_and_weights(c, dtype, ez, ew):
    """z w is past float32's range, the results are not: the largest is below 2^(ew + 3) sqrt(c)."""
    import torch
    t = types()[dtype]
    x = torch.ldexp(rand((9, c), 6, torch.float32), torch.tensor(ez)).to(t)
    w = torch.ldexp(rand((c,), 7, torch.float32).clamp(-3, 3), torch.tensor(min(ew, 118))).to(t)
    x[4] = 0.0
    y = norm_ref(x, w, 1e-5, None)[1]
    assert torch.finfo(torch.float32).max > y.abs().max() and (x.double() * w.double()).abs().max() > 2.0 ** 128
    q, scales = dyra.dyra_norm_quantize(x.cuda(), w.cuda(), 1e-5)
    check_rows(q, scales, y, True)
    assert (q[4] == 0).all() and scales[4] == 2.0 ** -126

"""Products of 8-bit integers whose scales are small or large: their own product may lie outside float32's normal range
where the result does not.  Weights' scales up to 2^97, as 2^30 of them (the largest sum) stay below 2^128."""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import rand
from test_gpu_ffn_shapes import on_gpu
from test_gpu_quantized import eight, gated_ref, linear_ref

pytestmark = pytest.mark.gpu

# few tokens, few features, small tiles, large tiles, K in parts
SIZES = [(5, 96, 40), (300, 1040, 9), (64, 528, 200), (4100, 272, 2050), (100, 9216, 300)]
# exponents of the tokens' and the weights' scales; the results' are theirs and the sums' (about 18)
EXPONENTS = [(-126, -10), (-126, 20), (-70, -60), (-10, -126), (30, -126), (97, -110), (-100, 97), (-120, 97)]


def close(got, ref, bound):
    """Without the allowance that the other tests make for tiny values."""
    off = (got.double().cpu() - ref).abs()
    assert (off <= bound).all(), (int((off > bound).sum()), off.numel(), float((off / bound).nan_to_num(0).max()))


def scaled(shape, seed, e):
    import torch
    q, s = eight(shape, seed)
    return q, torch.ldexp(1 + s / s.max() * 0.99, torch.tensor(e)).float().clamp(min=2.0 ** -126)


@pytest.mark.parametrize("N,c1,c2", SIZES)
@pytest.mark.parametrize("ex,ew", EXPONENTS)
def test_results_are_right_where_the_scales_product_is_not_a_normal_number(N, c1, c2, ex, ew):
    """The bounds of the other tests, and half a step of float32's subnormal numbers for the results that are one."""
    import torch
    f = torch.float32
    (x, sx), (w, sw) = scaled((N, c1), 1, ex), scaled((c2, c1), 2, min(ew, 96))
    d = [v.cuda() for v in (x, sx, w, sw)]
    y, bound = on_gpu(linear_ref, x, sx, w, sw, None, "none", None, f)
    assert y.abs().max() < 2.0 ** 127
    close(dyra.dyra_linear_quantized(*d, out_dtype=f), y, bound + 2.0 ** -148)
    y, bound = on_gpu(linear_ref, x, sx, w, sw, None, "relu", None, torch.bfloat16)
    close(dyra.dyra_linear_quantized(*d, act="relu"), y, bound + 2.0 ** -132)
    (u, _), su = eight((c2, c1), 3), torch.full((c2,), 2.0 ** -14)
    if abs(ex) <= 60:   # the pair's other product of ordinary size: its weights' scales make up for the tokens'
        y, bound = on_gpu(gated_ref, x, sx, w, sw, u, su * 2.0 ** -ex, None, None, "none", f)
        close(dyra.dyra_gated_quantized(*d, u.cuda(), (su * 2.0 ** -ex).cuda(), act="none", out_dtype=f), y, bound + 2.0 ** -130)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", SIZES)
def test_sums_of_zero_are_zero_under_any_finite_scales(N, c1, c2, out):
    """Tokens of zeros: the bias and the residual alone, though the product of the scales is past float32's range."""
    import torch
    o = torch.bfloat16 if out == "bf16" else torch.float32
    x, (w, sw) = torch.zeros(N, c1, dtype=torch.int8), scaled((c2, c1), 4, 96)
    sx = torch.full((N,), 2.0 ** 120)
    b, r = rand((c2,), 5, o), rand((N, c2), 6, o)
    d = [v.cuda() for v in (x, sx, w, sw)]
    y = dyra.dyra_linear_quantized(*d, bias=b.cuda(), act="relu", residual=r.cuda(), out_dtype=o)
    ref, bound = linear_ref(x, torch.ones(N), w, torch.ones(c2), b, "relu", r, o)
    close(y, ref, bound)
    y = dyra.dyra_gated_quantized(*d, d[2], d[3], bias_u=b.cuda(), act="none", out_dtype=o)
    assert (y == 0).all()

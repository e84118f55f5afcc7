"""Products of 8-bit integers give the same bits whatever kernel, tile or split of K a call's sizes choose, but for GELU
into bf16, which large tiles take from a table."""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import rand, types
from test_gpu_quantized import eight

pytestmark = pytest.mark.gpu

# (tokens, input features, features) of large tiles of 192 and of 256 rows, with tiles that end past the last token and feature
LARGE = [(4100, 9216, 2100), (7000, 2064, 2001), (2500, 1040, 8210)]


def parts(N, c2):
    """(rows, features) of the smaller calls: few tokens, few features, small tiles, at the start, within and at the end."""
    return [(slice(0, 16), slice(0, c2)), (slice(N - 20, N), slice(0, c2)), (slice(150, 250), slice(0, c2)), (slice(N - 300, N), slice(0, c2)),
            (slice(700, 1700), slice(0, c2)), (slice(N - 400, N), slice(c2 - 13, c2)), (slice(0, 40), slice(100, 141)), (slice(N - 900, N), slice(c2 - 700, c2))]


def compare(y, part, N, c2, what):
    import torch
    for rows, cols in parts(N, c2):
        got = part(rows, cols)
        off = got != y[rows, cols]
        assert got.dtype == y.dtype and not off.any(), (what, rows, cols, int(off.sum()), got[off][:3], y[rows, cols][off][:3])
    torch.cuda.synchronize()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", LARGE)
def test_linear_has_the_same_bits_in_every_kernel(N, c1, c2, out):
    o = types()[out]
    (x, sx), (w, sw) = ((v.cuda() for v in eight(s, 1 + i, scale)) for i, (s, scale) in enumerate((((N, c1), 1.0), ((c2, c1), c1 ** -0.5))))
    b, r = rand((c2,), 3, o).cuda(), rand((N, c2), 4, o).cuda()
    for act in ("none", "relu", "silu", "gelu_tanh") + (("gelu",) if out == "f32" else ()):
        for res in (True, False):
            call = lambda rows, cols: dyra.dyra_linear_quantized(  # noqa: E731
                x[rows], sx[rows], w[cols], sw[cols], bias=b[cols].clone(), act=act, residual=r[rows, cols] if res else None, out_dtype=o)
            compare(call(slice(0, N), slice(0, c2)), call, N, c2, f"{act} {res}")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", LARGE)
def test_gated_has_the_same_bits_in_every_kernel(N, c1, c2, out):
    o = types()[out]
    (x, sx), (g, sg), (u, su) = ((v.cuda() for v in eight(s, 5 + i, scale)) for i, (s, scale) in enumerate(
        (((N, c1), 1.0), ((c2, c1), c1 ** -0.5), ((c2, c1), c1 ** -0.5))))
    bg, bu = rand((c2,), 8, o).cuda(), rand((c2,), 9, o).cuda()
    for act in ("none", "silu", "gelu_tanh") + (("gelu",) if out == "f32" else ()):
        call = lambda rows, cols: dyra.dyra_gated_quantized(  # noqa: E731
            x[rows], sx[rows], g[cols], sg[cols], u[cols], su[cols], bias_g=bg[cols].clone(), bias_u=bu[cols].clone(), act=act, out_dtype=o)
        compare(call(slice(0, N), slice(0, c2)), call, N, c2, act)

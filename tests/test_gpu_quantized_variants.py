"""One case at least for every kernel variant of the products of 8-bit integers: test_quantized_variants holds these lists
against the rules that choose (csrc/ffn_choice.h).  Bounds as in test_gpu_quantized."""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import close, rand, types
from test_gpu_ffn_shapes import on_gpu
from test_gpu_quantized import eight, gated_ref, linear_ref

pytestmark = pytest.mark.gpu

# (tokens, input features, features): rows of K that end inside a slab, features that end inside a unit or tile
FEW_TOKENS = [(5, 2032, 8210), (16, 4096, 8210), (9, 8176, 8210), (16, 16384, 8210), (3, 24560, 8210), (20, 4080, 4120),
              (32, 8192, 4120), (31, 12272, 4120), (7, 1040, 100), (30, 4128, 100), (300, 1040, 9), (300, 2064, 30)]
TILES = {False: [(33, 1552, 35), (4144, 1552, 65), (193, 1552, 4174), (385, 1552, 4729), (2974, 1552, 1288), (5431, 1552, 1288),
                 (5431, 1552, 2065), (4729, 1552, 2842)],
         True: [(33, 1552, 35), (33, 1552, 4174), (65, 1552, 4174), (193, 1552, 4174), (385, 1552, 4729), (3208, 1552, 1177),
                (1219, 1552, 4618), (1804, 1552, 3619)]}


def shapes(gated):
    return FEW_TOKENS + TILES[gated]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", shapes(False))
def test_linear_variants(N, c1, c2, out):
    o = types()[out]
    (x, sx), (w, sw) = eight((N, c1), 1), eight((c2, c1), 2, c1 ** -0.5)
    b, r = rand((c2,), 3, o), rand((N, c2), 4, o)
    d = [v.cuda() for v in (x, sx, w, sw)]
    close(dyra.dyra_linear_quantized(*d, out_dtype=o), *on_gpu(linear_ref, x, sx, w, sw, None, "none", None, o))
    close(dyra.dyra_linear_quantized(*d, bias=b.cuda(), act="gelu_tanh", residual=r.cuda(), out_dtype=o),
          *on_gpu(linear_ref, x, sx, w, sw, b, "gelu_tanh", r, o), "epilogue")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", shapes(True))
def test_gated_variants(N, c1, c2, out):
    o = types()[out]
    (x, sx), (g, sg), (u, su) = eight((N, c1), 5), eight((c2, c1), 6, c1 ** -0.5), eight((c2, c1), 7, c1 ** -0.5)
    bg, bu = rand((c2,), 8, o), rand((c2,), 9, o)
    h = dyra.dyra_gated_quantized(*(v.cuda() for v in (x, sx, g, sg, u, su, bg, bu)), out_dtype=o)
    close(h, *on_gpu(gated_ref, x, sx, g, sg, u, su, bg, bu, "silu", o))

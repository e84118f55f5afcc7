"""One case at least for every kernel variant of the feed-forward calls, in every type: test_ffn_variants holds these
lists against the rules that choose (csrc/ffn_choice.h).

Rows of K end inside a slab and are long enough for every stage or ring place to be used again; features end inside a unit
or tile.  Bounds as in test_gpu_ffn and test_gpu_ffn_accuracy.
"""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import close, experts, gated_ref, linear_ref, rand, types
from test_gpu_ffn_accuracy import moe_ref_once
from test_gpu_ffn_shapes import moe_ref_grouped, on_gpu

pytestmark = pytest.mark.gpu

# (tokens, bytes of a row of X, features)
FEW_TOKENS = [(5, 2032, 8210), (16, 4096, 8210), (9, 8176, 8210), (16, 16384, 8210), (3, 24560, 8210), (20, 4080, 4120),
              (32, 8192, 4120), (31, 12272, 4120), (7, 1040, 100), (30, 4128, 100), (300, 1040, 9), (300, 2064, 30)]
# (tokens, input features, features)
TILES = {("bf16", False): [(33, 776, 35), (4144, 776, 65), (193, 776, 4174), (385, 776, 4729), (2974, 776, 1288), (5431, 776, 1288),
                           (5431, 776, 2065), (4729, 776, 2842)],
         ("bf16", True): [(33, 776, 35), (33, 776, 4174), (65, 776, 4174), (193, 776, 4174), (385, 776, 4729), (3208, 776, 1177),
                          (1219, 776, 4618), (1804, 776, 3619)],
         ("f32", False): [(33, 396, 35), (4144, 396, 65), (5548, 396, 155), (3559, 396, 844)],
         ("f32", True): [(33, 396, 35), (33, 396, 4174), (5548, 396, 65), (257, 396, 4951)]}
# tokens, experts, places, c, f
EXPERTS = [(5, 6, 2, 264, 520), (4, 20, 3, 8, 1048), (9, 20, 2, 8, 1048), (40, 3, 2, 520, 1304), (9, 5, 4, 8, 3000), (20, 3, 2, 72, 3000),
           (8, 4, 2, 2056, 1048), (40, 3, 2, 2056, 1304), (300, 4, 2, 2064, 264), (3, 5, 2, 1032, 520), (2, 3, 2, 2048, 264),
           (2, 3, 1, 1536, 264), (2, 3, 2, 3080, 264), (2, 3, 2, 4200, 264), (2, 3, 2, 6408, 264)]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def shapes(dtype, gated):
    """Every (tokens, input features, features) that the linear layer or the gated pair is tested at here."""
    return [(N, b // (2 if dtype == "bf16" else 4), c2) for N, b, c2 in FEW_TOKENS] + TILES[dtype, gated]


def workspaces(dtype, T, k, f):
    """Bytes of workspace, room for split sums, inner activations in two parts."""
    least = T * k * f * (2 if dtype == "bf16" else 4)
    return [(least, 0, 0), (least + 8192 * T, 1, 0)] + ([(2 * least + 8192 * T, 1, 1)] if dtype == "bf16" else [])


LINEAR = [(d, o, *s) for d, o in TYPES for s in shapes(d, False)]
GATED = [(d, *s) for d in ("bf16", "f32") for s in shapes(d, True)]


@pytest.mark.parametrize("dtype,out,N,c1,c2", LINEAR)
def test_linear_variants(dtype, out, N, c1, c2):
    t, o = types()[dtype], types()[out]
    x, w, b, r = rand((N, c1), 1, t), rand((c2, c1), 2, t, c1 ** -0.5), rand((c2,), 3, t), rand((N, c2), 4, o)
    d = [v.cuda() for v in (x, w, b, r)]
    close(dyra.dyra_linear(d[0], d[1], out_dtype=o), *on_gpu(linear_ref, x, w, None, "none", None, o))
    close(dyra.dyra_linear(d[0], d[1], bias=d[2], act="gelu_tanh", residual=d[3], out_dtype=o),
          *on_gpu(linear_ref, x, w, b, "gelu_tanh", r, o), "epilogue")


@pytest.mark.parametrize("dtype,N,c1,c2", GATED)
def test_gated_variants(dtype, N, c1, c2):
    t = types()[dtype]
    x, wg, wu = rand((N, c1), 5, t), rand((c2, c1), 6, t, c1 ** -0.5), rand((c2, c1), 7, t, c1 ** -0.5)
    bg, bu = rand((c2,), 8, t), rand((c2,), 9, t)
    d = [v.cuda() for v in (x, wg, wu, bg, bu)]
    close(dyra.dyra_gated(*d), *on_gpu(gated_ref, x, wg, wu, bg, bu, "silu", t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,c,f", EXPERTS)
def test_expert_variants(T, E, k, c, f, dtype):
    import torch
    t = types()[dtype]
    x, r, w3 = rand((T, c), 11, t), rand((T, c), 12, t), experts(E, c, f, 13, t)
    g = torch.Generator().manual_seed(16)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    ids[0] = torch.arange(k) % E
    w = torch.rand(T, k, generator=g)
    dev, args = [v.cuda() for v in (x, *w3, ids, w)], (x, *w3, ids, w, "silu", r)
    for n, parts, rest in workspaces(dtype, T, k, f):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        y = dyra.dyra_moe(*dev, residual=r.cuda(), workspace=ws)
        close(y, *on_gpu(moe_ref_once if rest else moe_ref_grouped, *args), f"parts {parts} rest {rest}")

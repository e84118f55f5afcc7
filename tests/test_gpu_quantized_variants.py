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

# K in parts: (tokens, input features, features); the last part shorter, tiles that end past the last row and feature
SPLIT = {False: [(34, 5264, 34), (211, 6128, 406), (33, 16400, 77), (33, 7376, 3322), (1463, 9216, 65), (3292, 11360, 65), (68, 11472, 3291),
                 (2352, 16416, 132), (857, 36512, 1161), (413, 65536, 265)],
         True: [(35, 5680, 33), (33, 25616, 358), (1372, 8976, 34), (781, 17056, 207), (70, 7376, 3091), (986, 12864, 517), (2781, 13040, 65),
                (1381, 10336, 1293)]}


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


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", SPLIT[False])
def test_linear_in_parts(N, c1, c2, out):
    """The same bits as without a workspace, and with one that holds other values; rows and outputs strided."""
    import torch
    o = types()[out]
    (x, sx), (w, sw) = eight((N, c1), 11), eight((c2, c1), 12, c1 ** -0.5)
    b, r = rand((c2,), 13, o), rand((N, c2), 14, o)
    d = [v.cuda() for v in (x, sx, w, sw)]
    size = dyra.dyra_quantized_workspace_bytes(N, c1, c2)
    assert size > 0
    ws = torch.full((size,), 90, dtype=torch.uint8, device="cuda")
    y = dyra.dyra_linear_quantized(*d, bias=b.cuda(), act="silu", residual=r.cuda(), out_dtype=o, workspace=ws)
    close(y, *on_gpu(linear_ref, x, sx, w, sw, b, "silu", r, o))
    less = dyra.dyra_linear_quantized(*d, bias=b.cuda(), act="silu", residual=r.cuda(), out_dtype=o, workspace=ws[:size - 16])
    assert torch.equal(y, less)
    wide = [torch.zeros(v.shape[0], c1 + 48, dtype=torch.int8, device="cuda") for v in (x, w)]
    for v, q in zip(wide, (x, w)):
        v[:, 32:32 + c1] = q.cuda()
    base = torch.full((N + 2, c2 + 5), 7.0, dtype=o, device="cuda")
    dyra.dyra_linear_quantized(wide[0][:, 32:32 + c1], d[1], wide[1][:, 32:32 + c1], d[3], bias=b.cuda(), act="silu", residual=r.cuda(),
                               out_dtype=o, Y=base[1:N + 1, 3:3 + c2])
    assert torch.equal(base[1:N + 1, 3:3 + c2], y)
    base[1:N + 1, 3:3 + c2] = 7.0
    assert (base == 7).all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", SPLIT[True])
def test_gated_in_parts(N, c1, c2, out):
    import torch
    o = types()[out]
    (x, sx), (g, sg), (u, su) = eight((N, c1), 15), eight((c2, c1), 16, c1 ** -0.5), eight((c2, c1), 17, c1 ** -0.5)
    bg, bu = rand((c2,), 18, o), rand((c2,), 19, o)
    d = [v.cuda() for v in (x, sx, g, sg, u, su, bg, bu)]
    size = dyra.dyra_quantized_workspace_bytes(N, c1, c2, True)
    assert size > 0
    h = dyra.dyra_gated_quantized(*d, out_dtype=o)
    close(h, *on_gpu(gated_ref, x, sx, g, sg, u, su, bg, bu, "silu", o))
    ws = torch.full((size + 32,), 90, dtype=torch.uint8, device="cuda")
    assert torch.equal(h, dyra.dyra_gated_quantized(*d, out_dtype=o, workspace=ws)) and (ws[size:] == 90).all()
    assert torch.equal(h, dyra.dyra_gated_quantized(*d, out_dtype=o, workspace=ws[:16]))


def test_parts_captured_and_on_two_streams():
    """Two graphs replayed in turn with eager work between; then two streams at once."""
    import torch
    (w, sw), (u, su) = ([v.cuda() for v in eight((300, 9216), s, 0.01)] for s in (21, 22))

    def both(x, sx, stream=None):
        return (dyra.dyra_linear_quantized(x, sx, w, sw, stream=stream), dyra.dyra_gated_quantized(x, sx, w, sw, u, su, stream=stream))

    assert dyra.dyra_quantized_workspace_bytes(200, 9216, 300) > 0 and dyra.dyra_quantized_workspace_bytes(200, 9216, 300, True) > 0
    static = [[v.cuda() for v in eight((200, 9216), 23 + i)] for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in static:
            both(*x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both(*x))
        graphs.append(g)
    for i in range(4):
        for k in range(2):
            for v, n in zip(static[k], eight((200, 9216), 30 + 2 * i + k)):
                v.copy_(n)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = [both(*x) for x in static]
        assert all(torch.equal(a, b) for o, e in zip(outs, eager) for a, b in zip(o, e)), f"replay {i}"
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [(both(*static[k], streams[k]), eager[k]) for _ in range(3) for k in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, e in got for a, b in zip(g, e))

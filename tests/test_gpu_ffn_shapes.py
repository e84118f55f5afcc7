"""The feed-forward operators over every tile shape and kernel variant, and at offsets past 32 bits.

Bounds as in test_gpu_ffn; references in float64 on the GPU.
"""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import close, experts, gated_ref, linear_ref, moe_ref, rand, route_ref, types, U

pytestmark = pytest.mark.gpu


def on_gpu(ref, *args):
    y, d = ref(*(a.cuda() if hasattr(a, "cuda") else a for a in args))
    return y.cpu(), d.cpu()


# rows and features that end inside a tile; the last slab of K partial; from one tile to several rounds of them
TILED = [(41, 520, 33), (1000, 264, 70), (4257, 312, 70), (4374, 280, 201), (4326, 272, 398), (1026, 264, 3632),
         (3225, 264, 2355), (3751, 264, 3073), (4781, 264, 2844), (4800, 1032, 1280), (33, 2056, 4100)]


@pytest.mark.parametrize("N,c1,c2", TILED)
def test_linear_tiles(N, c1, c2):
    import torch
    t = torch.bfloat16
    x, w, b = rand((N, c1), 1, t), rand((c2, c1), 2, t, c1 ** -0.5), rand((c2,), 3, t)
    r, r32 = rand((N, c2), 4, t), rand((N, c2), 5, torch.float32)
    xd, wd, bd, rd = (v.cuda() for v in (x, w, b, r))
    for act, bias, res in (("none", False, True), ("gelu", True, False), ("relu", True, True), ("silu", False, False),
                           ("gelu_tanh", False, True)):
        y = dyra.dyra_linear(xd, wd, bias=bd if bias else None, act=act, residual=rd if res else None)
        close(y, *on_gpu(linear_ref, x, w, b if bias else None, act, r if res else None, t), f"{act} {bias} {res}")
    y = dyra.dyra_linear(xd, wd, bias=bd, act="silu", residual=r32.cuda(), out_dtype=torch.float32)
    close(y, *on_gpu(linear_ref, x, w, b, "silu", r32, torch.float32), "float32 result")


@pytest.mark.parametrize("N,c1,c2", [(41, 272, 65), (4106, 280, 35), (129, 296, 2874), (4269, 280, 197), (670, 264, 2694),
                                     (4630, 280, 785), (2315, 264, 2447), (2935, 264, 2326), (2400, 1032, 1280)])
def test_gated_tiles(N, c1, c2):
    import torch
    t = torch.bfloat16
    x, wg, wu = rand((N, c1), 6, t), rand((c2, c1), 7, t, c1 ** -0.5), rand((c2, c1), 8, t, c1 ** -0.5)
    bg, bu = rand((c2,), 9, t), rand((c2,), 10, t)
    d = [v.cuda() for v in (x, wg, wu, bg, bu)]
    for act, i, j in (("silu", None, None), ("gelu", 3, 4), ("relu", 3, None), ("gelu_tanh", None, 4), ("none", None, None)):
        h = dyra.dyra_gated(*d[:3], bias_g=None if i is None else d[i], bias_u=None if j is None else d[j], act=act)
        close(h, *on_gpu(gated_ref, x, wg, wu, None if i is None else bg, None if j is None else bu, act, t), act)


@pytest.mark.parametrize("N,c1,c2", [(40, 276, 71), (2840, 268, 130), (2926, 260, 325), (1095, 260, 2693), (98, 260, 2082)])
def test_float32_tiles(N, c1, c2):
    import torch
    t = torch.float32
    x, w, w2, b, r = rand((N, c1), 11, t), rand((c2, c1), 12, t, c1 ** -0.5), rand((c2, c1), 13, t, c1 ** -0.5), rand((c2,), 14, t), rand((N, c2), 15, t)
    d = [v.cuda() for v in (x, w, w2, b, r)]
    close(dyra.dyra_linear(d[0], d[1], bias=d[3], act="gelu", residual=d[4]), *on_gpu(linear_ref, x, w, b, "gelu", r, t))
    close(dyra.dyra_gated(d[0], d[1], d[2], bias_g=d[3]), *on_gpu(gated_ref, x, w, w2, b, None, "silu", t))


# tokens around the groups of 16; K of every number of slabs a wavefront holds in registers, and past it
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 15, 16, 17, 32])
@pytest.mark.parametrize("row_bytes", [1024, 1040, 4096, 6160, 8192, 12304, 16400, 24576, 24592, 34816])
def test_few_tokens(N, row_bytes, dtype):
    t = types()[dtype]
    c1, c2 = row_bytes // (2 if dtype == "bf16" else 4), 77
    x, w, w2 = rand((N, c1), 21, t), rand((c2, c1), 22, t, c1 ** -0.5), rand((c2, c1), 23, t, c1 ** -0.5)
    b, r = rand((c2,), 24, t), rand((N, c2), 25, t)
    d = [v.cuda() for v in (x, w, w2, b, r)]
    close(dyra.dyra_linear(d[0], d[1], bias=d[3], act="silu", residual=d[4]), *on_gpu(linear_ref, x, w, b, "silu", r, t))
    close(dyra.dyra_gated(d[0], d[1], d[2], bias_u=d[3]), *on_gpu(gated_ref, x, w, w2, None, b, "silu", t))


# more units than workgroups, several a workgroup, an odd number
@pytest.mark.parametrize("N,c1,c2", [(1, 136, 9000), (3, 520, 20003), (20, 264, 12345), (32, 16392, 8200), (2, 13000, 8211)])
def test_few_tokens_many_features(N, c1, c2):
    import torch
    t = torch.bfloat16
    x, w, r = rand((N, c1), 26, t), rand((c2, c1), 27, t, c1 ** -0.5), rand((N, c2), 28, t)
    close(dyra.dyra_linear(x.cuda(), w.cuda(), residual=r.cuda(), act="gelu"), *on_gpu(linear_ref, x, w, None, "gelu", r, t))
    close(dyra.dyra_gated(x.cuda(), w.cuda(), w.flip(0).cuda()), *on_gpu(gated_ref, x, w, w.flip(0), None, None, "silu", t))


# long rows of x (past a wavefront's registers); 16 rows of Wd a workgroup and 8; slots of 8 pairs and of 16; more pairs
# than one chunk of them
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,c,f", [(2, 3, 2, 6408, 24), (1, 2, 2, 12808, 16), (9, 2, 2, 4104, 40), (9, 8, 2, 4200, 200),
                                       (2, 4, 2, 4100, 1304), (33, 3, 2, 72, 520), (64, 4, 4, 64, 1032), (300, 2, 1, 4112, 16),
                                       (1024, 5, 1, 40, 24), (512, 6, 2, 24, 72), (256, 1024, 4, 16, 8)])
def test_moe_variants(T, E, k, c, f, dtype):
    import torch
    t = types()[dtype]
    if dtype == "bf16":
        c, f = (c + 7) // 8 * 8, (f + 7) // 8 * 8
    x, r, w3 = rand((T, c), 31, t), rand((T, c), 32, t), experts(E, c, f, 33, t)
    g = torch.Generator().manual_seed(36)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand(T, k, generator=g)
    y = dyra.dyra_moe(*(v.cuda() for v in (x, *w3, ids, w)), residual=r.cuda())
    close(y, *on_gpu(moe_ref_grouped, x, *w3, ids, w, "silu", r))


def moe_ref_grouped(x, wg, wu, wd, ids, w, act, r):
    """moe_ref with the pairs of an expert together."""
    import torch
    t, f = x.dtype, wg.shape[1]
    y = r.double().clone()
    terms, d = y.abs().clone(), torch.zeros_like(y)
    for e in range(wg.shape[0]):
        at = (ids == e).nonzero()
        if not len(at):
            continue
        i, p = at[:, 0], w[at[:, 0], at[:, 1]].double()[:, None]
        h, dh = gated_ref(x[i], wg[e], wu[e], None, None, act, t)
        wde = wd[e].double()
        o, s, m = h @ wde.T, h.abs() @ wde.abs().T, dh @ wde.abs().T
        y.index_add_(0, i, p * o)
        terms.index_add_(0, i, p.abs() * o.abs())
        d.index_add_(0, i, p.abs() * (m + 2 * (f + 4) * U * (s + m)))
    d += 2 * (ids.shape[1] + 4) * U * (terms + d)
    return y, d + torch.finfo(t).eps / 2 * (y.abs() + d)


def far(rows, cols, stride, dtype, seed, scale=1.0):
    """A matrix whose rows lie `stride` elements apart; only its own elements are set."""
    import torch
    base = torch.empty((rows - 1) * stride + cols, dtype=dtype, device="cuda")
    m = base.as_strided((rows, cols), (stride, 1))
    m.copy_(rand((rows, cols), seed, dtype, scale))
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 30, 2500])
def test_offsets_past_32_bits(N, dtype):
    """Rows 2^20 elements apart, the last 4 GiB and more behind the first: of X (where N is large), W, residual and Y."""
    import torch
    t, ld = types()[dtype], 1 << 20
    c1, c2 = 136, 2120 if N < 100 else 40
    x = far(N, c1, ld if N > 100 else 136, t, 41)
    w = far(c2, c1, ld if N < 100 else 136, t, 42, c1 ** -0.5)
    step = (1 << 32) // 2 // (N - 1) // 8 * 8 + 16    # bf16: 2^32 bytes from the first row to the last
    r = far(N, c2, step, t, 43)
    base = torch.empty((N - 1) * step + c2, dtype=t, device="cuda")
    y = base.as_strided((N, c2), (step, 1))
    dyra.dyra_linear(x, w, residual=r, act="relu", Y=y)
    close(y, *on_gpu(linear_ref, x, w, None, "relu", r, t))
    dyra.dyra_gated(x, w, w, H=y)
    close(y, *on_gpu(gated_ref, x, w, w, None, None, "silu", t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_result_of_whole_tiles(dtype):
    """Y of 2^31 elements and more, its last tiles against the definition on their rows."""
    import torch
    t = types()[dtype]
    N, c1, c2 = 524544, 8, 4104
    x, w = rand((N, c1), 44, t), rand((c2, c1), 45, t, c1 ** -0.5)
    y = dyra.dyra_linear(x.cuda(), w.cuda(), act="silu")
    for s in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
        close(y[s], *linear_ref(x[s], w, None, "silu", None, t), str(s))


def test_router_offsets_past_32_bits():
    import torch
    T, E, ld = 1500, 64, 1 << 20
    logits = far(T, E, ld, torch.float32, 46)
    ids, w = dyra.dyra_route(logits, 4)
    rid, rw = route_ref(logits.cpu(), 4, "softmax", True, 1.0)
    assert (ids.cpu() == rid).all()
    close(w, rw, 400 * U * rw)


@pytest.mark.parametrize("T", [1, 40])
def test_experts_past_32_bits(T):
    """260 experts of 2^24 elements a matrix: 2^33 bytes and more behind the first."""
    import torch
    E, f, c, t = 260, 4096, 4096, torch.bfloat16
    used = [0, 127, 131, 258, 259]
    dev, host = [], []
    for i, shape in enumerate([(f, c), (f, c), (c, f)]):
        m = torch.empty(E, *shape, dtype=t, device="cuda")
        for e in used:
            m[e] = rand(shape, 50 + 10 * e + i, t, 4096 ** -0.5).cuda()
        dev.append(m)
        host.append(m[used].cpu())
    x, r = rand((T, c), 47, t), rand((T, c), 48, t)
    g = torch.Generator().manual_seed(49)
    at = torch.randint(0, len(used), (T, 4), generator=g, dtype=torch.int32)
    w = torch.rand(T, 4, generator=g)
    ids = torch.tensor(used, dtype=torch.int32)[at.long()]
    y = dyra.dyra_moe(x.cuda(), *dev, ids.cuda(), w.cuda(), residual=r.cuda())
    close(y, *on_gpu(moe_ref_grouped, x, *host, at, w, "silu", r))


def test_new_outputs_for_another_stream_are_not_memory_that_is_still_written():
    """A block freed on the current stream while a write to it is pending is not handed to a call on another stream."""
    import torch
    x, w = rand((64, 256), 61, torch.bfloat16).cuda(), rand((8192, 256), 62, torch.bfloat16).cuda()
    ref = dyra.dyra_linear(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        tmp = torch.empty(64, 8192, dtype=torch.bfloat16, device="cuda")
        torch.cuda._sleep(2_000_000)
        tmp.fill_(7.0)
        del tmp
        y = dyra.dyra_linear(x, w, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(y, ref)


def test_expert_layer_over_its_input():
    import torch
    T, E, k, c, f = 24, 4, 2, 128, 64
    x, w3 = rand((T, c), 63, torch.bfloat16), experts(E, c, f, 64, torch.bfloat16)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(67), dtype=torch.int32)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(68))
    y = x.cuda()
    dyra.dyra_moe(y, *(v.cuda() for v in (*w3, ids, w)), residual=y, Y=y)
    close(y, *moe_ref(x, *w3, ids, w, "silu", x))


# narrow layers: the second product shared among workgroups, runs that begin and end inside slots, experts without pairs
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,c,f", [(57, 9, 4, 360, 5432), (1, 3, 2, 8, 70000), (5, 40, 4, 72, 3000), (15, 20, 1, 456, 2056),
                                       (300, 6, 3, 16, 1032), (2, 6, 2, 1000, 9008), (64, 8, 8, 264, 1304)])
def test_moe_narrow(T, E, k, c, f, dtype):
    import torch
    t = types()[dtype]
    x, r, w3 = rand((T, c), 71, t), rand((T, c), 72, t), experts(E, c, f, 73, t)
    g = torch.Generator().manual_seed(76)
    ids = torch.randint(0, E + 1, (T, k), generator=g, dtype=torch.int32)
    ids[:, 0][ids[:, 0] == 2] = -1
    w = torch.rand(T, k, generator=g)
    dev = [v.cuda() for v in (x, *w3, ids, w)]
    ref = on_gpu(moe_ref_grouped, x, *w3, ids, w, "gelu", r)
    y = dyra.dyra_moe(*dev, act="gelu", residual=r.cuda())
    close(y, *ref)
    assert torch.equal(y, dyra.dyra_moe(*dev, act="gelu", residual=r.cuda()))
    small = torch.empty(dyra.dyra_moe_workspace_bytes(T, k, f, t), dtype=torch.uint8, device="cuda")   # not shared
    close(dyra.dyra_moe(*dev, act="gelu", residual=r.cuda(), workspace=small), *ref)
    wide = torch.full((T + 1, c + 3), 7.0, dtype=t, device="cuda")
    dyra.dyra_moe(*dev, act="gelu", residual=r.cuda(), Y=wide[:T, 1:1 + c])
    assert torch.equal(wide[:T, 1:1 + c], y) and (wide[T] == 7).all() and (wide[:, 0] == 7).all() and (wide[:, 1 + c:] == 7).all()


# few features of many tokens: one and two blocks of features, K that fits the registers and past it, ends inside a unit
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,c1,c2", [(33, 8, 1), (40, 520, 16), (1000, 2056, 17), (4097, 264, 32), (70, 4104, 5), (257, 6200, 31),
                                     (50, 12296, 16), (65, 16392, 9), (9000, 72, 6), (100, 1024, 33)])
def test_few_features(N, c1, c2, dtype, out):
    import torch
    t, o = types()[dtype], types()[out]
    x, w, w2 = rand((N, c1 + 16), 81, t), rand((c2, c1 + 8), 82, t, c1 ** -0.5), rand((c2, c1), 83, t, c1 ** -0.5)
    b, r = rand((c2,), 84, t), rand((N, c2), 85, o)
    xd, wd, w2d, bd, rd = (v.cuda() for v in (x, w, w2, b, r))
    x, w, xs, ws = x[:, 8:8 + c1], w[:, 8:8 + c1], xd[:, 8:8 + c1], wd[:, 8:8 + c1]
    close(dyra.dyra_linear(xs, ws, out_dtype=o), *on_gpu(linear_ref, x, w, None, "none", None, o))
    wide = torch.full((N + 1, c2 + 3), 7.0, dtype=o, device="cuda")
    dyra.dyra_linear(xs, ws, bias=bd, act="gelu", residual=rd, out_dtype=o, Y=wide[:N, 1:1 + c2])
    close(wide[:N, 1:1 + c2], *on_gpu(linear_ref, x, w, b, "gelu", r, o))
    assert (wide[N] == 7).all() and (wide[:, 0] == 7).all() and (wide[:, 1 + c2:] == 7).all()
    if dtype == out:
        w, ws = w.contiguous(), ws.contiguous()
        close(dyra.dyra_gated(xs, ws, w2d, bias_g=bd), *on_gpu(gated_ref, x, w, w2, b, None, "silu", t))
        close(dyra.dyra_gated(xs, w2d, ws, bias_u=bd, act="relu"), *on_gpu(gated_ref, x, w2, w, None, b, "relu", t))


def test_few_features_infinities_and_nan_stay_in_their_rows():
    import torch
    x, w = rand((400, 72), 86, torch.bfloat16), rand((20, 72), 87, torch.bfloat16)
    clean = dyra.dyra_linear(x.cuda(), w.cuda(), act="silu")
    x[1, 5], x[399, 71] = float("inf"), float("nan")
    y = dyra.dyra_linear(x.cuda(), w.cuda(), act="silu")
    rows = [i for i in range(400) if i not in (1, 399)]
    assert torch.equal(y[rows], clean[rows]) and y[399].isnan().all() and not y[1].isfinite().all()


# several units a workgroup: tokens in registers, K of every number of slabs they hold, and past it
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,row_bytes,c2", [(5, 1040, 8200), (16, 4112, 8211), (16, 8192, 8200), (7, 16400, 8200), (16, 24576, 8200),
                                            (16, 24592, 8200), (17, 4096, 4200), (32, 8208, 4200), (31, 12288, 4201), (32, 12304, 4200)])
def test_few_tokens_several_units(N, row_bytes, c2, dtype):
    t = types()[dtype]
    c1 = row_bytes // (2 if dtype == "bf16" else 4)
    x, w, b, r = rand((N, c1), 91, t), rand((c2, c1), 92, t, c1 ** -0.5), rand((c2,), 93, t), rand((N, c2), 94, t)
    d = [v.cuda() for v in (x, w, b, r)]
    close(dyra.dyra_linear(d[0], d[1], bias=d[2], act="gelu", residual=d[3]), *on_gpu(linear_ref, x, w, b, "gelu", r, t))
    w2 = w.flip(0)
    close(dyra.dyra_gated(d[0], d[1], w2.cuda(), bias_g=d[2]), *on_gpu(gated_ref, x, w, w2, b, None, "silu", t))


def test_narrow_layers_captured_and_on_two_streams():
    """A small router and a narrow expert layer (f shared among workgroups): two graphs replayed in turn, then two streams."""
    import torch
    T, E, k, c, f = 40, 12, 2, 264, 6000
    p = [v.cuda() for v in (rand((E, c), 95, torch.bfloat16, c ** -0.5), *experts(E, c, f, 96, torch.bfloat16))]

    def layer(x, stream=None):
        logits = dyra.dyra_linear(x, p[0], out_dtype=torch.float32, stream=stream)
        ids, w = dyra.dyra_route(logits, k, stream=stream)
        return logits, ids, w, dyra.dyra_moe(x, *p[1:], ids, w, residual=x, stream=stream)

    static = [rand((T, c), 101 + i, torch.bfloat16).cuda() for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in static:
            layer(x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(x))
        graphs.append(g)
    for i in range(4):
        for q in range(2):
            static[q].copy_(rand((T, c), 110 + 2 * i + q, torch.bfloat16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = [layer(x) for x in static]
        assert all(torch.equal(u, v) for o, e in zip(outs, eager) for u, v in zip(o, e)), f"replay {i}"
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [(layer(static[q], streams[q]), eager[q]) for _ in range(3) for q in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for g, r in got for u, v in zip(g, r))

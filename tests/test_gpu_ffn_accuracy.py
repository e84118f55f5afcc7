"""How near the feed-forward operators come to their definitions where a looser bound would hide it.

Bounds as in test_gpu_ffn, but for what each test says.
"""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import close, experts, gated_ref, half, rand, types, U
from test_gpu_ffn_shapes import moe_ref_grouped, on_gpu

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ inner activations of the expert layer

def moe_ref_once(x, wg, wu, wd, ids, w, act, r):
    """The expert layer with its output rounded once: inner activations in two bfloat16 parts.  The first leaves out at
    most half a step (2^-8 of them), the second half a step of that: 2^-16."""
    import torch
    t, f = x.dtype, wg.shape[1]
    y = r.double().clone()
    terms, d = y.abs().clone(), torch.zeros_like(y)
    for e in range(wg.shape[0]):
        at = (ids == e).nonzero()
        if not len(at):
            continue
        i, p = at[:, 0], w[at[:, 0], at[:, 1]].double()[:, None]
        h, dh = gated_ref(x[i], wg[e], wu[e], None, None, act, torch.float32)
        dh = dh + 2.0 ** -16 * (h.abs() + dh)
        wde = wd[e].double()
        o, s, m = h @ wde.T, h.abs() @ wde.abs().T, dh @ wde.abs().T
        y.index_add_(0, i, p * o)
        terms.index_add_(0, i, p.abs() * o.abs())
        # twice the terms: both parts are summed
        d.index_add_(0, i, p.abs() * (m + 2 * (2 * f + 4) * U * (s + m)))
    d += 2 * (ids.shape[1] + 4) * U * (terms + d)
    return y, d + half(t) * (y.abs() + d)


# 8 and 16 rows of Wd a workgroup, slots of 8 and of 16 pairs; more pairs than a chunk; f shared among workgroups
@pytest.mark.parametrize("T,E,k,c,f", [(1, 8, 3, 64, 40), (5, 8, 2, 256, 1000), (40, 4, 3, 72, 1032), (6, 4, 2, 2056, 520),
                                       (40, 3, 2, 2056, 1048), (150, 4, 2, 2064, 520), (57, 9, 4, 360, 5432), (200, 3, 5, 24, 72)])
def test_expert_layer_rounds_its_output_once(T, E, k, c, f):
    import torch
    t = torch.bfloat16
    x, r, w3 = rand((T, c), 1, t), rand((T, c), 2, t), experts(E, c, f, 3, t)
    g = torch.Generator().manual_seed(6)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand(T, k, generator=g)
    dev, args = [v.cuda() for v in (x, *w3, ids, w)], (x, *w3, ids, w, "silu", r)
    y = dyra.dyra_moe(*dev, residual=r.cuda())
    close(y, *on_gpu(moe_ref_once, *args))
    # workspaces without room for the second parts: the inner activations are rounded once more
    least = dyra.dyra_moe_workspace_bytes(T, k, f, t)
    for n in (least, least + 8192 * T, 2 * least + 8192 * T - 1):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        close(dyra.dyra_moe(*dev, residual=r.cuda(), workspace=ws), *on_gpu(moe_ref_grouped, *args), f"{n} bytes")
    ws = torch.empty(2 * least + 8192 * T, dtype=torch.uint8, device="cuda")
    assert torch.equal(y, dyra.dyra_moe(*dev, residual=r.cuda(), workspace=ws))


@pytest.mark.parametrize("T", [4, 30])
def test_infinite_inner_activations_stay_in_their_tokens(T):
    """An inner activation past bfloat16's range has no rest: its token's row is not finite, no other row changes."""
    import torch
    t, E, k, c, f = torch.bfloat16, 2, 1, 64, 48
    x, w3 = rand((T, c), 7, t), experts(E, c, f, 8, t)
    ids, w = torch.zeros(T, k, dtype=torch.int32), torch.ones(T, k)
    dev = [v.cuda() for v in w3]
    clean = dyra.dyra_moe(x.cuda(), *dev, ids.cuda(), w.cuda(), act="none")
    x[2] *= 1e30                    # gate and up about 1e30 each: their product overflows float32
    y = dyra.dyra_moe(x.cuda(), *dev, ids.cuda(), w.cuda(), act="none")
    rows = [i for i in range(T) if i != 2]
    assert torch.equal(y[rows], clean[rows]) and not y[2].isfinite().any()
    x[2] = 0
    w3[0][0, 5], w3[1][0, 5] = 0, 0  # one feature of 2e38 (1e19 * 2e19), the others 0: finite, and so is the result
    x[2, 0] = 1.0
    w3[0][0, :, 0], w3[1][0, :, 0] = 0, 0
    w3[0][0, 5, 0], w3[1][0, 5, 0] = 1e19, 2e19
    y = dyra.dyra_moe(x.cuda(), *(v.cuda() for v in w3), ids.cuda(), w.cuda(), act="none")
    assert y[2].isfinite().all()


# ------------------------------------------------------------------ gelu where it is small

def gelu_bound(v, out):
    """gelu(v) and the bound of a result: half a step of the type, and of the activation's own evaluation, for bfloat16
    results 2^-12 of it, also no more than 16 u |v|; for float32 erfc's: its argument is right to 2 u, which is
    2 (v^2 + 1) u of the result, itself and the products 20 u."""
    import math

    import torch
    v = v.double()
    y = 0.5 * v * torch.erfc(-v / math.sqrt(2))
    own = torch.minimum(2.0 ** -12 * y.abs(), 16 * U * v.abs()) if out == torch.bfloat16 else (2 * (v * v + 1) + 20) * U * y.abs()
    return y, own + half(out) * (y.abs() + own)


# the kernels for few tokens (in registers and through the ring), few features, tiles, and the largest tiles
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,c2", [(7, 48), (16, 8200), (300, 8), (300, 70), (4000, 2050)])
def test_gelu_is_right_where_it_is_small(N, c2, dtype, out):
    """Values from -12.75 on come through the product unchanged; gelu(-5) is -1.4e-6, gelu(-12.75) -2e-36."""
    import torch
    t, o = types()[dtype], types()[out]
    v = torch.linspace(-12.75, 6, N).to(t)
    v[:4] = torch.tensor([-3.5, -4.5, -5.0, -5.5])
    x, w, zero = torch.zeros(N, 8, dtype=t), torch.zeros(c2, 8, dtype=t), torch.zeros(c2, 8, dtype=t)
    x[:, 2], w[:, 2] = v, 1
    y, bound = gelu_bound(v, o)
    y, bound = y[:, None].expand(N, c2), bound[:, None].expand(N, c2)
    close(dyra.dyra_linear(x.cuda(), w.cuda(), act="gelu", out_dtype=o), y, bound)
    if dtype == out:
        one = torch.ones(c2, dtype=t, device="cuda")
        close(dyra.dyra_gated(x.cuda(), w.cuda(), zero.cuda(), bias_u=one, act="gelu"), y, bound, "gated")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gelu_of_experts_is_right_where_it_is_small(dtype):
    """One inner feature of gelu(v) * 1, taken to every output by ones: its two bfloat16 parts leave out 2^-16 of it."""
    import torch
    t = types()[dtype]
    T, c, f = 100, 16, 24
    v = torch.linspace(-12.75, 6, T).to(t)
    x = torch.zeros(T, c, dtype=t)
    x[:, 0], x[:, 1] = v, 1
    wg, wu, wd = torch.zeros(1, f, c, dtype=t), torch.zeros(1, f, c, dtype=t), torch.zeros(1, c, f, dtype=t)
    wg[0, 3, 0], wu[0, 3, 1], wd[0, :, 3] = 1, 1, 1
    y = dyra.dyra_moe(x.cuda(), wg.cuda(), wu.cuda(), wd.cuda(), torch.zeros(T, 1, dtype=torch.int32).cuda(),
                      torch.ones(T, 1).cuda(), act="gelu")
    ref, bound = gelu_bound(v, t)
    ref, bound = ref[:, None].expand(T, c), bound[:, None].expand(T, c)
    close(y, ref, bound + (2.0 ** -16 * ref.abs() if dtype == "bf16" else 0))


@pytest.mark.parametrize("N", [3, 100])
def test_gelu_of_infinity_and_nan(N):
    import torch
    x, w = torch.zeros(N, 8, dtype=torch.bfloat16), torch.zeros(40, 8, dtype=torch.bfloat16)
    x[:, 0], w[:, 0] = 1, 1
    x[0, 0], x[1, 0] = float("inf"), float("nan")
    for o in (torch.bfloat16, torch.float32):
        y = dyra.dyra_linear(x.cuda(), w.cuda(), act="gelu", out_dtype=o)
        assert (y[0] == float("inf")).all() and y[1].isnan().all() and y[2:].isfinite().all()


# ------------------------------------------------------------------ router

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(6, 8, 2), (9, 64, 8), (5, 200, 5), (4, 300, 20), (3, 1024, 64)])
def test_sigmoid_scores_of_low_logits_are_renormalised(T, E, k, dtype):
    """Scores below float32's range (logits under -88) have ratios all the same.  Bound as for the softmax: exponents of
    at most 40 to 44 u each, k terms, quotients."""
    import torch
    logits = rand((T, E), 11, types()[dtype], 2.0).double()
    logits += torch.tensor([-95.0, -200.0, -3.0, -1e4, 2.0, -88.0, -60.0, 0.0, -104.0])[:T, None]
    logits = logits.to(types()[dtype])
    logits[1, k:] = -float("inf")                 # fewer left than places
    logits[1, 0] = -float("inf")
    ids, w = dyra.dyra_route(logits.cuda(), k, score="sigmoid", scale=1.5)
    l = logits.double()
    order = torch.from_numpy((-l.numpy()).argsort(axis=1, kind="stable")[:, :k].copy())
    top = l.gather(1, order)
    s = torch.where(top == -float("inf"), top, torch.nn.functional.logsigmoid(top))
    ref = 1.5 * torch.softmax(s, dim=1)
    assert (ids.cpu() == torch.where(top == -float("inf"), -1, order).int()).all()
    close(w, ref, (2 * 44 + k + 16) * 2 * U * ref)
    lowest = torch.full((2, E), torch.finfo(types()[dtype]).min, dtype=types()[dtype], device="cuda")
    equal = torch.full((2, k), 1 / k, dtype=torch.float64)
    close(dyra.dyra_route(lowest, k, score="sigmoid")[1], equal, 4 * U * equal)


# ------------------------------------------------------------------ refusals

def test_too_many_pairs_are_refused_without_a_workspace():
    """16384 tokens through 8 places of 14336 features would need 7.5 GB of it."""
    import torch
    T, k, c, f = 16384, 8, 8, 14336
    x = torch.zeros(T, c, dtype=torch.bfloat16, device="cuda")
    w, wd = torch.zeros(1, f, c, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, c, f, dtype=torch.bfloat16, device="cuda")
    ids, p = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(dyra.DyraError) as err:
        dyra.dyra_moe(x, w, w, wd, ids, p)
    assert err.value.status == 2 and torch.cuda.max_memory_allocated() - before < 1 << 20


# ------------------------------------------------------------------ silu where it is small

@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,c2", [(7, 48), (16, 8200), (300, 8), (300, 70), (4000, 2050)])
def test_silu_is_right_where_it_is_small(N, c2, dtype, out):
    """silu(-87) is -1.4e-36.  In float32 exp is right to 4 u, the reciprocal to 2 u, the sum and the product to u each: 8 u
    in all.  For bfloat16 results exp's argument is right to 2 u |v| and the rest to 8 u."""
    import torch
    t, o = types()[dtype], types()[out]
    v = torch.linspace(-87, 6, N).to(t)
    x, w, zero = torch.zeros(N, 8, dtype=t), torch.zeros(c2, 8, dtype=t), torch.zeros(c2, 8, dtype=t)
    x[:, 2], w[:, 2] = v, 1
    v = v.double()
    y = v / (1 + torch.exp(-v))
    own = (8 * U + (2 * U * v.abs() if out == "bf16" else 0)) * y.abs()
    bound = own + half(o) * (y.abs() + own)
    y, bound = y[:, None].expand(N, c2), bound[:, None].expand(N, c2)
    close(dyra.dyra_linear(x.cuda(), w.cuda(), act="silu", out_dtype=o), y, bound)
    if dtype == out:
        one = torch.ones(c2, dtype=t, device="cuda")
        close(dyra.dyra_gated(x.cuda(), w.cuda(), zero.cuda(), bias_u=one, act="silu"), y, bound, "gated")

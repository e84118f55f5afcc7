"""The feed-forward operators on the GPU against their definitions in float64.

Every output element is held to a bound derived from the arithmetic, for the
operands as rounded (u = 2^-24, the half step of float32; h = eps / 2 of the
output type):

* a product z of depth K accumulated in float32: |dz| <= 2 (K + 4) u S with
  S = sum |x| |w| + |b|.  (K + 4) u S bounds any order of summation; the factor
  2 covers matrix instructions that truncate where an addition would round.
* an activation's slope is at most 1.13 (gelu; silu 1.10) and its own float32
  evaluation is right to 16 u of max(|z|, |act|): |da| <= 1.13 |dz| + 16 u |z|.
* a gate: |dh| <= |da| |up| + |act| |dup| + |da| |dup|.
* the last sum and the rounding to the output type: 2 u of the terms, h |y|.

In the expert layer the inner activations are rounded to the operand type once
more (h of each) before the second product.
"""
import math

import pytest

from structured_rank_matmul_amd import dyra

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
U = 2.0 ** -24


def half(dtype):
    import torch
    return torch.finfo(dtype).eps / 2


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


def phi(z, act):
    import torch
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def rand(shape, seed, dtype, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype)


def product(x, w, b):
    """z and the bound of its float32 evaluation; host float64."""
    x, w = x.double(), w.double()
    z, s = x @ w.T, x.abs() @ w.abs().T
    if b is not None:
        z, s = z + b.double(), s + b.double().abs()
    return z, 2 * (x.shape[1] + 4) * U * s


def activated(z, dz, act):
    a = phi(z, act)
    return a, 1.13 * dz + (16 * U * z.abs() if act != "none" else 0)


def linear_ref(x, w, b, act, r, out):
    a, da = activated(*product(x, w, b), act)
    y = a + (r.double() if r is not None else 0)
    terms = a.abs() + (r.double().abs() if r is not None else 0)
    return y, da + 2 * U * terms + half(out) * (y.abs() + da)


def gated_ref(x, wg, wu, bg, bu, act, out):
    a, da = activated(*product(x, wg, bg), act)
    u, du = product(x, wu, bu)
    y = a * u
    d = da * u.abs() + a.abs() * du + da * du
    return y, d + 2 * U * y.abs() + half(out) * (y.abs() + d)


def close(got, ref, bound, label=""):
    d = (got.double().cpu() - ref).abs()
    bad = d > bound + 1e-30
    assert not bad.any() and not d.isnan().any(), (
        f"{label}: {int(bad.sum())} of {d.numel()} outside, worst at {bad.nonzero()[:3].tolist()}, "
        f"ratio {float((d / (bound + 1e-30)).max()):.3g}")


# tokens around the kernels' token groups and tiles, odd features, K with and without a partial slice
SHAPES = [(1, 64, 48), (1, 4096, 100), (2, 40, 1), (3, 8, 33), (5, 1032, 257), (16, 512, 64), (17, 72, 130), (33, 328, 16),
          (64, 96, 1003), (65, 136, 31), (100, 64, 64), (129, 520, 200), (257, 256, 257), (1000, 24, 513), (700, 1152, 1400)]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,c1,c2", SHAPES)
def test_linear(N, c1, c2, dtype, out):
    t, o = types()[dtype], types()[out]
    x, w = rand((N, c1), 1, t), rand((c2, c1), 2, t, c1 ** -0.5)
    b, r = rand((c2,), 3, t), rand((N, c2), 4, o)
    xd, wd, bd, rd = (v.cuda() for v in (x, w, b, r))
    for i, (act, bias, res) in enumerate([("none", False, False), ("gelu", True, True), ("silu", False, True),
                                          ("relu", True, False), ("gelu_tanh", True, True)]):
        y = dyra.dyra_linear(xd, wd, bias=bd if bias else None, act=act, residual=rd if res else None, out_dtype=o)
        assert y.dtype == o and tuple(y.shape) == (N, c2)
        close(y, *linear_ref(x, w, b if bias else None, act, r if res else None, o), f"{act} {bias} {res}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", SHAPES)
def test_gated(N, c1, c2, dtype):
    t = types()[dtype]
    x, wg, wu = rand((N, c1), 5, t), rand((c2, c1), 6, t, c1 ** -0.5), rand((c2, c1), 7, t, c1 ** -0.5)
    bg, bu = rand((c2,), 8, t), rand((c2,), 9, t)
    d = [v.cuda() for v in (x, wg, wu, bg, bu)]
    for act, bias in (("silu", False), ("gelu", True), ("none", True)):
        h = dyra.dyra_gated(d[0], d[1], d[2], bias_g=d[3] if bias else None, bias_u=d[4] if bias else None, act=act)
        close(h, *gated_ref(x, wg, wu, bg if bias else None, bu if bias else None, act, t), f"{act} {bias}")


# enough 256 x 256 tiles to fill the chip; one to six slabs of K, whole and partial; rows and features past the last tile
@pytest.mark.parametrize("N,c1,c2", [(4000, 8, 2050), (3841, 64, 2304), (4096, 72, 2048), (4100, 128, 2001), (3900, 192, 2100),
                                     (2100, 264, 4000), (4097, 320, 1930), (33000, 40, 100)])
def test_many_tiles(N, c1, c2):
    import torch
    t = torch.bfloat16
    x, w, w2 = rand((N, c1), 81, t), rand((c2, c1), 82, t, c1 ** -0.5), rand((c2, c1), 83, t, c1 ** -0.5)
    b, r = rand((c2,), 84, t), rand((N, c2), 85, t)
    xd, wd, w2d, bd, rd = (v.cuda() for v in (x, w, w2, b, r))
    close(dyra.dyra_linear(xd, wd, bias=bd, act="gelu", residual=rd), *linear_ref(x, w, b, "gelu", r, t))
    close(dyra.dyra_linear(xd, wd, out_dtype=torch.float32), *linear_ref(x, w, None, "none", None, torch.float32))
    close(dyra.dyra_gated(xd, wd, w2d, bias_u=bd), *gated_ref(x, w, w2, None, b, "silu", t))
    if c1 > 8:   # a column slice: rows further apart than they are long
        k = c1 // 2 // 8 * 8
        y = dyra.dyra_linear(xd[:, 8:8 + k], wd[:, :k])
        close(y, *linear_ref(x[:, 8:8 + k], w[:, :k], None, "none", None, t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 50, 200, 400])
def test_strided_rows_and_untouched_gaps(N, dtype):
    """Every matrix a column slice of a wider one; what lies between the rows and behind the last keeps its bits."""
    import torch
    t, c1, c2 = types()[dtype], 136, 77
    wide_x, wide_w = rand((N + 2, c1 + 40), 11, t).cuda(), rand((c2, c1 + 16), 12, t, c1 ** -0.5).cuda()
    wide_r = rand((N, c2 + 5), 13, t).cuda()
    x, w, r = wide_x[:N, 16:16 + c1], wide_w[:, 8:8 + c1], wide_r[:, 3:3 + c2]
    wide_y = torch.full((N + 3, c2 + 9), 7.0, dtype=t, device="cuda")
    y = wide_y[:N, 4:4 + c2]
    dyra.dyra_linear(x, w, residual=r, act="relu", Y=y)
    close(y, *linear_ref(x.cpu(), w.cpu(), None, "relu", r.cpu(), t))
    keep = wide_y.clone()
    keep[:N, 4:4 + c2] = 7.0
    assert torch.equal(keep, torch.full_like(keep, 7.0))
    h = torch.full((N + 3, c2 + 9), 7.0, dtype=t, device="cuda")
    dyra.dyra_gated(x, w, w, H=h[:N, 4:4 + c2])
    close(h[:N, 4:4 + c2], *gated_ref(x.cpu(), w.cpu(), w.cpu(), None, None, "silu", t))
    h[:N, 4:4 + c2] = 7.0
    assert torch.equal(h, torch.full_like(h, 7.0))


@pytest.mark.parametrize("N", [1, 40, 300])
def test_residual_in_place_and_one_row_for_all(N):
    import torch
    c1, c2 = 64, 96
    x, w, r = rand((N, c1), 14, torch.bfloat16), rand((c2, c1), 15, torch.bfloat16), rand((N, c2), 16, torch.bfloat16)
    y = r.cuda()
    assert dyra.dyra_linear(x.cuda(), w.cuda(), residual=y, Y=y) is y
    close(y, *linear_ref(x, w, None, "none", r, torch.bfloat16))
    one = r[:1].expand(N, c2)
    y = dyra.dyra_linear(x.cuda(), w.cuda(), residual=r[:1].cuda().expand(N, c2))
    close(y, *linear_ref(x, w, None, "none", one, torch.bfloat16))


@pytest.mark.parametrize("N", [4, 40, 300])
def test_infinities_and_nan_stay_in_their_rows(N):
    import torch
    c1, c2 = 72, 90
    x, w = rand((N, c1), 17, torch.bfloat16), rand((c2, c1), 18, torch.bfloat16)
    clean = dyra.dyra_linear(x.cuda(), w.cuda(), act="silu")
    x[1, 5], x[3, 71] = float("inf"), float("nan")
    y = dyra.dyra_linear(x.cuda(), w.cuda(), act="silu")
    rows = [i for i in range(N) if i not in (1, 3)]
    assert torch.equal(y[rows], clean[rows])
    assert y[3].isnan().all() and not y[1].isfinite().all()
    assert dyra.dyra_linear(x.cuda(), w.cuda(), act="relu")[3].isnan().all()


def test_empty_batches():
    import torch
    x, w = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    assert tuple(dyra.dyra_linear(x, w).shape) == (0, 8)
    assert tuple(dyra.dyra_gated(x, w, w).shape) == (0, 8)
    ids, wt = dyra.dyra_route(torch.zeros(0, 6, device="cuda"), 2)
    assert tuple(ids.shape) == tuple(wt.shape) == (0, 2)
    e = torch.zeros(6, 16, 64, device="cuda", dtype=torch.bfloat16)
    assert tuple(dyra.dyra_moe(x, e, e, e.transpose(1, 2).contiguous(), ids, wt).shape) == (0, 64)


# ------------------------------------------------------------------ router

def route_ref(logits, k, score, renormalise, scale):
    import torch
    l = logits.double()
    l = torch.where(l.isnan(), torch.full_like(l, -math.inf), l)
    order = torch.from_numpy((-l.numpy()).argsort(axis=1, kind="stable")[:, :k].copy())
    top = l.gather(1, order)
    gone = top == -math.inf
    if score == "softmax":
        m = l.amax(dim=1, keepdim=True)
        e = torch.where(l == m, torch.ones_like(l), torch.exp(l - m))
        e = torch.where(l == -math.inf, torch.zeros_like(l), e)
        w = e.gather(1, order) / e.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        w = torch.sigmoid(top)
    w = torch.where(gone, torch.zeros_like(w), w)
    if renormalise:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return torch.where(gone, torch.full_like(order, -1), order).int(), scale * w


def check_route(logits, k, score="softmax", renormalise=True, scale=1.0):
    """ids exactly; weights to the float32 evaluation: an exponent of |l - m| <= 40 is right to 40 u + 4 u relative, a
    sum of E terms to (E + 4) u, a quotient and two products to 4 u."""
    ids, w = dyra.dyra_route(logits.cuda(), k, score=score, renormalise=renormalise, scale=scale)
    rid, rw = route_ref(logits, k, score, renormalise, scale)
    assert (ids.cpu() == rid).all()
    close(w, rw, (2 * 44 + logits.shape[1] + 16) * 2 * U * rw.abs())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 64, 8), (7, 65, 64), (33, 128, 8), (4, 257, 16), (3, 1024, 64),
                                   (1025, 60, 4), (2, 513, 1), (9, 3, 3)])
def test_route(T, E, k, dtype):
    # in bf16 many logits are equal: the lowest index is chosen first
    logits = rand((T, E), 21, types()[dtype], 2.0)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            check_route(logits, k, score, renormalise, 1.0 if renormalise else 2.5)


@pytest.mark.parametrize("E,k", [(6, 4), (64, 8), (128, 8), (200, 5)])
def test_route_masked_ties_and_special_values(E, k):
    import torch
    logits = rand((12, E), 22, torch.float32)
    logits[0] = -math.inf                      # nothing left
    logits[1, 1:] = -math.inf                  # one left, fewer than k
    logits[2] = 0.0                            # all equal
    logits[3, ::2], logits[3, 1::2] = 0.0, -0.0   # equal too
    logits[4, 3] = math.nan                    # never chosen
    logits[5, 2] = math.inf                    # takes all
    logits[6, :2] = math.inf                   # share it
    logits[7] = torch.finfo(torch.float32).min   # the lowest finite value is a value
    logits[8, :-1] = -math.inf
    logits[9, E // 2:] = torch.finfo(torch.float32).min
    logits[10] = math.nan
    for renormalise in (True, False):
        check_route(logits, k, "softmax", renormalise)
    ids, w = dyra.dyra_route(logits.cuda(), k, score="sigmoid")
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[10] == -1).all() and (w[10] == 0).all()
    assert ids[2].tolist() == list(range(k)) and ids[3].tolist() == list(range(k))


def test_route_strided_rows():
    import torch
    wide = rand((20, 50), 23, torch.float32).cuda()
    ids, w = dyra.dyra_route(wide[:, 5:35], 3)
    rid, rw = route_ref(wide[:, 5:35].cpu(), 3, "softmax", True, 1.0)
    assert (ids.cpu() == rid).all()
    close(w, rw, 400 * U * rw)


# ------------------------------------------------------------------ expert layer

def moe_ref(x, wg, wu, wd, ids, w, act, r):
    """Y and its bound, pair by pair."""
    import torch
    t = x.dtype
    T, c = x.shape
    y = torch.zeros(T, c, dtype=torch.float64) if r is None else r.double().clone()
    terms, d = y.abs().clone(), torch.zeros(T, c, dtype=torch.float64)
    f = wg.shape[1]
    for i in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[i, j])
            if not 0 <= e < wg.shape[0]:
                continue
            h, dh = gated_ref(x[i:i + 1], wg[e], wu[e], None, None, act, t)   # dh holds the rounding of h to t
            p, wde = float(w[i, j]), wd[e].double()
            o, s = h @ wde.T, h.abs() @ wde.abs().T
            y[i] += p * o[0]
            terms[i] += abs(p) * o[0].abs()
            d[i] += abs(p) * ((dh @ wde.abs().T)[0] + 2 * (f + 4) * U * (s + dh @ wde.abs().T)[0])
    d += 2 * (ids.shape[1] + 4) * U * (terms + d)
    return y, d + half(t) * (y.abs() + d)


def experts(E, c, f, seed, t):
    return (rand((E, f, c), seed, t, c ** -0.5), rand((E, f, c), seed + 1, t, c ** -0.5),
            rand((E, c, f), seed + 2, t, f ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,c,f", [(1, 4, 1, 64, 32), (1, 64, 8, 128, 96), (3, 8, 2, 72, 40), (16, 8, 2, 256, 136),
                                       (40, 4, 3, 64, 264), (64, 16, 8, 96, 64), (100, 3, 2, 40, 24), (128, 32, 8, 64, 48),
                                       (1, 1, 1, 8, 8), (5, 300, 6, 64, 16), (16, 1, 64, 64, 64), (1024, 2, 1, 32, 16)])
def test_moe(T, E, k, c, f, dtype):
    import torch
    t = types()[dtype]
    x, r = rand((T, c), 31, t), rand((T, c), 32, t)
    w3 = experts(E, c, f, 33, t)
    g = torch.Generator().manual_seed(36)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, dtype=torch.int32)   # -1 and E: empty places; repeats
    w = torch.rand(T, k, generator=g)
    w[ids < 0] = math.nan                                                    # an empty place's weight is not read into Y
    dev = [v.cuda() for v in (x, *w3, ids, w)]
    y = dyra.dyra_moe(*dev, act="silu", residual=r.cuda())
    close(y, *moe_ref(x, *w3, ids, w, "silu", r))
    y2 = dyra.dyra_moe(*dev, act="gelu")
    close(y2, *moe_ref(x, *w3, ids, w, "gelu", None))
    assert torch.equal(y2, dyra.dyra_moe(*dev, act="gelu"))


def test_moe_rows_with_no_expert_and_one_expert_for_all():
    import torch
    T, E, k, c, f = 20, 5, 2, 64, 48
    x, r, w3 = rand((T, c), 41, torch.bfloat16), rand((T, c), 42, torch.bfloat16), experts(E, c, f, 43, torch.bfloat16)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.ones(T, k)
    dev = [v.cuda() for v in (x, *w3)]
    assert torch.equal(dyra.dyra_moe(*dev, ids.cuda(), w.cuda(), residual=r.cuda()).cpu(), r)
    assert (dyra.dyra_moe(*dev, ids.cuda(), w.cuda()) == 0).all()
    ids[:] = 3                                                              # twice for every token
    close(dyra.dyra_moe(*dev, ids.cuda(), w.cuda(), residual=r.cuda()), *moe_ref(x, *w3, ids, w, "silu", r))
    y = r.cuda()                                                            # in place, and strided
    wide = torch.full((T + 1, c + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:T, 8:8 + c] = dev[0]
    dyra.dyra_moe(wide[:T, 8:8 + c], *dev[1:], ids.cuda(), w.cuda(), residual=y, Y=y)
    close(y, *moe_ref(x, *w3, ids, w, "silu", r))
    out = torch.full((T + 1, c + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    dyra.dyra_moe(*dev, ids.cuda(), w.cuda(), residual=r.cuda(), Y=out[:T, 1:1 + c])
    assert torch.equal(out[:T, 1:1 + c], y) and (out[T] == 7).all() and (out[:, 0] == 7).all() and (out[:, 1 + c:] == 7).all()


# ------------------------------------------------------------------ together, streams, graphs

def block(x, p, stream=None):
    """A mixture-of-experts block: router logits in float32, routing, the experts on top of the residual, then a dense
    gated MLP on top of that."""
    import torch
    logits = dyra.dyra_linear(x, p["router"], out_dtype=torch.float32, stream=stream)
    ids, w = dyra.dyra_route(logits, 4, stream=stream)
    y = dyra.dyra_moe(x, p["wg"], p["wu"], p["wd"], ids, w, residual=x, stream=stream)
    h = dyra.dyra_gated(y, p["gate"], p["up"], stream=stream)
    return ids, w, y, dyra.dyra_linear(h, p["down"], bias=p["bias"], residual=y, stream=stream)


def block_params(c=128, f=64, F=200, E=16, seed=51):
    import torch
    t = torch.bfloat16
    wg, wu, wd = experts(E, c, f, seed, t)
    host = {"router": rand((E, c), seed + 3, t, c ** -0.5), "wg": wg, "wu": wu, "wd": wd,
            "gate": rand((F, c), seed + 4, t, c ** -0.5), "up": rand((F, c), seed + 5, t, c ** -0.5),
            "down": rand((c, F), seed + 6, t, F ** -0.5), "bias": rand((c,), seed + 7, t)}
    return host, {k: v.cuda() for k, v in host.items()}


@pytest.mark.parametrize("T", [1, 7, 64, 128])
def test_block_of_all_operators(T):
    import torch
    host, p = block_params()
    x = rand((T, 128), 61, torch.bfloat16)
    ids, w, y, z = block(x.cuda(), p)
    # each step against its definition on the step's own inputs
    logits = dyra.dyra_linear(x.cuda(), p["router"], out_dtype=torch.float32).cpu()
    rid, rw = route_ref(logits, 4, "softmax", True, 1.0)
    assert (ids.cpu() == rid).all()
    close(w, rw, 400 * U * rw)
    close(y, *moe_ref(x, host["wg"], host["wu"], host["wd"], ids.cpu(), w.cpu(), "silu", x))
    h = dyra.dyra_gated(y, p["gate"], p["up"]).cpu()
    close(z, *linear_ref(h, host["down"], host["bias"], "none", y.cpu(), torch.bfloat16))


def test_gated_product_into_the_approximate_down_product():
    """The gated pair feeds dyra_forward, the library's approximate product, where the down layer is replaced by one."""
    import numpy as np
    import torch

    import oracle as orc
    from structured_rank_matmul_amd import synth
    from gpu_util import check_parity
    B, n, c, F = 3, 70, 96, 128
    W = synth.random_weight(F, c, 71, p=0.6)
    plan = dyra.dyra_prepare(W, 24, 8, 0.0, "bf16", 0)
    x = rand((B * n, c), 72, torch.bfloat16)
    wg, wu = rand((F, c), 73, torch.bfloat16, c ** -0.5), rand((F, c), 74, torch.bfloat16, c ** -0.5)
    h = dyra.dyra_gated(x.cuda(), wg.cuda(), wu.cuda())
    close(h, *gated_ref(x, wg, wu, None, None, "silu", torch.bfloat16))
    y = dyra.dyra_forward(h, B, n, plan).double().cpu().numpy()
    ref = orc.inference(h.double().cpu().numpy(), B, n, orc.offline_preparation(W.astype(np.float64), 24, 8, 0.0))
    check_parity(y, ref, n, "bf16", "gated -> dyra_forward")
    plan.close()


def test_two_streams_and_repeats_agree_bit_for_bit():
    import torch
    _, p = block_params()
    xa, xb = rand((64, 128), 62, torch.bfloat16).cuda(), rand((128, 128), 63, torch.bfloat16).cuda()
    ra, rb = block(xa, p), block(xb, p)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got.append((block(xa, p, s1), ra))
        got.append((block(xb, p, s2), rb))
    filler = [torch.full((128, 128), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(8)]
    torch.cuda.synchronize()
    for g, r in got:
        assert all(torch.equal(u, v) for u, v in zip(g, r))
    del filler


@pytest.mark.parametrize("T", [1, 40, 100])
def test_captured_block_replays_with_new_inputs(T):
    """Two graphs of the block, replayed in turn with eager work between: every replay equals the eager result."""
    import torch
    _, p = block_params()
    static = [rand((T, 128), 64 + i, torch.bfloat16).cuda() for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in static:
            block(x, p)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block(x, p))
        graphs.append(g)
    for i in range(5):
        for k in range(2):
            static[k].copy_(rand((T, 128), 80 + 2 * i + k, torch.bfloat16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            eager = block(static[k], p)
            assert all(torch.equal(u, v) for u, v in zip(outs[k], eager)), f"replay {i} of graph {k}"


def test_binding_refuses_mismatched_tensors():
    import torch
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(8, 64, device="cuda")
    bad = [lambda: dyra.dyra_linear(x, w.bfloat16()), lambda: dyra.dyra_linear(x, w[:, :32]),
           lambda: dyra.dyra_linear(x, w, bias=torch.zeros(9, device="cuda")),
           lambda: dyra.dyra_linear(x, w, bias=torch.zeros(8)), lambda: dyra.dyra_linear(x, w.cpu()),
           lambda: dyra.dyra_linear(x, w, residual=torch.zeros(4, 9, device="cuda")),
           lambda: dyra.dyra_linear(x, w, Y=torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)),
           lambda: dyra.dyra_linear(x, w, Y=torch.zeros(1, 8, device="cuda").expand(4, 8)),
           lambda: dyra.dyra_linear(x, w, act="swish"), lambda: dyra.dyra_linear(x.half(), w.half()),
           lambda: dyra.dyra_linear(x.t(), w), lambda: dyra.dyra_linear(x[0], w),
           lambda: dyra.dyra_gated(x, w, torch.zeros(9, 64, device="cuda")),
           lambda: dyra.dyra_gated(x, w, torch.zeros(8, 128, device="cuda")[:, :64]),
           lambda: dyra.dyra_route(x, 0), lambda: dyra.dyra_route(x, 65), lambda: dyra.dyra_route(x, 2, score="max")]
    e = torch.zeros(3, 16, 64, device="cuda")
    d, ids, wt = torch.zeros(3, 64, 16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    bad += [lambda: dyra.dyra_moe(x, e, e, e, ids, wt), lambda: dyra.dyra_moe(x, e, e, d, ids.long(), wt),
            lambda: dyra.dyra_moe(x, e, e, d, ids, wt.bfloat16()), lambda: dyra.dyra_moe(x, e, e, d, ids[:3], wt),
            lambda: dyra.dyra_moe(x, e.transpose(1, 2), e, d, ids, wt), lambda: dyra.dyra_moe(x, e, e, d, ids.cpu(), wt)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(dyra.DyraError) as err:      # rows of 60 floats end inside a 16-byte chunk of the last slice: fine;
        dyra.dyra_linear(x[:, :62].contiguous(), w[:, :62].contiguous())   # 62 do not
    assert err.value.status == 2
    with pytest.raises(dyra.DyraError) as err:
        dyra.dyra_moe(x, e, e, d, ids, wt, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert err.value.status == 8

"""The norm, the quantisation of rows and the products of 8-bit integers on the GPU against their definitions in float64.

Every element is held to a bound derived from the arithmetic (u = 2^-24, the half step of float32; h = eps / 2 of the
output type):

* rho = 1 / sqrt(mean z^2 + eps): the terms are positive, and every lane of 64 at least adds c / 64 of them before a tree
  joins the lanes' sums: (c / 64 + 16) u for the sum, half of it and 8 u after root and division; z itself is right to u,
  squared 2 u.  y = z rho w: 4 u more.  NORM(c) = (c / 64 + 32) u of |y| is above all of that.
* S: one addition and one rounding, u |z| + h |z|.
* scales: the largest |y| (right as y is) over 127: 4 u more.
* whole numbers: |q - y / s| <= 1/2 + 127 (NORM + 4 u): a division and a product, of values up to 127.
* dequantised values: u and h of themselves.
* products: sums of integers are exact; their conversion, the product of the scales and its product with the sum are
  right to u each: 4 u (|product| + |bias|); the epilogue as in test_gpu_ffn.
"""
import math

import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import activated, close, half, rand, types, U
from test_gpu_ffn_shapes import on_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5
LEAST = 127.0 * 2.0 ** -126


# ------------------------------------------------------------------ rows

def relative(c, normed=True):
    return (c / 64 + 32) * U if normed else 0.0


def norm_ref(x, w, eps, r):
    """z, y in float64."""
    z = x.double() if r is None else x.double() + r.double()
    y = z / (z.square().mean(dim=1, keepdim=True) + eps).sqrt()
    return z, y if w is None else y * w.double()


def check_norm(y, ref, c):
    d = relative(c) * ref.abs()
    close(y, ref, d + half(y.dtype) * (ref.abs() + d))


def check_sum(s, z):
    close(s, z, (U + half(s.dtype)) * z.abs() * 1.01)


def check_rows(q, scales, ref, normed):
    """Scales and whole numbers against the values they are taken of."""
    import torch
    off = relative(ref.shape[1], normed)
    step = ref.abs().amax(dim=1).clamp(min=LEAST) / 127
    assert q.dtype == torch.int8 and scales.dtype == torch.float32
    assert ((scales.cpu().double() - step).abs() <= (off + 4 * U) * step).all()
    q = q.cpu().double()
    assert q.abs().max() <= 127
    far = (q - ref / step[:, None]).abs()
    assert (far <= 0.5 + 127 * (off + 4 * U)).all(), float(far.max())
    assert (q.abs().amax(dim=1)[ref.abs().amax(dim=1) > LEAST] == 127).all()


# lengths from one element over every number of elements that a thread may hold, whole and not
LENGTHS = [1, 2, 3, 7, 8, 9, 31, 63, 64, 65, 127, 255, 257, 500, 511, 512, 513, 1003, 1024, 2040, 2047, 2048, 2049, 4095, 4096, 4097,
           6144, 8191, 8192, 8200, 12289, 14336, 16384, 16385, 20000, 32767, 32768, 32776, 40001, 65535, 65536]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", LENGTHS)
def test_rows_of_every_length(c, dtype):
    import torch
    t = types()[dtype]
    for N in (1, 5, 70) if c > 9000 else (1, 3, 70, 1030):
        x, r, w = rand((N, c), 1, t, 3.0), rand((N, c), 2, t), rand((c,), 3, t)
        xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
        z, y = norm_ref(x, w, EPS, r)
        got, s = dyra.dyra_norm(xd, wd, EPS, residual=rd)
        assert got.dtype == s.dtype == t and tuple(got.shape) == tuple(s.shape) == (N, c)
        check_norm(got, y, c)
        check_sum(s, z)
        check_norm(dyra.dyra_norm(xd, eps=0.5), norm_ref(x, None, 0.5, None)[1], c)
        q, scales, s2 = dyra.dyra_norm_quantize(xd, wd, EPS, residual=rd)
        check_rows(q, scales, y, True)
        assert torch.equal(s, s2)
        check_rows(*dyra.dyra_norm_quantize(xd, wd, EPS), norm_ref(x, w, EPS, None)[1], True)
        q, scales = dyra.dyra_quantize(xd)
        check_rows(q, scales, x.double(), False)
        for out in (torch.bfloat16, torch.float32):
            v = q.cpu().double() * scales.cpu().double()[:, None]
            close(dyra.dyra_dequantize(q, scales, out), v, (U + half(out)) * v.abs() * 1.01)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [1, 5, 64, 77, 1000, 4100, 14336, 33000])
def test_strided_rows_and_untouched_gaps(c, dtype):
    """Every matrix a column slice of a wider one, at odd offsets; what lies between the rows and behind the last keeps
    its bits."""
    import torch
    t, N = types()[dtype], 9
    wide = [rand((N + 2, c + 13), 4 + i, t).cuda() for i in range(2)]
    x, r, w = wide[0][1:N + 1, 3:3 + c], wide[1][1:N + 1, 5:5 + c], rand((c + 1,), 6, t).cuda()[1:]
    w = w.clone() if not w.is_contiguous() else w
    z, y = norm_ref(x.cpu(), w.cpu(), EPS, r.cpu())

    def outputs(dt, at):
        base = torch.full((N + 3, c + 11), 7, dtype=dt, device="cuda")
        return base, base[1:N + 1, at:at + c]

    def untouched(base, at):
        base[1:N + 1, at:at + c] = 7
        assert (base == 7).all()

    (by, vy), (bs, vs), (bq, vq) = outputs(t, 1), outputs(t, 4), outputs(torch.int8, 3)
    scales = torch.full((N + 4,), 7.0, device="cuda")
    dyra.dyra_norm(x, w, EPS, residual=r, S=vs, Y=vy)
    check_norm(vy, y, c)
    check_sum(vs, z)
    untouched(by, 1)
    untouched(bs, 4)
    dyra.dyra_norm_quantize(x, w, EPS, residual=r, S=vs, Q=vq, scales=scales[2:2 + N])
    check_rows(vq, scales[2:2 + N], y, True)
    check_sum(vs, z)
    v = vq.cpu().double() * scales[2:2 + N].cpu().double()[:, None]
    dyra.dyra_dequantize(vq, scales[2:2 + N], t, X=vy)
    close(vy, v, (U + half(t)) * v.abs() * 1.01)
    for b, at in ((by, 1), (bs, 4), (bq, 3)):
        untouched(b, at)
    scales[2:2 + N] = 7.0
    assert (scales == 7).all()
    dyra.dyra_quantize(x, Q=vq, scales=scales[1:1 + N])
    check_rows(vq, scales[1:1 + N], x.cpu().double(), False)
    untouched(bq, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,c", [(1, 77), (6, 4096), (300, 1000), (4, 20001)])
def test_residual_and_input_in_place_and_one_row_for_all(N, c, dtype):
    import torch
    t = types()[dtype]
    x, r, w = rand((N, c), 11, t), rand((N, c), 12, t), rand((c,), 13, t).cuda()
    z, y = norm_ref(x, w.cpu(), EPS, r)
    xd, rd = x.cuda(), r.cuda()
    got, s = dyra.dyra_norm(xd, w, EPS, residual=rd, S=rd, Y=xd)
    assert got is xd and s is rd
    check_norm(xd, y, c)
    check_sum(rd, z)
    rd = r.cuda()
    q, scales, s = dyra.dyra_norm_quantize(x.cuda(), w, EPS, residual=rd, S=rd)
    assert s is rd
    check_rows(q, scales, y, True)
    check_sum(rd, z)
    z, y = norm_ref(x, w.cpu(), EPS, r[:1].expand(N, c))
    got, s = dyra.dyra_norm(x.cuda(), w, EPS, residual=r[:1].cuda().expand(N, c))
    check_norm(got, y, c)
    check_sum(s, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [3, 64, 1000, 4096, 9000])
def test_rows_of_zeros_extremes_and_values_that_are_not_finite(c, dtype):
    """Rows that cannot be scaled or normed as the others; no other row changes."""
    import torch
    t = types()[dtype]
    x = rand((40, c), 21, t)
    clean = x.clone()
    big = torch.finfo(t).max
    special = {3: 0.0, 5: math.inf, 7: math.nan, 9: -math.inf, 11: big, 13: torch.finfo(t).tiny, 15: -big}
    for row, v in special.items():
        x[row, c // 2] = v
    x[3], x[13] = 0.0, torch.finfo(t).tiny       # all zeros; all at the smallest normal number
    x[17] = clean[17].double().mul(1e30).to(t)   # squares past float32's range
    x[19] = clean[19].double().mul(1e-30).to(t)  # and below it
    x[21] = big                                  # every one the largest
    same = [i for i in range(40) if i not in (*special, 17, 19, 21)]
    bad = [5, 7, 9]
    fine = [i for i in range(40) if i not in bad]
    w = rand((c,), 22, t)
    z, y = norm_ref(x[fine], w, EPS, None)
    got = dyra.dyra_norm(x.cuda(), w.cuda(), EPS)
    check_norm(got[fine], y, c)
    assert torch.equal(got[same], dyra.dyra_norm(clean.cuda(), w.cuda(), EPS)[same])
    for i in bad:
        assert got[i, c // 2].isnan() and (got[i].isnan() | (got[i] == 0)).all()
    assert got[7].isnan().all()
    for q, scales, ref in ((*dyra.dyra_quantize(x.cuda()), x[fine].double()),
                           (*dyra.dyra_norm_quantize(x.cuda(), w.cuda(), EPS), y)):
        check_rows(q[fine], scales[fine], ref, True)
        assert scales[bad].isnan().all() and (q[bad] == 0).all() and (q[3] == 0).all() and scales[3] == 2.0 ** -126
        assert dyra.dyra_dequantize(q, scales)[bad].isnan().all()
    q, scales = dyra.dyra_quantize(x.cuda())
    q2, scales2 = dyra.dyra_quantize(clean.cuda())
    assert torch.equal(q[same], q2[same]) and torch.equal(scales[same], scales2[same])


def test_masked_values_and_weights():
    """A residual that lifts a row to the type's lowest value and past it; weights of zero and of infinity."""
    import torch
    N, c = 6, 300
    x, r, w = rand((N, c), 23, torch.bfloat16), rand((N, c), 24, torch.bfloat16), rand((c,), 25, torch.bfloat16)
    low = torch.finfo(torch.bfloat16).min
    r[1], x[2, 5], r[2, 5] = low, low, low       # the sum of the last leaves float32's range
    w[:10] = 0.0
    fine = [0, 1, 3, 4, 5]
    z, y = norm_ref(x, w, EPS, r)
    got, s = dyra.dyra_norm(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    check_norm(got[fine], y[fine], c)
    check_sum(s[fine], z[fine])
    assert s[2, 5] == -math.inf and got[2, 5].isnan()
    q, scales, _ = dyra.dyra_norm_quantize(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    check_rows(q[fine], scales[fine], y[fine], True)
    assert scales[2].isnan() and (q[2] == 0).all()
    w[20] = math.inf
    q, scales, _ = dyra.dyra_norm_quantize(x.cuda(), w.cuda(), EPS, residual=r.cuda())
    assert scales.isnan().all() and (q == 0).all()


def spread(rows, cols, stride, dtype):
    import torch
    return torch.empty((rows - 1) * stride + cols, dtype=dtype, device="cuda").as_strided((rows, cols), (stride, 1))


@pytest.mark.parametrize("N,c", [(5, 1000), (300, 72)])
def test_rows_past_32_bits(N, c):
    """Rows whose last lies 2^32 elements and more behind the first, of every matrix."""
    import torch
    t, step = torch.bfloat16, (1 << 32) // (N - 1) + 17
    x, r, w = spread(N, c, step, t), spread(N, c, step, t), rand((c,), 33, t)
    x.copy_(rand((N, c), 31, t))
    r.copy_(rand((N, c), 32, t))
    z, y = norm_ref(x.cpu(), w, EPS, r.cpu())
    s, out, q = spread(N, c, step, t), spread(N, c, step, t), spread(N, c, step, torch.int8)
    dyra.dyra_norm(x, w.cuda(), EPS, residual=r, S=s, Y=out)
    check_norm(out, y, c)
    check_sum(s, z)
    _, scales, _ = dyra.dyra_norm_quantize(x, w.cuda(), EPS, residual=r, S=s, Q=q)
    check_rows(q, scales, y, True)
    _, scales = dyra.dyra_quantize(x, Q=q)
    check_rows(q, scales, x.cpu().double(), False)
    v = q.cpu().double() * scales.cpu().double()[:, None]
    dyra.dyra_dequantize(q, scales, X=out)
    close(out, v, (U + half(t)) * v.abs() * 1.01)


def test_many_rows():
    """More rows than a launch has workgroups of them, and more elements than 2^31."""
    import torch
    N, c, t = 3_000_017, 720, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(41)
    x = torch.empty(N, c, dtype=t, device="cuda").normal_(generator=g)
    w = rand((c,), 42, t)
    out = dyra.dyra_norm(x, w.cuda(), EPS)
    q, scales = dyra.dyra_quantize(x)
    back = dyra.dyra_dequantize(q, scales)
    for s in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
        xs = x[s].cpu()
        check_norm(out[s], norm_ref(xs, w, EPS, None)[1], c)
        check_rows(q[s], scales[s], xs.double(), False)
        v = q[s].cpu().double() * scales[s].cpu().double()[:, None]
        close(back[s], v, (U + half(t)) * v.abs() * 1.01)


def test_empty_batches():
    import torch
    x = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(8, 64, device="cuda", dtype=torch.int8)
    sw = torch.ones(8, device="cuda")
    assert tuple(dyra.dyra_norm(x).shape) == (0, 64)
    q, scales, s = dyra.dyra_norm_quantize(x, residual=x)
    assert tuple(q.shape) == tuple(s.shape) == (0, 64) and tuple(scales.shape) == (0,)
    assert tuple(dyra.dyra_dequantize(*dyra.dyra_quantize(x)).shape) == (0, 64)
    assert tuple(dyra.dyra_linear_quantized(q, scales, w, sw).shape) == (0, 8)
    assert tuple(dyra.dyra_gated_quantized(q, scales, w, sw, w, sw).shape) == (0, 8)


# ------------------------------------------------------------------ products

def eight(shape, seed, scale=1.0):
    """(int8 over the whole range, float32 scales of about `scale` / 74, so that a value is about `scale`)."""
    import torch
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)
    return q, (torch.rand(shape[0], generator=g) + 0.5) * (scale / 74)


def product(x, sx, w, sw, b):
    """z and the bound of its evaluation."""
    z = (x.double() @ w.double().T.contiguous()) * sx.double()[:, None] * sw.double()
    s = z.abs()
    if b is not None:
        z, s = z + b.double(), s + b.double().abs()
    return z, 4 * U * s


def linear_ref(x, sx, w, sw, b, act, r, out):
    a, da = activated(*product(x, sx, w, sw, b), act)
    y = a + (r.double() if r is not None else 0)
    terms = a.abs() + (r.double().abs() if r is not None else 0)
    return y, da + 2 * U * terms + half(out) * (y.abs() + da)


def gated_ref(x, sx, g, sg, u, su, bg, bu, act, out):
    a, da = activated(*product(x, sx, g, sg, bg), act)
    p, dp = product(x, sx, u, su, bu)
    y = a * p
    d = da * p.abs() + a.abs() * dp + da * dp
    return y, d + 2 * U * y.abs() + half(out) * (y.abs() + d)


# tokens around the kernels' token groups and tiles, odd features, K of one step and of partial slabs
SHAPES = [(1, 64, 48), (1, 4096, 100), (2, 48, 1), (3, 16, 33), (5, 1040, 257), (16, 512, 64), (17, 80, 130), (33, 336, 16),
          (64, 96, 1003), (65, 144, 31), (100, 64, 64), (129, 528, 200), (257, 256, 257), (1000, 32, 513), (700, 1152, 1400)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", SHAPES)
def test_linear(N, c1, c2, out):
    o = types()[out]
    (x, sx), (w, sw) = eight((N, c1), 51), eight((c2, c1), 52, c1 ** -0.5)
    b, r = rand((c2,), 53, o), rand((N, c2), 54, o)
    xd, sxd, wd, swd, bd, rd = (v.cuda() for v in (x, sx, w, sw, b, r))
    for act, bias, res in [("none", False, False), ("gelu", True, True), ("silu", False, True), ("relu", True, False),
                           ("gelu_tanh", True, True)]:
        y = dyra.dyra_linear_quantized(xd, sxd, wd, swd, bias=bd if bias else None, act=act, residual=rd if res else None, out_dtype=o)
        assert y.dtype == o and tuple(y.shape) == (N, c2)
        close(y, *linear_ref(x, sx, w, sw, b if bias else None, act, r if res else None, o), f"{act} {bias} {res}")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,c1,c2", SHAPES)
def test_gated(N, c1, c2, out):
    o = types()[out]
    (x, sx), (g, sg), (u, su) = eight((N, c1), 55), eight((c2, c1), 56, c1 ** -0.5), eight((c2, c1), 57, c1 ** -0.5)
    bg, bu = rand((c2,), 58, o), rand((c2,), 59, o)
    d = [v.cuda() for v in (x, sx, g, sg, u, su)]
    for act, bias in (("silu", False), ("gelu", True), ("none", True)):
        b = (bg, bu) if bias else (None, None)
        h = dyra.dyra_gated_quantized(*d, *(v.cuda() if v is not None else None for v in b), act=act, out_dtype=o)
        assert h.dtype == o
        close(h, *gated_ref(x, sx, g, sg, u, su, *b, act, o), f"{act} {bias}")


@pytest.mark.parametrize("c2", [2304, 4096])
def test_gelu_of_large_tiles(c2):
    """bf16 results of large tiles take Phi from lines of 1 / 256: off by h^2 t^2 / 16 of themselves at most (1.6e-4 at
    12.9) and a rounding of each line's two coefficients (t^2 u each), from an argument off by 2 u (t^2 2 u)."""
    import torch
    N, c1 = 4096, 16
    x, w = torch.zeros(N, c1, dtype=torch.int8), torch.zeros(c2, c1, dtype=torch.int8)
    x[:, 3], w[:, 3] = 1, 1
    sx, sw = torch.linspace(-13.0, 13.0, N), 1.0 - torch.arange(c2) * 2.0 ** -17
    sx[:6] = torch.tensor([float("nan"), float("inf"), float("-inf"), -1e30, -13.3, 1e30])
    d = [v.cuda() for v in (x, sx, w, sw)]
    z = sx.double()[:, None] * sw.double()
    t2 = z[6:] * z[6:]
    ref = 0.5 * z[6:] * torch.special.erfc(-z[6:] * 0.5 ** 0.5)
    bound = (half(torch.bfloat16) + 1.002 * (t2 + 1) / 16 / 65536 + 4 * U * (t2 + 2)) * ref.abs() + 1e-36
    one = torch.ones(c2, dtype=torch.bfloat16, device="cuda")
    linear = dyra.dyra_linear_quantized(*d, act="gelu").double().cpu()
    gated = dyra.dyra_gated_quantized(*d, torch.zeros_like(d[2]), d[3], bias_u=one, act="gelu").double().cpu()
    assert (linear[1] == float("inf")).all() and (linear[2] == 0).all()
    assert gated[1:3].isnan().all()   # the up sums of 0 times an infinite scale
    for y in (linear, gated):
        assert y[0].isnan().all() and (y[3:5].abs() <= 1e-36).all()
        assert ((y[5] / z[5] - 1).abs() <= half(torch.bfloat16)).all()
        close(y[6:], ref, bound)


# enough large tiles to fill the chip; one slab of K to several, whole and partial; rows and features past the last tile
@pytest.mark.parametrize("N,c1,c2", [(4000, 16, 2050), (3841, 128, 2304), (4096, 144, 2048), (4100, 256, 2001), (3900, 384, 2100),
                                     (2100, 528, 4000), (4097, 640, 1930), (33000, 80, 100)])
def test_many_tiles(N, c1, c2):
    import torch
    t = torch.bfloat16
    (x, sx), (w, sw), (u, su) = eight((N, c1), 61), eight((c2, c1), 62, c1 ** -0.5), eight((c2, c1), 63, c1 ** -0.5)
    b, r = rand((c2,), 64, t), rand((N, c2), 65, t)
    d = [v.cuda() for v in (x, sx, w, sw)]
    close(dyra.dyra_linear_quantized(*d, bias=b.cuda(), act="gelu", residual=r.cuda()), *on_gpu(linear_ref, x, sx, w, sw, b, "gelu", r, t))
    f = torch.float32
    close(dyra.dyra_linear_quantized(*d, out_dtype=f), *on_gpu(linear_ref, x, sx, w, sw, None, "none", None, f))
    close(dyra.dyra_gated_quantized(*d, u.cuda(), su.cuda(), bias_u=b.cuda()), *on_gpu(gated_ref, x, sx, w, sw, u, su, None, b, "silu", t))
    close(dyra.dyra_gated_quantized(*d, u.cuda(), su.cuda(), out_dtype=f), *on_gpu(gated_ref, x, sx, w, sw, u, su, None, None, "silu", f))
    if c1 > 16:   # a column slice: rows further apart than they are long
        k = c1 // 2 // 16 * 16
        y = dyra.dyra_linear_quantized(d[0][:, 16:16 + k], d[1], d[2][:, :k], d[3])
        close(y, *on_gpu(linear_ref, x[:, 16:16 + k], sx, w[:, :k], sw, None, "none", None, t))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 50, 200, 400, 3000])
def test_strided_products_and_untouched_gaps(N, out):
    import torch
    o, c1, c2 = types()[out], 272, 77 if N < 1000 else 2100
    (wx, sx), (ww, sw) = eight((N + 2, c1 + 80), 66), eight((c2, c1 + 32), 67, c1 ** -0.5)
    wide_r = rand((N, c2 + 5), 68, o).cuda()
    wx, ww, sx, sw = wx.cuda(), ww.cuda(), sx.cuda()[:N], sw.cuda()
    x, w, r = wx[:N, 32:32 + c1], ww[:, 16:16 + c1], wide_r[:, 3:3 + c2]
    base = torch.full((N + 3, c2 + 9), 7.0, dtype=o, device="cuda")
    y = base[:N, 4:4 + c2]
    dyra.dyra_linear_quantized(x, sx, w, sw, residual=r, act="relu", out_dtype=o, Y=y)
    close(y, *on_gpu(linear_ref, x, sx, w, sw, None, "relu", r, o))
    y.fill_(7.0)
    assert (base == 7).all()
    dyra.dyra_gated_quantized(x, sx, w, sw, w, sw, out_dtype=o, H=y)
    close(y, *on_gpu(gated_ref, x, sx, w, sw, w, sw, None, None, "silu", o))
    y.fill_(7.0)
    assert (base == 7).all()


@pytest.mark.parametrize("N", [1, 40, 300])
def test_product_residual_in_place_and_one_row_for_all(N):
    import torch
    (x, sx), (w, sw) = eight((N, 64), 71), eight((96, 64), 72)
    r = rand((N, 96), 73, torch.bfloat16)
    d = [v.cuda() for v in (x, sx, w, sw)]
    y = r.cuda()
    assert dyra.dyra_linear_quantized(*d, residual=y, Y=y) is y
    close(y, *linear_ref(x, sx, w, sw, None, "none", r, torch.bfloat16))
    y = dyra.dyra_linear_quantized(*d, residual=r[:1].cuda().expand(N, 96))
    close(y, *linear_ref(x, sx, w, sw, None, "none", r[:1].expand(N, 96), torch.bfloat16))


@pytest.mark.parametrize("N,c2", [(1, 40), (20, 40), (300, 9), (100, 300), (3000, 2100)])
def test_the_longest_rows_of_the_largest_values_are_exact(N, c2):
    """65536 products of -128 and -128: 2^30, a float32; and with signs that cancel all but one product."""
    import torch
    c1 = 65536
    x = torch.full((N, c1), -128, dtype=torch.int8, device="cuda")
    w = torch.full((c2, c1), -128, dtype=torch.int8, device="cuda")
    w[c2 // 2, ::2] = 127
    w[c2 // 2, 1] = 1
    sx, sw = torch.ones(N, device="cuda"), torch.ones(c2, device="cuda")
    y = dyra.dyra_linear_quantized(x, sx, w, sw, out_dtype=torch.float32)
    rest = [j for j in range(c2) if j != c2 // 2]
    assert (y[:, rest] == 2.0 ** 30).all()
    exact = -128 * (127 * 32768 - 128 * 32767 + 1)
    assert float(torch.tensor(exact, dtype=torch.float32)) == exact and (y[:, c2 // 2] == exact).all()


@pytest.mark.parametrize("N", [4, 40, 300, 3000])
def test_scales_of_zero_infinity_and_nan_stay_in_their_rows_and_features(N):
    import torch
    c2 = 90 if N < 1000 else 2100
    (x, sx), (w, sw) = eight((N, 80), 74), eight((c2, 80), 75)
    clean = dyra.dyra_linear_quantized(*(v.cuda() for v in (x, sx, w, sw)), act="silu")
    sx[1], sx[2], sx[3], sw[7], sw[8], sw[9] = 0.0, math.nan, math.inf, 0.0, math.nan, -1e-3
    y = dyra.dyra_linear_quantized(*(v.cuda() for v in (x, sx, w, sw)), act="silu")
    rows, cols = [i for i in range(N) if i not in (1, 2, 3)], [j for j in range(c2) if j not in (7, 8, 9)]
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
    assert y[2].isnan().all() and y[:, 8].isnan().all() and (y[1, cols] == 0).all() and (y[rows, 7] == 0).all()
    y, bound = linear_ref(x, sx, w, sw, None, "none", None, torch.bfloat16)
    got = dyra.dyra_linear_quantized(*(v.cuda() for v in (x, sx, w, sw)))
    close(got[rows, 9], y[rows, 9], bound[rows, 9])


@pytest.mark.parametrize("N", [2, 30, 2500])
def test_product_offsets_past_32_bits(N):
    """Rows 2^20 elements apart of X (where N is large) and W; residual and Y of 2^32 elements and more."""
    import torch
    t, ld = torch.bfloat16, 1 << 20
    c1, c2 = 144, 4300 if N < 100 else 40
    (x, sx), (w, sw) = eight((N, c1), 76), eight((c2, c1), 77, c1 ** -0.5)
    X, W = spread(N, c1, ld if N > 100 else c1, torch.int8), spread(c2, c1, ld if N < 100 else c1, torch.int8)
    X.copy_(x)
    W.copy_(w)
    step = (1 << 32) // (N - 1) // 8 * 8 + 8200
    r, y = spread(N, c2, step, t), spread(N, c2, step, t)
    r.copy_(rand((N, c2), 78, t))
    sx, sw = sx.cuda(), sw.cuda()
    dyra.dyra_linear_quantized(X, sx, W, sw, residual=r, act="relu", Y=y)
    close(y, *on_gpu(linear_ref, X, sx, W, sw, None, "relu", r, t))
    dyra.dyra_gated_quantized(X, sx, W, sw, W, sw, H=y)
    close(y, *on_gpu(gated_ref, X, sx, W, sw, W, sw, None, None, "silu", t))


# ------------------------------------------------------------------ together, streams, graphs

def layer_params(c=256, f=416, seed=81):
    """A gated MLP with its norm, weights in 8 bits by the library."""
    import torch
    t = torch.bfloat16
    p = {"w": rand((c,), seed, t).cuda()}
    for i, (n, shape) in enumerate((("g", (f, c)), ("u", (f, c)), ("d", (c, f)))):
        p[n] = dyra.dyra_quantize(rand(shape, seed + 1 + i, t, shape[1] ** -0.5).cuda())
    return p


def layer(x, r, p, stream=None):
    """norm with the residual, gate and up products, quantisation, down product onto the residual stream."""
    q, scales, s = dyra.dyra_norm_quantize(x, p["w"], EPS, residual=r, stream=stream)
    h = dyra.dyra_gated_quantized(q, scales, *p["g"], *p["u"], stream=stream)
    hq, hs = dyra.dyra_quantize(h, stream=stream)
    return q, scales, s, h, hq, hs, dyra.dyra_linear_quantized(hq, hs, *p["d"], residual=s, stream=stream)


@pytest.mark.parametrize("N", [1, 7, 64, 300, 5000])
def test_layer_of_all_operators(N):
    """Each step against its definition on the step's own inputs, and the whole against the layer in float64 on the
    weights' values: quantisation leaves out half a step of 1/127 of a row's largest value, twice."""
    import torch
    t = torch.bfloat16
    p = layer_params()
    x, r = rand((N, 256), 91, t), rand((N, 256), 92, t)
    q, scales, s, h, hq, hs, y = layer(x.cuda(), r.cuda(), p)
    z, ref = norm_ref(x, p["w"].cpu(), EPS, r)
    check_rows(q, scales, ref, True)
    check_sum(s, z)
    close(h, *on_gpu(gated_ref, q, scales, *p["g"], *p["u"], None, None, "silu", t))
    check_rows(hq, hs, h.double().cpu(), False)
    close(y, *on_gpu(linear_ref, hq, hs, *p["d"], None, "none", s, t))
    wide = {n: dyra.dyra_dequantize(*p[n], torch.float32).double().cpu() for n in "gud"}
    g = ref @ wide["g"].T
    whole = z + (g * torch.sigmoid(g) * (ref @ wide["u"].T)) @ wide["d"].T
    assert (y.double().cpu() - whole).norm() <= 0.03 * whole.norm()


def test_quantized_layer_beside_the_approximate_and_the_exact_product():
    """norm -> dyra_forward, the library's approximate product, and 8-bit rows dequantised into dyra_linear."""
    import numpy as np
    import torch

    import oracle as orc
    from structured_rank_matmul_amd import synth
    from gpu_util import check_parity
    from test_gpu_ffn import linear_ref as exact_ref
    B, n, c, F = 3, 70, 96, 128
    W = synth.random_weight(c, F, 71, p=0.6)
    plan = dyra.dyra_prepare(W, 24, 8, 0.0, "bf16", 0)
    x, r = rand((B * n, c), 93, torch.bfloat16), rand((B * n, c), 94, torch.bfloat16)
    h, _ = dyra.dyra_norm(x.cuda(), None, EPS, residual=r.cuda())
    y = dyra.dyra_forward(h, B, n, plan).double().cpu().numpy()
    ref = orc.inference(h.double().cpu().numpy(), B, n, orc.offline_preparation(W.astype(np.float64), 24, 8, 0.0))
    check_parity(y, ref, n, "bf16", "norm -> dyra_forward")
    plan.close()
    wd = dyra.dyra_dequantize(*dyra.dyra_quantize(torch.from_numpy(W.T.copy()).cuda()))
    close(dyra.dyra_linear(h, wd), *exact_ref(h.cpu(), wd.cpu(), None, "none", None, torch.bfloat16))


def test_two_streams_and_repeats_agree_bit_for_bit():
    import torch
    p = layer_params()
    a, b = [(rand((N, 256), 95 + N, torch.bfloat16).cuda(), rand((N, 256), 96 + N, torch.bfloat16).cuda()) for N in (20, 900)]
    ra, rb = layer(*a, p), layer(*b, p)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    s2.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got.append((layer(*a, p, s1), ra))
        got.append((layer(*b, p, s2), rb))
    filler = [torch.full((256, 256), 3.0, device="cuda", dtype=torch.bfloat16) for _ in range(8)]
    torch.cuda.synchronize()
    for g, r in got:
        assert all(torch.equal(u, v) for u, v in zip(g, r))
    del filler


@pytest.mark.parametrize("N", [1, 40, 600])
def test_captured_layer_replays_with_new_inputs(N):
    """Two graphs of the layer, replayed in turn with eager work between: every replay equals the eager result."""
    import torch
    p = layer_params()
    static = [(rand((N, 256), 101 + i, torch.bfloat16).cuda(), rand((N, 256), 103 + i, torch.bfloat16).cuda()) for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in static:
            layer(*x, p)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for x in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(*x, p) + (dyra.dyra_norm(x[0], p["w"]), dyra.dyra_dequantize(*p["d"])))
        graphs.append(g)
    for i in range(5):
        for k in range(2):
            for j in range(2):
                static[k][j].copy_(rand((N, 256), 110 + 4 * i + 2 * k + j, torch.bfloat16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for k in range(2):
            eager = layer(*static[k], p) + (dyra.dyra_norm(static[k][0], p["w"]), dyra.dyra_dequantize(*p["d"]))
            assert all(torch.equal(u, v) for u, v in zip(outs[k], eager)), f"replay {i} of graph {k}"


def test_binding_refuses_mismatched_tensors():
    import torch
    x, q = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    w, s, sw = torch.zeros(8, 64, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"), torch.ones(8, device="cuda")
    lin, gat = dyra.dyra_linear_quantized, dyra.dyra_gated_quantized
    bad = [lambda: lin(x, s, w, sw), lambda: lin(q, s, w.float(), sw), lambda: lin(q, sw, w, sw), lambda: lin(q, s, w, s),
           lambda: lin(q, s.double(), w, sw), lambda: lin(q, s.cpu(), w, sw), lambda: lin(q, s, w[:, :32], sw), lambda: lin(q, s, w.cpu(), sw),
           lambda: lin(q, s, w, sw, bias=torch.zeros(8, device="cuda")), lambda: lin(q, s, w, sw, act="swish"),
           lambda: lin(q, s, w, sw, residual=torch.zeros(4, 8, device="cuda")), lambda: lin(q, s, w, sw, out_dtype=torch.float16),
           lambda: lin(q, s, w, sw, out_dtype=torch.int8), lambda: lin(q.view(torch.uint8), s, w, sw), lambda: lin(q, s, w.view(torch.uint8), sw),
           lambda: lin(q, s, w, sw, Y=torch.zeros(4, 8, device="cuda")), lambda: lin(q.cpu(), s, w, sw), lambda: lin(q.t(), s, w, sw),
           lambda: lin(q, torch.ones(8, device="cuda")[::2], w, sw), lambda: lin(q, s, w, sw, workspace=torch.zeros(64)),
           lambda: gat(q, s, w, sw, w, sw, workspace=torch.zeros(64, device="cuda")[::2]),
           lambda: gat(q, s, w, sw, w[:4], sw), lambda: gat(q, s, w, sw, torch.zeros(8, 128, dtype=torch.int8, device="cuda")[:, :64], sw),
           lambda: gat(q, s, w, sw, w, s), lambda: gat(q, s, w, s, w, sw), lambda: gat(x, s, w, sw, w, sw),
           lambda: dyra.dyra_norm(q), lambda: dyra.dyra_norm(x.half()), lambda: dyra.dyra_norm(x, torch.ones(63, device="cuda")),
           lambda: dyra.dyra_norm(x, torch.ones(64, device="cuda", dtype=torch.bfloat16)), lambda: dyra.dyra_norm(x, residual=x.bfloat16()),
           lambda: dyra.dyra_norm(x, S=torch.empty_like(x)), lambda: dyra.dyra_norm(x, residual=x[:2]), lambda: dyra.dyra_norm(x[0]),
           lambda: dyra.dyra_norm(x.cpu()), lambda: dyra.dyra_norm(x, Y=x.bfloat16()), lambda: dyra.dyra_quantize(q),
           lambda: dyra.dyra_quantize(x, Q=torch.zeros(4, 64, device="cuda")), lambda: dyra.dyra_quantize(x, scales=sw),
           lambda: dyra.dyra_quantize(x, Q=torch.zeros(1, 64, dtype=torch.int8, device="cuda").expand(4, 64)),
           lambda: dyra.dyra_norm_quantize(x, Q=q.t()), lambda: dyra.dyra_dequantize(x, s), lambda: dyra.dyra_dequantize(q, sw),
           lambda: dyra.dyra_dequantize(q, s, torch.int8), lambda: dyra.dyra_dequantize(q, s, X=torch.zeros(4, 64, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    for call, status in ((lambda: lin(q[:, :56].contiguous(), s, w[:, :56].contiguous(), sw), 2), (lambda: dyra.dyra_norm(x, eps=0.0), 1),
                         (lambda: dyra.dyra_quantize(torch.zeros(1, 65537, device="cuda")), 2),
                         (lambda: lin(torch.zeros(4, 72, dtype=torch.int8, device="cuda")[:, 8:], s, w, sw), 4)):
        with pytest.raises(dyra.DyraError) as err:
            call()
        assert err.value.status == status


def test_more_rows_than_a_launch_has_threads_for():
    """2^24 rows and more of 256 threads each: several launches, of which the rows around the joins and the last are checked.
    The norm in place, so that its rows are read and written where a wrong offset would show."""
    import torch
    t, c = torch.bfloat16, 2056
    N, joins = (1 << 24) + 70, [1 << 23, 1 << 24]     # 2^31 / 256 rows a launch
    x = torch.empty(N, c, dtype=t, device="cuda")
    at = [slice(0, 20)] + [slice(j - 20, j + 20) for j in joins] + [slice(N - 20, N)]
    rows = [rand((x[s].shape[0], c), 120 + i, t) for i, s in enumerate(at)]
    for s, r in zip(at, rows):
        x[s] = r.cuda()
    w = rand((c,), 130, t)
    q, scales = dyra.dyra_quantize(x)
    for s, r in zip(at, rows):
        check_rows(q[s], scales[s], r.double(), False)
    out = dyra.dyra_norm(x, w.cuda(), EPS, Y=x)
    assert out is x
    for s, r in zip(at, rows):
        check_norm(x[s], norm_ref(r, w, EPS, None)[1], c)
    dyra.dyra_dequantize(q, scales, X=x)
    for s in at:
        v = q[s].cpu().double() * scales[s].cpu().double()[:, None]
        close(x[s], v, (U + half(t)) * v.abs() * 1.01)

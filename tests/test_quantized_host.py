"""CPU-side tests of the argument checks of the norm, the quantisation and the products of 8-bit integers: every refusal
is made on the host, before anything is enqueued.  Pointers are stand-in addresses; a refused call never reads them."""
import pytest

from structured_rank_matmul_amd import dyra

F32, BF16 = 0, 1
ARG, SHAPE, DTYPE, ALIGN = 1, 2, 3, 4
P = 4096   # 16-byte aligned stand-in addresses: multiples of it
NAN, INF = float("nan"), float("inf")


def norm(X=P, ldx=64, N=8, c=61, dtype=BF16, res=None, ldr=0, w=2 * P, eps=1e-5, S=None, lds=0, Y=3 * P, ldy=64):
    return dyra.load().dyra_norm(X, ldx, N, c, dtype, res, ldr, w, eps, S, lds, Y, ldy, None)


def norm_quantize(X=P, ldx=64, N=8, c=61, dtype=BF16, res=None, ldr=0, w=2 * P, eps=1e-5, S=None, lds=0, Q=3 * P, ldq=64,
                  scales=4 * P):
    return dyra.load().dyra_norm_quantize(X, ldx, N, c, dtype, res, ldr, w, eps, S, lds, Q, ldq, scales, None)


def quantize(X=P, ldx=64, N=8, c=61, dtype=BF16, Q=2 * P, ldq=64, scales=3 * P):
    return dyra.load().dyra_quantize(X, ldx, N, c, dtype, Q, ldq, scales, None)


def dequantize(Q=P, ldq=64, scales=2 * P, N=8, c=61, dtype=BF16, X=3 * P, ldx=64):
    return dyra.load().dyra_dequantize(Q, ldq, scales, N, c, dtype, X, ldx, None)


def linear(X=P, ldx=64, sx=2 * P, Wt=3 * P, ldw=64, sw=4 * P, N=8, c1=64, c2=48, bias=None, act=0, res=None, ldr=0, out=BF16,
           Y=5 * P, ldy=48, ws=None, size=0):
    return dyra.load().dyra_linear_quantized(X, ldx, sx, Wt, ldw, sw, N, c1, c2, bias, act, res, ldr, out, Y, ldy, ws, size, None)


def gated(X=P, ldx=64, sx=2 * P, Wg=3 * P, sg=4 * P, Wu=5 * P, su=6 * P, ldw=64, N=8, c1=64, c2=48, bg=None, bu=None, act=4,
          out=BF16, H=7 * P, ldh=48, ws=None, size=0):
    return dyra.load().dyra_gated_quantized(X, ldx, sx, Wg, sg, Wu, su, ldw, N, c1, c2, bg, bu, act, out, H, ldh, ws, size, None)


def test_empty_calls_are_no_ops():
    assert norm(N=0, X=None, Y=None) == 0
    assert norm_quantize(N=0, X=None, Q=None, scales=None) == 0
    assert quantize(N=0, X=None, Q=None, scales=None) == 0
    assert dequantize(N=0, Q=None, X=None, scales=None) == 0
    assert linear(N=0, X=None, sx=None, Y=None) == 0
    assert gated(N=0, X=None, sx=None, H=None) == 0


ROWS = [(DTYPE, dict(dtype=2)), (DTYPE, dict(dtype=-1)), (SHAPE, dict(N=-1)), (SHAPE, dict(c=0)), (SHAPE, dict(N=(1 << 25) + 1)),
        (SHAPE, dict(c=65537, ldx=65600, ldy=65600, ldq=65600)), (ARG, dict(ldx=60)), (ARG, dict(X=None))]
NORMS = ROWS + [(ARG, dict(eps=0.0)), (ARG, dict(eps=-1e-5)), (ARG, dict(eps=NAN)), (ARG, dict(eps=INF)), (ARG, dict(eps=1e-39)),
                (ARG, dict(res=5 * P, ldr=60)), (ARG, dict(res=5 * P, ldr=-1)), (ARG, dict(S=5 * P, lds=60)),
                (ALIGN, dict(X=P + 1)), (ALIGN, dict(w=P + 1)), (ALIGN, dict(res=P + 1, ldr=61)), (ALIGN, dict(S=P + 1, lds=61)),
                (ALIGN, dict(dtype=F32, X=P + 2)), (ARG, dict(S=2 * P, lds=61)), (ARG, dict(S=P, lds=64)),
                (ARG, dict(res=5 * P, ldr=64, S=5 * P, lds=61)), (ARG, dict(res=5 * P, ldr=0, S=5 * P, lds=61))]


@pytest.mark.parametrize("status,kw", NORMS + [(ARG, dict(ldy=60)), (ARG, dict(Y=None)), (ALIGN, dict(Y=P + 1)), (ARG, dict(Y=2 * P)),
                                               (ARG, dict(res=5 * P, ldr=64, Y=5 * P)), (ARG, dict(S=5 * P, lds=64, Y=5 * P)),
                                               (ARG, dict(Y=P, ldy=61))])
def test_norm_refuses(status, kw):
    kw.pop("ldq", None)
    assert norm(**kw) == status


@pytest.mark.parametrize("status,kw", NORMS + [(ARG, dict(ldq=60)), (ARG, dict(Q=None)), (ARG, dict(scales=None)), (ALIGN, dict(scales=P + 2)),
                                               (ARG, dict(Q=P)), (ARG, dict(Q=2 * P)), (ARG, dict(res=5 * P, ldr=64, Q=5 * P)),
                                               (ARG, dict(S=5 * P, lds=64, Q=5 * P)), (ARG, dict(Q=4 * P)), (ARG, dict(scales=P)),
                                               (ARG, dict(scales=2 * P)), (ARG, dict(res=5 * P, ldr=64, scales=5 * P)),
                                               (ARG, dict(S=5 * P, lds=64, scales=5 * P))])
def test_norm_quantize_refuses(status, kw):
    kw = {k: v for k, v in kw.items() if k != "ldy"}
    assert norm_quantize(**kw) == status


@pytest.mark.parametrize("status,kw", ROWS + [(ARG, dict(ldq=60)), (ARG, dict(Q=None)), (ARG, dict(scales=None)), (ALIGN, dict(scales=P + 2)),
                                              (ALIGN, dict(X=P + 1)), (ARG, dict(Q=P)), (ARG, dict(Q=3 * P)), (ARG, dict(scales=P))])
def test_quantize_refuses(status, kw):
    kw = {k: v for k, v in kw.items() if k != "ldy"}
    assert quantize(**kw) == status


@pytest.mark.parametrize("status,kw", [r for r in ROWS if "X" not in r[1]] + [
    (ARG, dict(ldq=60)), (ARG, dict(Q=None)), (ARG, dict(X=None)), (ARG, dict(scales=None)), (ALIGN, dict(scales=P + 2)),
    (ALIGN, dict(X=P + 1)), (ARG, dict(X=P)), (ARG, dict(X=2 * P))])
def test_dequantize_refuses(status, kw):
    kw = {k: v for k, v in kw.items() if k != "ldy"}
    assert dequantize(**kw) == status


PRODUCTS = [(DTYPE, dict(out=2)), (ARG, dict(act=5)), (ARG, dict(act=-1)), (SHAPE, dict(N=-1)), (SHAPE, dict(c1=0)), (SHAPE, dict(c2=0)),
            (SHAPE, dict(N=(1 << 25) + 1)), (SHAPE, dict(c2=(1 << 25) + 1)), (SHAPE, dict(c1=56)), (SHAPE, dict(c1=65552, ldx=65552, ldw=65552)),
            (SHAPE, dict(ldx=(1 << 20) + 16)), (SHAPE, dict(ldw=(1 << 20) + 16)), (ARG, dict(ldx=48)), (ARG, dict(ldw=48)),
            (ALIGN, dict(ldx=72)), (ALIGN, dict(ldw=72)), (ARG, dict(X=None)), (ARG, dict(sx=None)), (ALIGN, dict(X=P + 8)),
            (ALIGN, dict(sx=P + 2)), (ALIGN, dict(ws=P + 8, size=1 << 20))]


@pytest.mark.parametrize("status,kw", PRODUCTS + [
    (ARG, dict(ldy=47)), (ARG, dict(Wt=None)), (ARG, dict(sw=None)), (ARG, dict(Y=None)), (ALIGN, dict(Wt=P + 8)), (ALIGN, dict(sw=P + 1)),
    (ALIGN, dict(Y=P + 1)), (ALIGN, dict(out=F32, Y=P + 2)), (ALIGN, dict(bias=P + 1)), (ALIGN, dict(out=F32, bias=P + 2)),
    (ARG, dict(res=6 * P, ldr=47)), (ALIGN, dict(res=P + 1, ldr=48)), (ARG, dict(res=5 * P, ldr=56)), (ARG, dict(bias=5 * P))]
    + [(ARG, dict(Y=i * P)) for i in (1, 2, 3, 4)] + [(ARG, dict(ws=i * P, bias=6 * P, res=7 * P, ldr=48)) for i in range(1, 8)])
def test_linear_refuses(status, kw):
    assert linear(**kw) == status


@pytest.mark.parametrize("status,kw", PRODUCTS + [
    (ARG, dict(ldh=47)), (ARG, dict(H=None)), (ALIGN, dict(H=P + 1)), (ALIGN, dict(bg=P + 1)), (ALIGN, dict(bu=P + 1))]
    + [(ARG, {n: None}) for n in ("Wg", "sg", "Wu", "su")] + [(ALIGN, {n: P + 2}) for n in ("Wg", "sg", "Wu", "su")]
    + [(ARG, dict(H=i * P)) for i in (1, 2, 3, 4, 5, 6)] + [(ARG, dict(bg=7 * P)), (ARG, dict(bu=7 * P))]
    + [(ARG, dict(ws=i * P, bg=8 * P, bu=9 * P)) for i in range(1, 10)])
def test_gated_refuses(status, kw):
    assert gated(**kw) == status


@pytest.mark.parametrize("N,c1,c2", [(0, 14336, 64), (-1, 14336, 64), (64, 14328, 64), (64, 65552, 64), (64, 0, 64), (64, 14336, 0),
                                     ((1 << 25) + 1, 14336, 64), (64, 14336, (1 << 25) + 1), (16, 14336, 4096), (4096, 14336, 4096)])
def test_no_workspace_for_refused_sizes_and_where_none_is_used(N, c1, c2):
    for gated_ in (0, 1):
        assert dyra.load().dyra_quantized_workspace_bytes(N, c1, c2, gated_) == 0

"""CPU-side tests of the feed-forward calls' argument checks: every refusal is
made on the host, before anything is enqueued, so none needs a GPU.  Pointers
are stand-in addresses; a refused call never reads them."""
import pytest

from structured_rank_matmul_amd import dyra

F32, BF16 = 0, 1
ARG, SHAPE, DTYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 8
P = 4096   # a 16-byte aligned stand-in address


def linear(X=P, ldx=64, Wt=P, ldw=64, N=8, c1=64, c2=48, dtype=BF16, bias=None, act=0, res=None, ldr=0, out=BF16, Y=P,
           ldy=48):
    return dyra.load().dyra_linear(X, ldx, Wt, ldw, N, c1, c2, dtype, bias, act, res, ldr, out, Y, ldy, None)


def gated(X=P, ldx=64, Wg=P, Wu=P, ldw=64, N=8, c1=64, c2=48, dtype=BF16, bg=None, bu=None, act=4, H=P, ldh=48):
    return dyra.load().dyra_gated(X, ldx, Wg, Wu, ldw, N, c1, c2, dtype, bg, bu, act, H, ldh, None)


def route(logits=P, ld=16, T=4, experts=16, topk=2, dtype=F32, score=0, renorm=1, scale=1.0, ids=P, w=P):
    return dyra.load().dyra_route(logits, ld, T, experts, topk, dtype, score, renorm, scale, ids, w, None)


def moe(X=P, ldx=64, T=4, c=64, f=32, Wg=P, Wu=P, Wd=P, experts=8, ids=P, w=P, topk=2, dtype=BF16, act=4, res=None,
        ldr=0, Y=P, ldy=64, ws=P, nbytes=4 * 2 * 32 * 2):
    return dyra.load().dyra_moe(X, ldx, T, c, f, Wg, Wu, Wd, experts, ids, w, topk, dtype, act, res, ldr, Y, ldy, ws,
                                nbytes, None)


def test_empty_calls_are_no_ops():
    assert linear(N=0, X=None, Y=None) == 0
    assert gated(N=0, X=None, H=None) == 0
    assert route(T=0, logits=None, ids=None, w=None) == 0
    assert moe(T=0, X=None, Y=None, ws=None, nbytes=0) == 0


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dtype=2)), (DTYPE, dict(out=7)), (DTYPE, dict(dtype=F32, out=BF16)),
    (ARG, dict(act=5)), (ARG, dict(act=-1)),
    (SHAPE, dict(N=-1)), (SHAPE, dict(c1=0)), (SHAPE, dict(c2=0)), (SHAPE, dict(N=(1 << 30) + 1)),
    (SHAPE, dict(c1=60)), (SHAPE, dict(c1=62, dtype=F32, out=F32)),
    (ARG, dict(ldx=56)), (ARG, dict(ldw=56)), (ARG, dict(ldy=47)), (ARG, dict(res=P, ldr=47)), (ARG, dict(res=P, ldr=-1)),
    (ALIGN, dict(ldx=68)), (ALIGN, dict(ldw=68)),
    (ARG, dict(X=None)), (ARG, dict(Wt=None)), (ARG, dict(Y=None)),
    (ALIGN, dict(X=P + 8)), (ALIGN, dict(Wt=P + 2)), (ALIGN, dict(Y=P + 1)), (ALIGN, dict(bias=P + 1)),
    (ALIGN, dict(res=P + 1, ldr=48)), (ALIGN, dict(out=F32, Y=P + 2)),
])
def test_linear_refuses(status, kw):
    assert linear(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dtype=5)), (ARG, dict(act=9)), (SHAPE, dict(c1=4)), (SHAPE, dict(N=-3)), (SHAPE, dict(c2=-1)),
    (ARG, dict(ldx=8)), (ARG, dict(ldh=40)), (ALIGN, dict(ldw=66)), (ARG, dict(Wg=None)), (ARG, dict(Wu=None)),
    (ARG, dict(H=None)), (ALIGN, dict(Wu=P + 8)), (ALIGN, dict(bu=P + 1)), (ALIGN, dict(H=P + 1)),
])
def test_gated_refuses(status, kw):
    assert gated(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dtype=3)), (ARG, dict(score=2)), (ARG, dict(scale=float("nan"))), (ARG, dict(scale=float("inf"))),
    (SHAPE, dict(T=-1)), (SHAPE, dict(experts=0)), (SHAPE, dict(experts=1025, ld=1025)), (SHAPE, dict(topk=0)),
    (SHAPE, dict(topk=17)), (SHAPE, dict(experts=128, ld=128, topk=65)), (ARG, dict(ld=15)),
    (ARG, dict(logits=None)), (ARG, dict(ids=None)), (ARG, dict(w=None)), (ALIGN, dict(logits=P + 2)),
    (ALIGN, dict(ids=P + 2)), (ALIGN, dict(w=P + 1)),
])
def test_route_refuses(status, kw):
    assert route(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(dtype=4)), (ARG, dict(act=6)), (SHAPE, dict(T=-1)), (SHAPE, dict(c=60, ldx=64)), (SHAPE, dict(f=30)),
    (SHAPE, dict(f=0)), (SHAPE, dict(experts=0)), (SHAPE, dict(experts=1025)), (SHAPE, dict(topk=0)),
    (SHAPE, dict(topk=65)), (SHAPE, dict(T=513, topk=2)), (ARG, dict(ldx=56)), (ARG, dict(ldy=56)),
    (ARG, dict(res=P, ldr=8)), (ALIGN, dict(ldx=68)), (ARG, dict(X=None)), (ARG, dict(Wg=None)), (ARG, dict(Wu=None)),
    (ARG, dict(Wd=None)), (ARG, dict(ids=None)), (ARG, dict(w=None)), (ARG, dict(Y=None)), (ALIGN, dict(Wd=P + 4)),
    (ALIGN, dict(X=P + 8)), (ALIGN, dict(ids=P + 1)), (ALIGN, dict(Y=P + 1)), (ALIGN, dict(res=P + 1, ldr=64)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(nbytes=4 * 2 * 32 * 2 - 1)), (ALIGN, dict(ws=P + 4)),
])
def test_moe_refuses(status, kw):
    assert moe(**kw) == status


def test_moe_workspace_bytes():
    assert dyra.dyra_moe_workspace_bytes(4, 2, 32, "bf16") == 4 * 2 * 32 * 2
    assert dyra.dyra_moe_workspace_bytes(128, 8, 1408, "f32") == 128 * 8 * 1408 * 4
    assert dyra.dyra_moe_workspace_bytes(0, 2, 32, "bf16") == 0
    assert dyra.dyra_moe_workspace_bytes(1024, 2, 32, "bf16") == 0   # more pairs than one call takes
    assert dyra.load().dyra_moe_workspace_bytes(4, 2, 32, 9) == 0


def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros(4, 64), torch.zeros(8, 64)
    with pytest.raises(ValueError):
        dyra.dyra_linear(x, w)
    with pytest.raises(ValueError):
        dyra.dyra_gated(x, w, w)
    with pytest.raises(ValueError):
        dyra.dyra_route(x, 2)
    with pytest.raises(ValueError):
        dyra.dyra_moe(x, torch.zeros(2, 16, 64), torch.zeros(2, 16, 64), torch.zeros(2, 64, 16),
                      torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1))


Q = 1 << 30   # addresses of their own
APART = dict(X=Q, Wt=2 * Q, Y=3 * Q)


@pytest.mark.parametrize("kw", [dict(Y=Q), dict(Y=2 * Q), dict(res=3 * Q, ldr=56), dict(res=3 * Q, ldr=0)])
def test_linear_refuses_an_output_over_another_input(kw):
    assert linear(**{**APART, **kw}) == ARG


def test_gated_and_experts_refuse_an_output_over_another_input():
    for h in (Q, 2 * Q, 3 * Q):
        assert gated(X=Q, Wg=2 * Q, Wu=3 * Q, H=h) == ARG
    apart = dict(X=Q, Wg=2 * Q, Wu=3 * Q, Wd=4 * Q, Y=5 * Q, ws=6 * Q)
    for kw in (dict(Y=2 * Q), dict(Y=3 * Q), dict(Y=4 * Q), dict(ws=5 * Q), dict(ws=Q), dict(res=5 * Q, ldr=72),
               dict(res=6 * Q, ldr=64)):
        assert moe(**{**apart, **kw}) == ARG


@pytest.mark.parametrize("kw", [dict(N=(1 << 25) + 1), dict(c2=(1 << 25) + 1, ldy=1 << 26), dict(c1=(1 << 20) + 8, ldx=1 << 21)])
def test_sizes_past_the_limits(kw):
    assert linear(**{**APART, **kw}) == SHAPE
    assert route(T=(1 << 25) + 1) == SHAPE

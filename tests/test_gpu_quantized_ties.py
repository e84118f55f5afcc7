"""Rows in 8 bits where a value lies in the middle of two whole numbers: it goes to the even one, as 127 x / max |x| rounds in
float64, where these halves are exact."""
import pytest

from structured_rank_matmul_amd import dyra
from test_gpu_ffn import rand, types, U

pytestmark = pytest.mark.gpu


def halves(dtype, c=520):
    """Rows whose largest value has every mantissa of bf16, at several exponents, and every other value +-half of it, or, in
    the last rows, 127 with all of k + 1/2 up to 126.5.  Signs and the rest are random."""
    import torch
    g = torch.Generator().manual_seed(7)
    a = torch.cat([torch.arange(128, 256, dtype=torch.float32) * 2.0 ** e for e in (-140 if dtype == torch.float32 else -120, -30, -7, 20, 100, 119)])
    x = (torch.rand(len(a) + 6, c, generator=g) * 2 - 1).to(torch.bfloat16).float()
    x[: len(a)] *= a[:, None] * 0.99
    x[: len(a), ::2] = a[:, None] / 2
    x[: len(a), 4] = a
    for i in range(6):
        row = x[len(a) + i]
        row *= 100
        row[1:255:2], row[0] = torch.arange(127) + 0.5, 127.0
        row *= 2.0 ** (-60 + 20 * i)
    x *= torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)
    return x.to(dtype)


def check(q, scales, x):
    import torch
    a = x.double().abs().amax(dim=1)
    assert torch.equal(scales.cpu(), (a.float().clamp(min=127 * 2.0 ** -126) / 127))
    ref = 127 * x.double() / a[:, None].clamp(min=127 * 2.0 ** -126)
    off = q.cpu().double() != ref.round()
    if x.dtype == torch.float32:   # other values next to a middle may go to either neighbour
        off &= (ref - ref.floor() == 0.5) | ((ref - ref.floor() - 0.5).abs() > 127 * 4 * U)
    assert not off.any(), (int(off.sum()), ref[off][:4], q.cpu()[off][:4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_halves_go_to_the_even_number(dtype):
    x = halves(types()[dtype])
    check(*dyra.dyra_quantize(x.cuda()), x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
def test_halves_of_a_norm_go_to_the_even_number(dtype, weighted):
    """The ratio of two values of a row does not depend on its norm; weights are powers of two."""
    import torch
    x = halves(types()[dtype])
    w = torch.where(torch.arange(x.shape[1]) % 3 == 0, 2.0, 0.5).to(x.dtype) if weighted else None
    y = x if w is None else x.float() * w.float()
    fine = (y.abs().amax(dim=1) < 2.0 ** 126) & (y.abs().amax(dim=1) > 2.0 ** -100)
    q, scales = dyra.dyra_norm_quantize(x.cuda(), None if w is None else w.cuda(), 2.0 ** -126)
    a = y.double().abs().amax(dim=1, keepdim=True)
    ref = 127 * y.double() / a
    # rows whose norm is below eps's, and lie where scales begin, are left to the bounds of the other tests
    at = scales.cpu() > 2.0 ** -126
    assert at[fine].all()
    off = q.cpu().double() != ref.round()
    if x.dtype == torch.float32:
        off &= (ref - ref.floor() == 0.5) | ((ref - ref.floor() - 0.5).abs() > 127 * 4 * U)
    assert not off[fine].any(), (int(off[fine].sum()), ref[fine][off[fine]][:4], q.cpu()[fine][off[fine]][:4])


def test_random_rows_equal_the_definition():
    """bf16 rows of a gated pair.  With mantissas of 8 bits, x = m 2^-j and a = n of one unit, 127 x / a = 254 m 2^-j / (2 n)
    lies 2^-j / 510 at least from a middle that it does not hit; it is at most 253 2^-j, and the kernel's is right to
    2^-24 of that, 2^-16 2^-j: every value rounds as the exact ratio does."""
    import torch
    g, u = (rand((300, 14336), s, torch.float32) for s in (1, 2))
    x = (u * g * torch.sigmoid(g)).bfloat16()
    q, _ = dyra.dyra_quantize(x.cuda())
    ref = (127 * x.double() / x.double().abs().amax(dim=1, keepdim=True)).round()
    assert torch.equal(q.cpu().double(), ref), int((q.cpu().double() != ref).sum())

"""The binding of the 8-bit calls without a GPU: where the tensors' device is not the current one, a call is made again with
every argument in its place."""
import inspect

import pytest

from structured_rank_matmul_amd import dyra


class Matrix:
    """What the first lines of a call ask of a tensor."""
    shape, dtype = (4, 64), "int8"

    def dim(self):
        return 2

    def get_device(self):
        return 1

    def stride(self):
        return 64, 1


CALLS = [dyra.dyra_norm, dyra.dyra_norm_quantize, dyra.dyra_quantize, dyra.dyra_dequantize, dyra.dyra_linear_quantized,
         dyra.dyra_gated_quantized]


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_arguments_on_another_device(call, monkeypatch):
    again = []
    monkeypatch.setattr(dyra, "_stream_on", lambda dev, stream: None)
    monkeypatch.setattr(dyra, "_with_device", lambda dev, f, *a, **kw: again.append((dev, f, a, kw)) or "done")
    names = list(inspect.signature(call).parameters)
    given = {n: Matrix() if i == 0 else object() for i, n in enumerate(names)}
    assert call(**given) == "done"
    (dev, f, a, kw), = again
    assert dev == 1 and f is call
    assert inspect.signature(call).bind(*a, **kw).arguments == given

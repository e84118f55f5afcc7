"""Every kernel variant that some sizes of the products of 8-bit integers reach is reached by a case of
test_gpu_quantized_variants."""
import pytest

import test_gpu_quantized_variants as cases
from ffn_variants import Choice


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return Choice(str(tmp_path_factory.mktemp("choice")))


TOKENS = [1, 8, 16, 17, 32, 33, 64, 100, 128, 200, 256, 400, 700, 1000, 1024, 1500, 2048, 3000, 4096, 5000, 8000, 12000, 16384, 30000, 65536]
FEATURES = [1, 8, 16, 17, 30, 32, 33, 64, 100, 200, 400, 800, 1024, 1300, 2048, 2100, 3000, 4096, 4200, 6000, 8200, 12000, 20000]
BYTES = [16, 128, 512, 1024, 2048, 3008, 4096, 6144, 8192, 12288, 16384, 20480, 24576, 28672, 65536]


def kernel(choice, gated, N, c1, c2):
    L = choice.lib
    if N <= L.skinny_tokens():
        slabs, blocks = divmod(L.few(gated, N, c2, c1), 4)
        return ("registers", slabs, blocks) if slabs else ("ring", (N + 15) // 16)
    if L.narrow(1, gated, N, c2):
        return ("narrow", 2 if gated or c2 > 16 else 1)
    return ("tile", L.tile(1, gated, N, c2, c1))


@pytest.mark.parametrize("gated", [False, True])
def test_variants_are_tested(choice, gated):
    tested = {kernel(choice, gated, *s) for s in cases.shapes(gated)}
    reached = {kernel(choice, gated, N, b, c2) for N in TOKENS for c2 in FEATURES for b in BYTES}
    assert reached <= tested, sorted(reached - tested)
    assert len(reached) == 2 + 8 + (1 if gated else 2) + 8   # ring, registers, narrow, tiles

"""Every kernel variant that some sizes of the products of 8-bit integers reach is reached by a case of
test_gpu_quantized_variants."""
import pytest

import test_gpu_quantized_variants as cases
from quantized_variants import Choice
from structured_rank_matmul_amd import dyra


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return Choice(str(tmp_path_factory.mktemp("choice")))


TOKENS = [1, 8, 16, 17, 32, 33, 64, 100, 128, 200, 256, 400, 700, 1000, 1024, 1500, 2048, 3000, 4096, 5000, 8000, 12000, 16384, 30000, 65536]
FEATURES = [1, 8, 16, 17, 30, 32, 33, 64, 100, 200, 400, 800, 1024, 1300, 2048, 2100, 3000, 4096, 4200, 6000, 8200, 12000, 20000]
BYTES = [16, 128, 512, 1024, 2048, 3008, 4096, 6144, 8192, 12288, 16384, 20480, 24576, 28672, 65536]
SIZES = [(N, b, c2) for N in TOKENS for c2 in FEATURES for b in BYTES]


@pytest.mark.parametrize("gated", [False, True])
def test_variants_are_tested(choice, gated):
    tested = {choice.whole(gated, *s) for s in cases.shapes(gated)}
    reached = {choice.whole(gated, *s) for s in SIZES}
    assert reached <= tested, sorted(reached - tested)
    assert len(reached) == 2 + 8 + (1 if gated else 2) + 7   # ring, registers, narrow, tiles (224 x 256 is bf16's)


@pytest.mark.parametrize("gated", [False, True])
def test_splits_are_tested(choice, gated):
    split = {s: choice.parts(gated, *s) for s in SIZES}
    tested = {choice.parts(gated, *s)[1] for s in cases.SPLIT[gated] if choice.parts(gated, *s)[0] > 1}
    reached = {tile for parts, tile in split.values() if parts > 1}
    assert reached <= tested, sorted(reached - tested)
    assert {1, 2, 3} <= reached
    # the workspace is what the parts need, and never more than it says
    for (N, c1, c2), (parts, _) in split.items():
        size = choice.lib.split_size(gated, N, c2, parts)
        assert dyra.load().dyra_quantized_workspace_bytes(N, c1, c2, gated) == size
        assert size <= 64 << 20 and (size == 0) == (parts == 1) and parts <= 16

"""Every kernel variant that some sizes of the feed-forward calls reach is reached by a case of test_gpu_ffn_variants."""
import pytest

import test_gpu_ffn_variants as cases
from ffn_variants import Choice


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    return Choice(str(tmp_path_factory.mktemp("choice")))


TOKENS = [1, 8, 16, 17, 32, 33, 64, 100, 128, 200, 256, 400, 700, 1000, 1024, 1500, 2048, 3000, 4096, 5000, 8000, 12000, 16384, 30000, 65536]
FEATURES = [1, 8, 16, 17, 30, 32, 33, 64, 100, 200, 400, 800, 1024, 1300, 2048, 2100, 3000, 4096, 4200, 6000, 8200, 12000, 20000]
BYTES = [16, 128, 512, 1024, 2048, 3000 // 16 * 16, 4096, 6144, 8192, 12288, 16384, 20480, 24576, 28672, 65536]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_and_gated_variants_are_tested(choice, dtype, gated):
    tested = {choice.linear(gated, dtype, *s) for s in cases.shapes(dtype, gated)}
    size = 2 if dtype == "bf16" else 4
    reached = {choice.linear(gated, dtype, N, b // size, c2) for N in TOKENS for c2 in FEATURES for b in BYTES}
    assert reached <= tested, sorted(reached - tested)
    assert len(reached) == 2 + 8 + (1 if gated else 2) + (8 if dtype == "bf16" else 4)   # ring, registers, narrow, tiles


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expert_variants_are_tested(choice, dtype):
    size = 2 if dtype == "bf16" else 4

    def down(T, E, k, c, f):
        return {choice.moe_down(dtype, T, k, E, c, f, parts, rest) for _, parts, rest in cases.workspaces(dtype, T, k, f)}

    def up(c):
        slabs = choice.moe_up(dtype, c)
        return slabs, c * size > 1024 * slabs   # the second: tokens are loaded anew for every unit

    tested = set().union(*(down(*s) for s in cases.EXPERTS))
    reached = set().union(*(down(T, E, k, c, f) for T in (1, 4, 8, 9, 20, 40, 64, 130, 300, 1024) for k in (1, 2, 4, 8) if T * k <= 1024
                            for E in (1, 3, 8, 20, 60) for c in (8, 72, 264, 1024, 1032, 2048, 2056, 4096) for f in (8, 264, 1048, 3000, 5432, 14336)))
    assert reached <= tested, sorted(reached - tested)
    assert {v[:3] for v in reached} == {(r, s, x) for r in (8, 16) for s in (8, 16) for x in ((0, 1) if dtype == "bf16" else (0,))}
    tested, reached = {up(s[3]) for s in cases.EXPERTS}, {up(c) for c in range(8, 9000, 8)}
    assert reached <= tested, sorted(reached - tested)
    # a run of the second product that begins inside a slot: its sums go through the workgroup's `head`
    assert any(s[4] * size > 128 * 8 and choice.moe_down(dtype, s[0], s[2], s[1], s[3], s[4], 0, 0)[:2] == (16, 16) for s in cases.EXPERTS)

"""What the header says of the feed-forward calls' arguments, beyond the single refusals of test_ffn_host: outputs and
workspaces at the address of every other argument, and sizes that are refused have no workspace.  No GPU."""
import pytest

from structured_rank_matmul_amd import dyra
from test_ffn_host import ARG, BF16, F32, Q, SHAPE, gated, linear, moe, route

LINEAR = dict(X=Q, Wt=2 * Q, bias=3 * Q, Y=4 * Q)
GATED = dict(X=Q, Wg=2 * Q, Wu=3 * Q, bg=4 * Q, bu=5 * Q, H=6 * Q)
ROUTE = dict(logits=Q, ids=2 * Q, w=3 * Q)
MOE = dict(X=Q, Wg=2 * Q, Wu=3 * Q, Wd=4 * Q, ids=5 * Q, w=6 * Q, res=7 * Q, ldr=64, Y=8 * Q, ws=9 * Q)


@pytest.mark.parametrize("name", ["X", "Wt", "bias"])
def test_linear_output_over_an_input(name):
    assert linear(**{**LINEAR, "Y": LINEAR[name]}) == ARG


@pytest.mark.parametrize("name", ["X", "Wg", "Wu", "bg", "bu"])
def test_gated_output_over_an_input(name):
    assert gated(**{**GATED, "H": GATED[name]}) == ARG


@pytest.mark.parametrize("kw", [dict(ids=Q), dict(w=Q), dict(ids=3 * Q), dict(ids=Q, w=Q)])
def test_router_outputs_over_the_logits_and_each_other(kw):
    assert route(**{**ROUTE, **kw}) == ARG


@pytest.mark.parametrize("name", ["Wg", "Wu", "Wd", "ids", "w"])
def test_experts_output_over_an_input(name):
    assert moe(**{**MOE, "Y": MOE[name]}) == ARG


@pytest.mark.parametrize("name", ["X", "Wg", "Wu", "Wd", "ids", "w", "res", "Y"])
def test_experts_workspace_over_another_argument(name):
    assert moe(**{**MOE, "ws": MOE[name]}) == ARG


@pytest.mark.parametrize("topk,f,dtype", [(65, 32, BF16), (128, 32, F32), (2, 30, BF16), (2, 4, BF16), (2, 34, F32), (2, 0, F32),
                                          (2, (1 << 18) + 8, BF16), (0, 32, BF16)])
def test_no_workspace_for_refused_sizes(topk, f, dtype):
    assert dyra.load().dyra_moe_workspace_bytes(4, topk, f, dtype) == 0
    assert moe(topk=topk, f=f, dtype=dtype, nbytes=1 << 40) == SHAPE

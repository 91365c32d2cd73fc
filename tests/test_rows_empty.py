"""Tensors without elements overlap nothing, wherever they lie: an empty slice of a
buffer is inside it (no GPU: with no rows these calls have nothing to do)."""
import pytest

from split_bf16_gemm_gb300 import binding as bd
from test_fp8_grouped_contract import L, at  # noqa: F401
from test_rows_checks import norm


@pytest.mark.parametrize("args", [dict(y=at(2, 16)), dict(s=at(2, 64)), dict(mu=at(3, 32)), dict(rs=at(2, 112)), dict(x=at(2, 16), y=at(2, 32))],
                         ids=lambda a: "-".join(a))
def test_empty_outputs_inside_an_input(L, args):
    assert norm(L, M=0, **args) == bd.OK
    assert norm(L, M=1, **args) == bd.ERR_ALIAS


def test_empty_rows_inside_the_norms_weight(L):
    assert L.rmsnorm_fp8(at(0), None, at(1), None, None, at(1, 16), at(1, 32), 0, 64, 1e-5, bd.BF16, None) == bd.OK

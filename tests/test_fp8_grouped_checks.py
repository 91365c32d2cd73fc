"""What the checks of the 8-bit and grouped entry points refuse, and in which
order (no GPU: every call here fails its checks before any CUDA call)."""
import pytest

from split_bf16_gemm_gb300 import binding as bd
from test_fp8_grouped_contract import L, at, norm  # noqa: F401


@pytest.mark.parametrize("M", [1, 4])
def test_in_place_means_x_or_residual(L, M):
    # the weight has as many bytes as a single row
    assert norm(L, s=at(2), M=M) == bd.ERR_ALIAS
    assert norm(L, s=at(2), res=None, M=M) == bd.ERR_ALIAS
    assert norm(L, s=at(0, 16), M=M) == bd.ERR_ALIAS
    assert norm(L, s=at(1, 512), M=2) == bd.ERR_ALIAS        # the residual's second row and beyond
    # in place is for `sum` alone
    assert norm(L, y=at(0), M=M) == bd.ERR_ALIAS
    assert norm(L, s=at(4), y=at(4), M=M) == bd.ERR_ALIAS
    # x, whose memory the weight is too
    assert norm(L, x=at(2), s=at(2), M=1) == bd.ERR_ALIAS

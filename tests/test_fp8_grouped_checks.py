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


# Every kind of fault in one call, and then one fewer at a time: the order is
# shape, dtype, NULL, alignment, overlap, and eps last.
def grouped16(name):
    def call(L, a=at(0), b=at(1), offs=at(2), out=at(3), T=4, G=2, N=104, K=256, dt=bd.BF16, odt=bd.F32):
        return getattr(L, name)(a, b, offs, out, T, G, N, K, dt, odt, None)
    return call


def gfp8(L, a=at(0), sa=at(1), b=at(2), sb=at(3), offs=at(4), out=at(5), T=4, G=2, N=100, K=256, dt=bd.BF16):
    return L.gemm_grouped_fp8_bt(a, sa, b, sb, offs, out, T, G, N, K, dt, None)


ORDERS = {
    "rmsnorm_fp8": (norm, [(bd.ERR_SHAPE, dict(K=24)), (bd.ERR_DTYPE, dict(dt=9)), (bd.ERR_NULL, dict(w=None)),
                           (bd.ERR_ALIGN, dict(x=at(0, 4))), (bd.ERR_ALIAS, dict(q=at(1))),
                           (bd.ERR_CONFIG, dict(eps=-1.0))]),
    "gemm_grouped_fp8_bt": (gfp8, [(bd.ERR_SHAPE, dict(K=24)), (bd.ERR_DTYPE, dict(dt=9)), (bd.ERR_NULL, dict(offs=None)),
                                   (bd.ERR_ALIGN, dict(a=at(0, 4))), (bd.ERR_ALIAS, dict(out=at(3)))]),
    **{n: (grouped16(n), [(bd.ERR_SHAPE, dict(K=12)), (bd.ERR_DTYPE, dict(dt=bd.F32)), (bd.ERR_NULL, dict(offs=None)),
                          (bd.ERR_ALIGN, dict(a=at(0, 4))), (bd.ERR_ALIAS, dict(out=at(1)))])
       for n in ("gemm_grouped_bt", "gemm_grouped_kn", "gemm_grouped_dw")},
}


@pytest.mark.parametrize("name", ORDERS)
def test_order_of_the_checks(L, name):
    call, faults = ORDERS[name]
    for first in range(len(faults)):
        args = {k: v for _, f in reversed(faults[first:]) for k, v in f.items()}
        assert call(L, **args) == faults[first][0], args


def test_offsets_are_checked_with_the_other_tensors(L):
    for call in (gfp8, *(grouped16(n) for n in ("gemm_grouped_bt", "gemm_grouped_kn", "gemm_grouped_dw"))):
        # their alignment before another tensor's overlap
        bad = dict(out=at(1)) if call is not gfp8 else dict(out=at(2))
        assert call(L, offs=at(6, 2), **bad) == bd.ERR_ALIGN
        assert call(L, out=at(6), offs=at(6, 4)) == bd.ERR_ALIAS      # inside the output
        assert call(L, offs=at(6, 4), **bad) == bd.ERR_ALIAS          # four bytes suffice


def test_too_many_tiles_is_a_shape(L):
    # T / 32 tiles of rows for each 128 of N, and one more a run: 2^31 and more
    for call in (gfp8, grouped16("gemm_grouped_bt")):
        assert call(L, T=1 << 22, N=1 << 22, dt=9) == bd.ERR_SHAPE
    assert grouped16("gemm_grouped_dw")(L, G=1024, N=1 << 22, K=1 << 22, dt=9) == bd.ERR_SHAPE


def test_grouped_override_validation(L):
    for columns, splits in [(16, 0), (96, 1), (512, 1), (-32, 0), (0, 3), (64, 16), (0, -1)]:
        assert L.splitk_set_grouped_override(columns, splits) == bd.ERR_CONFIG
    for columns in (0, 32, 64, 128, 256):
        for splits in (0, 1, 2, 4, 8):
            assert L.splitk_set_grouped_override(columns, splits) == bd.OK
    assert L.splitk_set_grouped_override(0, 0) == bd.OK

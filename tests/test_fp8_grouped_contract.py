"""Refusals of the 8-bit and grouped entry points (no GPU): every call fails
its checks before any CUDA call, so the made-up addresses are never read."""
import pytest

import split_bf16_gemm_gb300 as sk
from split_bf16_gemm_gb300 import binding as bd

F32, F16, BF16 = bd.F32, bd.F16, bd.BF16
MAX = 1 << 22
SPACE = 1 << 40          # made-up addresses this far apart never overlap


def at(i, off=0):
    return (i + 1) * SPACE + off


@pytest.fixture(scope="module")
def L():
    sk.build()
    return sk.lib()


def norm(L, x=at(0), res=at(1), w=at(2), s=at(3), y=at(4), q=at(5), sc=at(6), M=4, K=256, eps=1e-6, dt=BF16):
    return L.rmsnorm_fp8(x, res, w, s, y, q, sc, M, K, eps, dt, None)


def quant(L, x=at(0), q=at(1), sc=at(2), M=4, K=256, dt=BF16):
    return L.fp8_quantize(x, q, sc, M, K, dt, None)


def prep(L, b=at(0), q=at(1), sc=at(2), G=2, N=100, K=256, dt=BF16):
    return L.fp8_prepare_bt(b, q, sc, G, N, K, dt, None)


def fp8(L, a=at(0), sa=at(1), b=at(2), sb=at(3), out=at(4), M=4, N=100, K=256, dt=BF16):
    return L.gemm_fp8_bt(a, sa, b, sb, out, M, N, K, dt, None)


def gfp8(L, a=at(0), sa=at(1), b=at(2), sb=at(3), offs=at(4), out=at(5), T=4, G=2, N=100, K=256, dt=BF16):
    return L.gemm_grouped_fp8_bt(a, sa, b, sb, offs, out, T, G, N, K, dt, None)


def grouped(name):
    def call(L, a=at(0), b=at(1), offs=at(2), out=at(3), T=4, G=2, N=104, K=256, dt=BF16, odt=F32):
        return getattr(L, name)(a, b, offs, out, T, G, N, K, dt, odt, None)
    return call


bt, kn, dw = (grouped("gemm_grouped_" + n) for n in ("bt", "kn", "dw"))

REFUSED = [
    # shapes
    (norm, dict(K=24), bd.ERR_SHAPE), (norm, dict(K=0), bd.ERR_SHAPE), (norm, dict(M=-1), bd.ERR_SHAPE),
    (norm, dict(M=MAX + 1), bd.ERR_SHAPE), (norm, dict(K=MAX + 16), bd.ERR_SHAPE),
    (quant, dict(K=8), bd.ERR_SHAPE), (prep, dict(N=0), bd.ERR_SHAPE), (prep, dict(G=1025), bd.ERR_SHAPE),
    (prep, dict(K=40), bd.ERR_SHAPE), (prep, dict(G=1024, N=MAX, K=MAX), bd.ERR_SHAPE),
    (fp8, dict(K=40), bd.ERR_SHAPE), (fp8, dict(N=0), bd.ERR_SHAPE), (fp8, dict(M=-1), bd.ERR_SHAPE),
    (gfp8, dict(G=0), bd.ERR_SHAPE), (gfp8, dict(G=1025), bd.ERR_SHAPE), (gfp8, dict(K=24), bd.ERR_SHAPE),
    (gfp8, dict(T=MAX + 1), bd.ERR_SHAPE),
    (bt, dict(K=12), bd.ERR_SHAPE), (kn, dict(N=100), bd.ERR_SHAPE), (dw, dict(N=100), bd.ERR_SHAPE),
    (dw, dict(K=12), bd.ERR_SHAPE), (dw, dict(T=-1), bd.ERR_SHAPE), (bt, dict(N=MAX + 8), bd.ERR_SHAPE),
    (dw, dict(G=1024, N=MAX, K=MAX), bd.ERR_SHAPE),
    # element types
    (norm, dict(dt=3), bd.ERR_DTYPE), (quant, dict(dt=-1), bd.ERR_DTYPE), (prep, dict(dt=7), bd.ERR_DTYPE),
    (fp8, dict(dt=3), bd.ERR_DTYPE), (gfp8, dict(dt=9), bd.ERR_DTYPE), (bt, dict(dt=F32), bd.ERR_DTYPE),
    (kn, dict(dt=F32), bd.ERR_DTYPE), (dw, dict(dt=F32), bd.ERR_DTYPE), (bt, dict(odt=4), bd.ERR_DTYPE),
    # NULL
    (norm, dict(x=None), bd.ERR_NULL), (norm, dict(w=None), bd.ERR_NULL), (norm, dict(q=None), bd.ERR_NULL),
    (norm, dict(sc=None), bd.ERR_NULL), (quant, dict(q=None), bd.ERR_NULL), (prep, dict(sc=None), bd.ERR_NULL),
    (fp8, dict(sa=None), bd.ERR_NULL), (fp8, dict(sb=None), bd.ERR_NULL), (fp8, dict(out=None), bd.ERR_NULL),
    (gfp8, dict(offs=None), bd.ERR_NULL), (bt, dict(offs=None), bd.ERR_NULL), (kn, dict(b=None), bd.ERR_NULL),
    (dw, dict(out=None), bd.ERR_NULL),
    # alignment
    (norm, dict(x=at(0, 8)), bd.ERR_ALIGN), (norm, dict(res=at(1, 2)), bd.ERR_ALIGN),
    (norm, dict(y=at(4, 4)), bd.ERR_ALIGN), (quant, dict(sc=at(2, 4)), bd.ERR_ALIGN),
    (fp8, dict(a=at(0, 1)), bd.ERR_ALIGN), (fp8, dict(sb=at(3, 8)), bd.ERR_ALIGN),
    (gfp8, dict(offs=at(4, 2)), bd.ERR_ALIGN), (bt, dict(out=at(3, 4)), bd.ERR_ALIGN),
    # overlap
    (norm, dict(q=at(0)), bd.ERR_ALIAS), (norm, dict(s=at(0, 16)), bd.ERR_ALIAS),
    (norm, dict(y=at(1)), bd.ERR_ALIAS), (norm, dict(y=at(5, 16)), bd.ERR_ALIAS),
    (norm, dict(s=at(4)), bd.ERR_ALIAS), (quant, dict(q=at(0, 16)), bd.ERR_ALIAS),
    (prep, dict(q=at(0)), bd.ERR_ALIAS), (fp8, dict(out=at(2, 16)), bd.ERR_ALIAS),
    (fp8, dict(out=at(1)), bd.ERR_ALIAS), (gfp8, dict(out=at(4)), bd.ERR_ALIAS), (bt, dict(out=at(2)), bd.ERR_ALIAS),
    (dw, dict(out=at(1, 32)), bd.ERR_ALIAS),
    # eps
    (norm, dict(eps=-1.0), bd.ERR_CONFIG), (norm, dict(eps=float("nan")), bd.ERR_CONFIG),
]


@pytest.mark.parametrize("call,args,status", REFUSED,
                         ids=[f"{i}-{c.__name__}-{'-'.join(a)}" for i, (c, a, _) in enumerate(REFUSED)])
def test_refused(L, call, args, status):
    assert call(L, **args) == status


def test_no_rows_is_no_work(L):
    # nothing to write: accepted without a launch (there is no device here)
    assert norm(L, M=0) == bd.OK
    assert quant(L, M=0) == bd.OK
    assert fp8(L, M=0) == bd.OK
    assert gfp8(L, T=0) == bd.OK
    assert bt(L, T=0) == bd.OK
    assert kn(L, T=0) == bd.OK
    # a tensor without elements may have no address; the weights still need one
    assert gfp8(L, T=0, a=None, sa=None, out=None) == bd.OK
    assert norm(L, M=0, x=None, res=None, s=None, y=None, q=None, sc=None) == bd.OK
    assert fp8(L, M=0, b=None) == bd.ERR_NULL


def test_optional_and_in_place_arguments_pass_the_checks(L):
    # M = 0 stops after the checks; an extent of 0 bytes overlaps nothing, so
    # overlap is checked by the refusals above and on the GPU
    assert norm(L, res=None, s=None, y=None, M=0) == bd.OK
    assert norm(L, s=at(0), M=0) == bd.OK


def test_python_errors_carry_the_status(L):
    with pytest.raises(sk.SplitKError) as e:
        sk.gemm_fp8_bt(at(0), at(1), at(2), at(3), at(4), 4, 64, 24, "bf16", stream=0)
    assert e.value.status == bd.ERR_SHAPE

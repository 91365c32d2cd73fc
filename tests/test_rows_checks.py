"""Refusals of routing, sorted rows, layer norm and the gradient norm, and the
order of the checks (no GPU: every call fails its checks, or has nothing to do,
before any CUDA call, so the made-up addresses are never read)."""
import ctypes

import pytest

import split_bf16_gemm_gb300 as sk
from split_bf16_gemm_gb300 import binding as bd
from test_fp8_grouped_contract import L, at  # noqa: F401

F32, F16, BF16 = bd.F32, bd.F16, bd.BF16
MAX = 1 << 22


def route(L, l=at(0), e=at(1), s=at(2), M=4, G=16, top=2, only=0, dt=BF16):
    return L.moe_route(l, e, s, M, G, top, only, dt, None)


def route_grad(L, l=at(0), e=at(1), d=at(2), o=at(3), M=4, G=16, top=2, only=0, dt=BF16):
    return L.moe_route_grad(l, e, d, o, M, G, top, only, dt, None)


def sort(L, e=at(0), o=at(1), s=at(2), src=at(3), M=4, top=2, G=16):
    return L.moe_sort(e, o, s, src, M, top, G, None)


def send(L, e=at(0), x=at(1), o=at(2), s=at(3), src=at(4), r=at(5), M=4, top=2, G=16, K=64, dt=BF16):
    return L.moe_dispatch(e, x, o, s, src, r, M, top, G, K, dt, None)


def send8(L, e=at(0), x=at(1), sc=at(2), o=at(3), s=at(4), src=at(5), r=at(6), rs=at(7), M=4, top=2, G=16, K=64):
    return L.moe_dispatch_fp8(e, x, sc, o, s, src, r, rs, M, top, G, K, None)


def back(L, r=at(0), s=at(1), w=at(2), o=at(3), M=4, top=2, K=64, dt=BF16, odt=F32):
    return L.moe_combine(r, s, w, o, M, top, K, dt, odt, None)


def back_grad(L, d=at(0), r=at(1), s=at(2), w=at(3), dr=at(4), ds=at(5), M=4, top=2, K=64, dt=BF16):
    return L.moe_combine_grad(d, r, s, w, dr, ds, M, top, K, dt, None)


def norm(L, x=at(0), res=at(1), w=at(2), b=at(3), s=at(4), y=at(5), mu=at(6), rs=at(7), M=4, K=64, eps=1e-5, dt=BF16):
    return L.layernorm(x, res, w, b, s, y, mu, rs, M, K, eps, dt, None)


def norm_grad(L, dy=at(0), h=at(1), w=at(2), mu=at(3), rs=at(4), ds=at(5), dx=at(6), dw=at(7), db=at(8), ws=at(9), nb=1 << 20, M=4,
              K=64, dt=BF16):
    return L.layernorm_grad(dy, h, w, mu, rs, ds, dx, dw, db, ws, nb, M, K, dt, None)


def tensors(addresses, sizes, dtypes):
    n = len(sizes)
    return (ctypes.c_void_p * n)(*addresses), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*dtypes)


def total(L, g=(at(0), at(1)), n=(8, 9), dt=(F32, BF16), count=2, norm=at(4), ws=at(5), nb=1 << 20):
    p, s, d = tensors(g, n, dt)
    return L.grad_norm(p, s, d, count, norm, ws, nb, None)


def clip(L, g=(at(0), at(1)), out=(at(2), at(3)), n=(8, 9), dt=(F32, BF16), count=2, most=1.0, norm=at(4), ws=at(5), nb=1 << 20):
    p, s, d = tensors(g, n, dt)
    o = None if out is None else tensors(out, n, dt)[0]
    return L.grad_clip(p, o, s, d, count, most, norm, ws, nb, None)


SHAPE, DTYPE, NULL, ALIGN, ALIAS, WORK, CONFIG = (bd.ERR_SHAPE, bd.ERR_DTYPE, bd.ERR_NULL, bd.ERR_ALIGN, bd.ERR_ALIAS, bd.ERR_WORKSPACE,
                                                  bd.ERR_CONFIG)
REFUSED = [
    (route, dict(M=-1), SHAPE), (route, dict(M=MAX + 1, top=1), SHAPE), (route, dict(top=0), SHAPE), (route, dict(top=33, G=64), SHAPE),
    (route, dict(top=17), SHAPE), (route, dict(G=1025), SHAPE), (route, dict(M=MAX), SHAPE), (route, dict(dt=3), DTYPE),
    (route, dict(l=None), NULL), (route, dict(e=None), NULL), (route, dict(s=None), NULL), (route, dict(l=at(0, 8)), ALIGN),
    (route, dict(e=at(1, 2)), ALIGN), (route, dict(s=at(2, 4)), ALIGN), (route, dict(s=at(0, 16)), ALIAS), (route, dict(e=at(2)), ALIAS),
    (route, dict(only=2), CONFIG), (route, dict(only=-1), CONFIG),
    (route_grad, dict(top=0), SHAPE), (route_grad, dict(G=1), SHAPE), (route_grad, dict(dt=-1), DTYPE), (route_grad, dict(d=None), NULL),
    (route_grad, dict(o=None), NULL), (route_grad, dict(e=at(1, 1)), ALIGN), (route_grad, dict(o=at(0)), ALIAS),
    (route_grad, dict(o=at(1, 16)), ALIAS), (route_grad, dict(only=3), CONFIG),
    (sort, dict(M=-1), SHAPE), (sort, dict(top=33), SHAPE), (sort, dict(G=0), SHAPE), (sort, dict(G=1025), SHAPE), (sort, dict(M=MAX), SHAPE),
    (sort, dict(e=None), NULL), (sort, dict(o=None), NULL), (sort, dict(s=None), NULL), (sort, dict(s=at(2, 2)), ALIGN),
    (sort, dict(o=at(0, 4)), ALIAS), (sort, dict(src=at(2)), ALIAS), (sort, dict(s=at(1, 64)), ALIAS),
    (send, dict(K=12), SHAPE), (send, dict(K=0), SHAPE), (send, dict(K=MAX + 8), SHAPE), (send, dict(G=0), SHAPE), (send, dict(dt=4), DTYPE),
    (send, dict(x=None), NULL), (send, dict(r=None), NULL), (send, dict(x=at(1, 8)), ALIGN), (send, dict(r=at(1)), ALIAS),
    (send, dict(r=at(1, 496)), ALIAS), (send, dict(s=at(5, 16)), ALIAS),
    (send8, dict(K=24), SHAPE), (send8, dict(sc=None), NULL), (send8, dict(rs=None), NULL), (send8, dict(rs=at(7, 4)), ALIGN),
    (send8, dict(r=at(1)), ALIAS), (send8, dict(rs=at(2)), ALIAS),
    (back, dict(K=20), SHAPE), (back, dict(top=0), SHAPE), (back, dict(dt=5), DTYPE), (back, dict(odt=5), DTYPE), (back, dict(r=None), NULL),
    (back, dict(s=None), NULL), (back, dict(o=None), NULL), (back, dict(w=at(2, 8)), ALIGN), (back, dict(o=at(0, 16)), ALIAS),
    (back, dict(o=at(1)), ALIAS),
    (back_grad, dict(K=4), SHAPE), (back_grad, dict(dt=9), DTYPE), (back_grad, dict(dr=None, ds=None), NULL),
    (back_grad, dict(r=None), NULL), (back_grad, dict(d=None), NULL), (back_grad, dict(dr=at(4, 4)), ALIGN),
    (back_grad, dict(dr=at(0)), ALIAS), (back_grad, dict(dr=at(1, 16)), ALIAS), (back_grad, dict(ds=at(3)), ALIAS),
    (back_grad, dict(ds=at(4, 16)), ALIAS),
    (norm, dict(K=4), SHAPE), (norm, dict(M=MAX + 1), SHAPE), (norm, dict(dt=3), DTYPE), (norm, dict(w=None), NULL), (norm, dict(y=None), NULL),
    (norm, dict(b=at(3, 8)), ALIGN), (norm, dict(mu=at(6, 4)), ALIGN), (norm, dict(y=at(0)), ALIAS), (norm, dict(y=at(1)), ALIAS),
    (norm, dict(s=at(0, 16)), ALIAS), (norm, dict(s=at(2), M=1), ALIAS), (norm, dict(rs=at(6)), ALIAS), (norm, dict(s=at(5)), ALIAS),
    (norm, dict(eps=-1.0), CONFIG), (norm, dict(eps=float("nan")), CONFIG),
    (norm_grad, dict(K=4), SHAPE), (norm_grad, dict(M=-1), SHAPE), (norm_grad, dict(dt=3), DTYPE), (norm_grad, dict(h=None), NULL),
    (norm_grad, dict(mu=None), NULL), (norm_grad, dict(dw=None), NULL), (norm_grad, dict(ws=None), NULL), (norm_grad, dict(ws=at(9, 8)), ALIGN),
    (norm_grad, dict(dx=at(1)), ALIAS), (norm_grad, dict(dx=at(0, 16)), ALIAS), (norm_grad, dict(dw=at(2)), ALIAS),
    (norm_grad, dict(db=at(7)), ALIAS), (norm_grad, dict(ws=at(6)), ALIAS), (norm_grad, dict(nb=2 * 64 * 4 - 1), WORK),
    (total, dict(count=-1), SHAPE), (total, dict(count=65537), SHAPE), (total, dict(n=(8, -1)), SHAPE), (total, dict(n=(8, (1 << 34) + 1)), SHAPE),
    (total, dict(dt=(F32, 3)), DTYPE), (total, dict(g=(at(0), None)), NULL), (total, dict(norm=None), NULL), (total, dict(ws=None), NULL),
    (total, dict(g=(at(0), at(1, 8))), ALIGN), (total, dict(norm=at(4, 2)), ALIGN), (total, dict(norm=at(0, 4)), ALIAS),
    (total, dict(norm=at(5, 4)), ALIAS), (total, dict(ws=at(1)), ALIAS), (total, dict(nb=100), WORK),
    (clip, dict(out=(at(2), None)), NULL), (clip, dict(out=(at(2, 4), at(3))), ALIGN), (clip, dict(out=(at(2), at(2))), ALIAS),
    (clip, dict(out=(at(1), at(3))), ALIAS), (clip, dict(out=(at(0, 16), at(3))), ALIAS), (clip, dict(g=(at(0), at(0)), out=None), ALIAS),
    (clip, dict(out=None, norm=at(0)), ALIAS), (clip, dict(nb=1), WORK), (clip, dict(most=-1.0), CONFIG), (clip, dict(most=float("nan")), CONFIG),
    (clip, dict(most=float("inf")), CONFIG),
]


@pytest.mark.parametrize("call,args,status", REFUSED, ids=[f"{i}-{c.__name__}-{'-'.join(a)}" for i, (c, a, _) in enumerate(REFUSED)])
def test_refused(L, call, args, status):
    assert call(L, **args) == status


ORDERS = {
    "moe_route": (route, [(SHAPE, dict(top=0)), (DTYPE, dict(dt=9)), (NULL, dict(e=None)), (ALIGN, dict(l=at(0, 4))), (ALIAS, dict(s=at(0, 16))),
                          (CONFIG, dict(only=7))]),
    "moe_dispatch": (send, [(SHAPE, dict(K=9)), (DTYPE, dict(dt=9)), (NULL, dict(o=None)), (ALIGN, dict(x=at(1, 4))), (ALIAS, dict(r=at(3)))]),
    "moe_combine": (back, [(SHAPE, dict(K=9)), (DTYPE, dict(odt=9)), (NULL, dict(s=None)), (ALIGN, dict(w=at(2, 4))), (ALIAS, dict(o=at(0)))]),
    "moe_combine_grad": (back_grad, [(SHAPE, dict(K=9)), (DTYPE, dict(dt=9)), (NULL, dict(s=None)), (ALIGN, dict(w=at(3, 4))), (ALIAS, dict(dr=at(0)))]),
    "layernorm": (norm, [(SHAPE, dict(K=9)), (DTYPE, dict(dt=9)), (NULL, dict(w=None)), (ALIGN, dict(b=at(3, 4))), (ALIAS, dict(y=at(0))),
                         (CONFIG, dict(eps=-1.0))]),
    "layernorm_grad": (norm_grad, [(SHAPE, dict(K=9)), (DTYPE, dict(dt=9)), (NULL, dict(w=None)), (ALIGN, dict(h=at(1, 4))), (ALIAS, dict(dw=at(0))),
                                   (WORK, dict(nb=0))]),
    "grad_clip": (clip, [(SHAPE, dict(n=(8, -1))), (DTYPE, dict(dt=(9, F32))), (NULL, dict(norm=None)), (ALIGN, dict(g=(at(0, 4), at(1)))),
                         (ALIAS, dict(out=(at(2), at(5)))), (WORK, dict(nb=0)), (CONFIG, dict(most=-1.0))]),
}


@pytest.mark.parametrize("name", ORDERS)
def test_order_of_the_checks(L, name):
    call, faults = ORDERS[name]
    for first in range(len(faults)):
        args = {k: v for _, f in reversed(faults[first:]) for k, v in f.items()}
        assert call(L, **args) == faults[first][0], args


def test_no_tokens_is_no_work(L):
    assert route(L, M=0) == bd.OK and route(L, M=0, l=None, e=None, s=None) == bd.OK
    assert route_grad(L, M=0) == bd.OK
    assert back(L, M=0) == bd.OK and back(L, M=0, r=None, s=None, w=None, o=None) == bd.OK
    assert back_grad(L, M=0) == bd.OK
    assert norm(L, M=0) == bd.OK
    assert norm(L, M=0, w=None) == bd.ERR_NULL


def test_workspace_sizes(L):
    assert L.layernorm_grad_workspace_bytes(4, 12) == 0
    assert L.layernorm_grad_workspace_bytes(-1, 64) == 0
    assert 0 < L.layernorm_grad_workspace_bytes(4, 64) <= 4 * 2 * 64 * 4
    for M, K in ((100000, 64), (100000, 8192), (5, 1 << 20), (1 << 22, 1 << 22)):
        assert 0 < L.layernorm_grad_workspace_bytes(M, K) <= 512 * 2 * K * 4
    assert L.grad_norm_workspace_bytes() > 0


def test_gradients_of_a_list():
    torch = pytest.importorskip("torch")
    a, b = torch.zeros(3, 5), torch.zeros(0, dtype=torch.bfloat16)
    g = sk.grad_list([a, b])
    assert g.count == 2 and list(g.sizes) == [15, 0] and list(g.dtypes) == [F32, BF16] and g.pointers[0] == a.data_ptr()
    assert sk.grad_list(g) is g
    with pytest.raises(ValueError):
        sk.grad_list([a.t()])
    with pytest.raises(ValueError):
        sk.grad_clip([a], 1.0, None, None, 0, out=[b], stream=0)
    with pytest.raises(sk.SplitKError) as e:
        sk.moe_combine(at(0), at(1), at(2), at(3), 4, 2, 12, "bf16", "f32", stream=0)
    assert e.value.status == bd.ERR_SHAPE

"""Layer norm, its gradients, and the gradient norm, on the GPU against their
definitions in 64 bits.

Tolerances (U = 2^-24, half a step of F32).  Layer norm: a sum over a row adds at
most c = K / 256 + 64 terms one after another (a thread's own, then lanes and warps;
a thread adds K / 128 at most where K <= 1024, K / 512 in long rows), so the mean of
h - mean is within c U of the mean magnitude, 1 / sqrt of the variance within (c + 8) U,
and y = n w + b within U (c (|n| + mean |n|) |w| + |b|) times 2 for the products.
Gradients: the same sums; dweight and dbias add M / 148 rows in a block (M / 8 of
rows longer than 8192), then at most 304 parts."""
import math

import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402
from rows_reference import DT, U, within  # noqa: E402
from test_gpu_fp8_grouped import Guarded, gen, randn, sk  # noqa: E402,F401

pytestmark = pytest.mark.gpu
EPS = 1e-5


def row_terms(K):
    return K / 256 + 64


def forward(sk, x, res, w, b, dtype, eps=EPS, in_place=None, stats=True):
    """y, mean, rstd and the sum (None where it is not asked for)."""
    M, K = x.shape
    y = Guarded((M, K), DT[dtype])
    mean, rstd = (Guarded((M,), torch.float32) if stats else None for _ in range(2))
    own = Guarded((M, K), DT[dtype]) if res is not None and in_place is None else None
    total = in_place if own is None else own.data
    sk.layernorm(x, w, b, y.data, M, K, dtype, eps=eps, residual=res, sum_out=total, mean=mean and mean.data, rstd=rstd and rstd.data)
    for t in (y, mean, rstd, own):
        assert t is None or t.intact()
    return y.data, mean and mean.data, rstd and rstd.data, total


def check_forward(y, mean, rstd, h, w, b, dtype, eps=EPS):
    want, m, r, n = ref.layernorm(h, w, b, eps)
    c = row_terms(h.shape[1])
    bias = 0 if b is None else b.double().abs()
    within(y, want, 2 * U * (c * (n.abs() + n.abs().mean(1, keepdim=True)) * w.double().abs() + bias), dtype)
    if mean is not None:
        spread = (h.double() - m[:, None]).abs().mean(1)
        within(mean, m, 2 * U * (m.abs() + c * spread))
        within(rstd, r, (c + 8) * U * r)


ROWS = [(1, 8), (2, 16), (3, 72), (65, 264), (7, 1000), (5, 1024), (33, 1032), (4, 2048), (300, 2056), (9, 4096), (3, 4104), (2, 8192),
        (3, 8200), (2, 16384), (3, 16392), (2, 50008), (700, 256)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", ROWS)
def test_layernorm(sk, M, K, dtype):
    g = gen(M * 13 + K)
    x, res = (2 * randn(g, M, K) + 3).to(DT[dtype]), randn(g, M, K).to(DT[dtype])
    w, b = (1 + 0.3 * randn(g, K)).to(DT[dtype]), randn(g, K).to(DT[dtype])
    y, mean, rstd, _ = forward(sk, x, None, w, b, dtype)
    check_forward(y, mean, rstd, x, w, b, dtype)
    h = (x.float() + res.float()).to(DT[dtype])
    y, mean, rstd, total = forward(sk, x, res, w, None, dtype)
    assert torch.equal(total, h)
    check_forward(y, mean, rstd, h, w, None, dtype)
    # the sum in the place of x or of the residual; without the statistics
    for which in (0, 1):
        pair = [x.clone(), res.clone()]
        z, _, _, _ = forward(sk, *pair, w, None, dtype, in_place=pair[which], stats=False)
        assert torch.equal(pair[which], h) and torch.equal(z, y)
    # x itself as the sum, where there is no residual
    z, _, _, total = forward(sk, x, None, w, None, dtype, in_place=torch.empty_like(x))
    assert torch.equal(total, x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [64, 2048, 16392])
def test_large_offset_small_spread(sk, K, dtype):
    """Equal values give the bias, and values of 1000 with a spread of a part in 128
    their norm: the mean's own rounding does not reach y."""
    g = gen(K)
    w, b = (1 + 0.3 * randn(g, K)).to(DT[dtype]), randn(g, K).to(DT[dtype])
    x = torch.full((2, K), 1000.0, device="cuda").to(DT[dtype])
    y, _, _, _ = forward(sk, x, None, w, b, dtype)
    assert torch.equal(y, b.expand(2, K))
    x = (1000 + 8 * torch.randint(-1, 2, (4, K), device="cuda", generator=g)).to(DT[dtype])
    y, mean, rstd, _ = forward(sk, x, None, w, b, dtype)
    check_forward(y, mean, rstd, x, w, b, dtype)


@pytest.mark.parametrize("K", [64, 1000, 4096, 16392])
@pytest.mark.parametrize("size", [3e38, 1e30, 1e19, 1e-19, 1e-30, 1e-36])
def test_rows_of_any_size(sk, K, size):
    """Finite rows have their norm also where their squares, or their sum, leave F32's
    range (eps 0: the norm does not depend on the size)."""
    g = gen(K)
    x = torch.rand(3, K, device="cuda", generator=g).mul(0.8).add(0.2) * size
    x[1] *= torch.where(torch.rand(K, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    w, b = 1 + 0.3 * randn(g, K), randn(g, K)
    y, mean, rstd, _ = forward(sk, x, None, w, b, "f32", eps=0.0)
    want, m, r, n = ref.layernorm(x, w, b, 0.0)
    c = row_terms(K)
    # h - mean and its mean are rounded to 2^-149 at best
    steps = 2.0 ** -149 * r.double()[:, None]
    within(y, want, 2 * U * (c * (n.abs() + n.abs().mean(1, keepdim=True)) * w.double().abs() + b.double().abs()) + 4 * steps * w.double().abs())
    within(mean, m, 2 * U * (m.abs() + c / r))
    within(rstd, r, (c + 8) * U * r)
    dy = randn(g, 3, K)
    check_backward(sk, dy, x, w, mean, rstd, None, "f32", scale=True)


def test_rows_with_nan_and_infinity(sk):
    for K in (256, 16392):
        x = randn(gen(1), 4, K)
        x[1, 5], x[2, 7] = math.nan, math.inf
        w, b = torch.ones(K, device="cuda"), torch.zeros(K, device="cuda")
        y, mean, rstd, _ = forward(sk, x, None, w, b, "f32")
        assert y[1].isnan().all() and y[2].isnan().all()
        clean = randn(gen(1), 4, K)
        z, _, _, _ = forward(sk, clean, None, w, b, "f32")
        assert torch.equal(y[[0, 3]], z[[0, 3]])


def backward(sk, dy, h, w, mean, rstd, dsum, dtype, dx=None, bias=True):
    M, K = dy.shape
    out = Guarded((M, K), DT[dtype]) if dx is None else None
    dw, db = Guarded((K,), torch.float32), Guarded((K,), torch.float32) if bias else None
    nbytes = sk.layernorm_grad_workspace_bytes(M, K)
    ws = Guarded((nbytes,), torch.uint8)
    sk.layernorm_grad(dy, h, w, mean, rstd, out.data if out else dx, dw.data, db and db.data, ws.data, nbytes, M, K, dtype, dsum=dsum)
    for t in (out, dw, db, ws):
        assert t is None or t.intact()
    return out.data if out else dx, dw.data, db and db.data


def check_backward(sk, dy, h, w, mean, rstd, dsum, dtype, scale=False):
    M, K = dy.shape
    dx, dw, db = backward(sk, dy, h, w, mean, rstd, dsum, dtype)
    wx, ww, wb, size, sw, sb = ref.layernorm_grad(dy, h, w, mean, rstd, dsum)
    c, rows = row_terms(K), M / (148 if K <= 8192 else 8) + 304 + 8
    # rows at the ends of the range: rstd may be a subnormal number, 2 rstd and its products are rounded to 2^-149
    more = 4 * 2.0 ** -149 * (1 + dy.double().abs().amax()) * (1 + w.double().abs().amax()) * K if scale else 0.0
    within(dx, wx, (c + 16) * U * size + more, dtype)
    within(dw, ww, (rows + 4) * U * sw + more)
    within(db, wb, rows * U * sb)
    return dx, dw, db


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", ROWS + [(1500, 136), (2000, 1032), (309, 8192), (333, 512), (170, 12288), (150, 16392), (40, 400008),
                                        (40003, 72), (20001, 136), (9001, 264), (2503, 2056), (700, 5120), (321, 16384), (1 << 22, 8)])
def test_layernorm_grad(sk, M, K, dtype):
    g = gen(M * 17 + K)
    h, w = (2 * randn(g, M, K) + 0.5).to(DT[dtype]), (1 + 0.3 * randn(g, K)).to(DT[dtype])
    dy, dsum = randn(g, M, K).to(DT[dtype]), randn(g, M, K).to(DT[dtype])
    _, mean, rstd, _ = forward(sk, h, None, w, None, dtype)
    check_backward(sk, dy, h, w, mean, rstd, None, dtype)
    dx, dw, db = check_backward(sk, dy, h, w, mean, rstd, dsum, dtype)
    # in the place of either gradient, without the bias's, and the same bits again
    for which in (0, 1):
        pair = [dy.clone(), dsum.clone()]
        x2, w2, _ = backward(sk, pair[0], h, w, mean, rstd, pair[1], dtype, dx=pair[which], bias=False)
        assert torch.equal(x2, dx) and torch.equal(w2, dw)


def test_gradients_by_differences(sk):
    M, K = 3, 16
    g = gen(8)
    h, w, b, dy = randn(g, M, K), 1 + 0.3 * randn(g, K), randn(g, K), randn(g, M, K)
    _, mean, rstd, _ = forward(sk, h, None, w, b, "f32")
    dx, dw, db = backward(sk, dy, h, w, mean, rstd, None, "f32")
    D = dy.double().cpu()

    def loss(h, w, b):
        return (ref.layernorm(h, w, b, EPS)[0] * D).sum()

    H, W, B = h.double().cpu(), w.double().cpu(), b.double().cpu()
    # third derivatives: at most about 15 rstd^3 sum |g|, times 1e-10 / 6; F32 as above
    size = float((D * W).abs().sum()) * float(rstd.max()) ** 3
    for got, want in ((dx, ref.differences(lambda t: loss(t, W, B), H)), (dw, ref.differences(lambda t: loss(H, t, B), W)),
                      (db, ref.differences(lambda t: loss(H, W, t), B))):
        within(got, want, torch.full_like(want, 1e-8 * (1 + size) + 512 * U * (1 + size)))


def test_no_rows(sk):
    K = 264
    dw, db = Guarded((K,), torch.float32), Guarded((K,), torch.float32)
    w = torch.ones(K, device="cuda")
    assert sk.layernorm_grad_workspace_bytes(0, K) == 0
    sk.layernorm_grad(None, None, w, None, None, None, dw.data, db.data, None, 0, 0, K, "f32")
    assert dw.data.eq(0).all() and db.data.eq(0).all() and dw.intact() and db.intact()


def test_nan_stays_in_its_row_and_columns(sk):
    M, K = 400, 264
    g = gen(2)
    h, w, dy = randn(g, M, K), 1 + 0.1 * randn(g, K), randn(g, M, K)
    _, mean, rstd, _ = forward(sk, h, None, w, None, "f32")
    dx, dw, db = backward(sk, dy, h, w, mean, rstd, None, "f32")
    dy[7, 3] = math.nan
    x2, w2, b2 = backward(sk, dy, h, w, mean, rstd, None, "f32")
    keep = [i for i in range(M) if i != 7]
    assert x2[7].isnan().all() and torch.equal(x2[keep], dx[keep])
    cols = [i for i in range(K) if i != 3]
    assert w2[3].isnan() and b2[3].isnan() and torch.equal(w2[cols], dw[cols]) and torch.equal(b2[cols], db[cols])


# ------------------------------------------------------------------ the norm of all gradients
#
# A thread adds 32 squares (31 U, all of one sign) and the root halves it; the rest
# is in 64 bits.  The norm is rounded once more: within 18 U.  The factor takes one
# more rounding, and so does each product.

NORM = 18 * U


def gradients(g, sizes, names, scale=1.0):
    return [(randn(g, max(n, 1))[:n] * scale).to(DT[d]) for n, d in zip(sizes, names)]


def exact_norm(grads):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))


def check_clip(sk, grads, most):
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm, other = Guarded((nbytes,), torch.uint8), Guarded((1,), torch.float32), Guarded((1,), torch.float32)
    out = [Guarded(tuple(t.shape), t.dtype) for t in grads]
    kept = [t.clone() for t in grads]
    want = exact_norm(grads)
    sk.grad_norm(grads, norm.data, ws.data, nbytes)
    within(norm.data, torch.tensor([want]), torch.tensor([NORM * want]))
    sk.grad_clip(grads, most, other.data, ws.data, nbytes, out=[o.data for o in out])
    assert torch.equal(norm.data, other.data)
    f = min(1.0, most / want) if want else 1.0
    for t, k, o in zip(grads, kept, out):
        name = next(n for n, d in DT.items() if d == t.dtype)
        assert torch.equal(t, k)
        within(o.data, t.double() * f, (NORM + 2 * U) * f * t.double().abs(), name)
        assert o.intact()
    assert norm.intact() and other.intact() and ws.intact()
    sk.grad_clip(grads, most, other.data, ws.data, nbytes)               # in place
    for t, o in zip(grads, out):
        assert torch.equal(t, o.data)
    return want


def test_some_in_place(sk):
    g = gen(11)
    grads = gradients(g, [5000, 33, 70000], ["f32", "bf16", "f16"])
    kept, want = [t.clone() for t in grads], exact_norm(grads)
    other = [torch.empty_like(t) for t in grads]
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    sk.grad_clip(grads, want / 4, norm, ws, nbytes, out=[grads[0], other[1], grads[2]])
    for got, k, name in ((grads[0], kept[0], "f32"), (other[1], kept[1], "bf16"), (grads[2], kept[2], "f16")):
        within(got, k.double() / 4, (NORM + 2 * U) * k.double().abs() / 4, name)
    assert torch.equal(grads[1], kept[1])
    sk.grad_clip([grads[0], other[1]], 1e9, norm, ws, nbytes, out=[grads[0], other[0][:33].bfloat16()])   # a factor of 1, one in place


SETS = [[1], [8], [7, 0, 1], [8191, 8192, 8193], [3] * 40, [100003], [1 << 20, 5, 1 << 18, 77], [129] * 600, [1 + 37 * i % 999 for i in range(1100)]]


@pytest.mark.parametrize("names", [("f32",), ("bf16",), ("f16",), ("bf16", "f32", "f16")], ids="-".join)
@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(sk, sizes, names):
    g = gen(sum(sizes))
    grads = gradients(g, sizes, [names[i % len(names)] for i in range(len(sizes))])
    check_clip(sk, [t.clone() for t in grads], 0.5)
    check_clip(sk, [t.clone() for t in grads], 1e9)                      # nothing to scale: the same bits
    check_clip(sk, [t.clone() for t in grads], 0.0)


@pytest.mark.parametrize("scale", [1e37, 1e25, 1e-25, 1e-40])
def test_gradients_of_any_size(sk, scale):
    """Squares beyond F32's range at either end; subnormal values are 2^-149 exact."""
    g = gen(3)
    grads = gradients(g, [5000, 33, 70001], ["f32", "bf16", "f32"], scale)
    grads = [t.clamp(-3e38, 3e38) for t in grads]
    want = check_clip(sk, [t.clone() for t in grads], scale)
    assert want > 0
    # one large value among small ones, and zeros
    mixed = [torch.full((9000,), 1e-30, device="cuda"), torch.zeros(100, device="cuda"), torch.full((3,), scale, device="cuda")]
    check_clip(sk, mixed, 1e-3 * scale)


def test_no_gradients_and_zeros(sk):
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.full((1,), 7.0, device="cuda")
    sk.grad_norm([], norm, ws, nbytes)
    assert norm.item() == 0.0
    zeros = [torch.zeros(1000, device="cuda"), torch.zeros(0, device="cuda")]
    norm.fill_(7)
    sk.grad_clip(zeros, 1.0, norm, ws, nbytes)
    assert norm.item() == 0.0 and zeros[0].eq(0).all()


def test_nan_and_infinite_gradients(sk):
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    for bad in (math.nan, math.inf):
        a, b = torch.ones(10000, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16)
        a[4321] = bad
        sk.grad_clip([a, b], 1.0, norm, ws, nbytes)
        if math.isnan(bad):
            assert norm.isnan() and a.isnan().all() and b.isnan().all()
        else:
            assert norm.isinf() and a[4321].isnan() and a[:4321].eq(0).all() and b.eq(0).all()


def test_many_launches_and_a_large_tensor(sk):
    """Over 512 tensors (several launches) with a tensor of more than 2^31 values."""
    big = torch.ones((1 << 31) + 12345, device="cuda", dtype=torch.float16)
    grads = [torch.full((i % 50,), 2.0, device="cuda") for i in range(700)] + [big] + [torch.full((100,), 3.0, device="cuda") for _ in range(400)]
    total = big.numel() + 4 * sum(i % 50 for i in range(700)) + 9 * 100 * 400
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    sk.grad_clip(grads, math.sqrt(total) / 2, norm, ws, nbytes)
    within(norm, torch.tensor([math.sqrt(total)]), torch.tensor([NORM * math.sqrt(total)]))
    # halves up to the factor's error: 20 U of it, far below half a step of F16
    assert big.eq(0.5).all() and (grads[-1] - 1.5).abs().max() < 1.5 * 20 * U and (grads[49] - 1).abs().max() < 20 * U


def test_captured_clip_and_shared_lists(sk):
    """Captured, replayed on new values; two calls that follow one another share a
    workspace; a tensor twice has its squares twice in the norm."""
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm, second = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    g = gen(6)
    grads = gradients(g, [5000, 3, 40000], ["f32", "f16", "bf16"])
    lst = sk.grad_list(grads)
    sk.grad_norm(lst, norm, ws, nbytes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sk.grad_clip(lst, 1.0, norm, ws, nbytes)
        sk.grad_norm(lst, second, ws, nbytes)
    for scale in (1.0, 5.0, 1e-3):
        new = gradients(g, [5000, 3, 40000], ["f32", "f16", "bf16"], scale)
        for t, n in zip(grads, new):
            t.copy_(n)
        graph.replay()
        want = exact_norm(new)
        within(norm, torch.tensor([want]), torch.tensor([NORM * want]))
        # the scaled tensors hold roundings of their own, half a step a value at most
        assert abs(second.item() - min(1.0, want)) < 2.0 ** -8 * min(1.0, want)
    a = randn(g, 1000)
    sk.grad_norm([a, a], norm, ws, nbytes)
    within(norm, torch.tensor([exact_norm([a, a])]), torch.tensor([NORM * exact_norm([a, a])]))

"""Layer norm of rows at the ends of F32's range, on the GPU against its definition in
64 bits.

Tolerances: those of the layer norm's other tests (U = 2^-24, c = K / 256 + 64 terms of
a sum one after another).  A row that is done again is multiplied by powers of two
alone, which round nothing where no square leaves F32's normal numbers."""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402
from rows_reference import DT, U, within  # noqa: E402
from test_gpu_fp8_grouped import Guarded, gen, randn, sk  # noqa: E402,F401
from test_gpu_layernorm import EPS, check_backward, check_forward, forward, row_terms  # noqa: E402

pytestmark = pytest.mark.gpu
# a row to a warp, to blocks of every size, and longer than any block's registers
LENGTHS = [64, 304, 1024, 2048, 4096, 8192, 16392, 50008]


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -90])
@pytest.mark.parametrize("size", [1e-11, 1e-12, 9e-13, 5e-13, 2e-13, 1e-14, 5e17, 1e18, 2e18])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", LENGTHS)
def test_variances_on_either_side_of_the_range(sk, K, dtype, size, eps):
    """Standard deviations about where the squares stop being taken as they are (2^-40 and
    2^60): of one sign, of both, and in a single value among zeros."""
    g = gen(K)
    x = torch.rand(4, K, device="cuda", generator=g).mul(0.8).add(0.2) * size
    x[1] *= torch.where(torch.rand(K, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    x[2:] = 0
    x[2, K // 3] = size * K ** 0.5
    x[3, K // 3] = -size
    x = x.to(DT[dtype])
    w, b = (1 + 0.3 * randn(g, K)).to(DT[dtype]), randn(g, K).to(DT[dtype])
    y, mean, rstd, _ = forward(sk, x, None, w, b, dtype, eps=eps)
    check_forward(y, mean, rstd, x, w, b, dtype, eps=eps)
    check_backward(sk, randn(g, 4, K).to(DT[dtype]), x, w, mean, rstd, None, dtype)


def equal_rows(sk, x, w, b, dtype, value, eps=EPS):
    """Rows of equal values: n = 0, so y is the bias and rstd 1 / sqrt(eps).  Where the
    values are taken less their mean as it came out, that is off by at most the root of the
    variance (else the row is done again), and what its own rounding leaves in y is below
    c U of that, and in the variance the same part of it."""
    K = x.shape[1]
    c, v = row_terms(K), torch.full((x.shape[0],), value, dtype=torch.float64, device="cuda")
    y, mean, rstd, _ = forward(sk, x, None, w, b, dtype, eps=eps)
    bias = (b.double() if b is not None else torch.zeros(K, dtype=torch.float64, device="cuda")).expand(*x.shape)
    within(y, bias, 2 * U * (c * w.double().abs() + bias.abs()), dtype)
    r = torch.full_like(v, float(torch.tensor(eps)) ** -0.5)
    within(mean, v, 2 * U * (v.abs() + c / r))
    within(rstd, r, (c + 8) * U * r)
    return mean, rstd


VALUES = [3e38, -1e36, 3e31, 1.7e20, 1234500032512000.0, 1e10, -1e6, 60000.0, 3.0, 1e-30, 3e-39]


@pytest.mark.parametrize("dtype,value", [(d, v) for d in ("f32", "bf16") for v in VALUES] + [("f16", 60000.0), ("f16", 3.0)])
@pytest.mark.parametrize("K", [8, 64, 392, 1000, 1968, 2048, 2256, 5120, 8200, 16392, 50008])
def test_equal_values_of_any_size(sk, K, dtype, value):
    """Also where their sum leaves F32's range, and where the mean's rounding, squared, is
    beyond eps."""
    g = gen(K)
    x = torch.full((3, K), value, device="cuda").to(DT[dtype])
    w, b = (1 + 0.3 * randn(g, K)).to(DT[dtype]), randn(g, K).to(DT[dtype])
    mean, rstd = equal_rows(sk, x, w, b, dtype, float(x[0, 0]))
    equal_rows(sk, x, w, None, dtype, float(x[0, 0]))
    check_backward(sk, randn(g, 3, K).to(DT[dtype]), x, w, mean, rstd, None, dtype)


@pytest.mark.parametrize("eps", [1e-38, 1e-30, 1e-12, 1.0, 1e5, 1e20, 1e38])
@pytest.mark.parametrize("value", [3e38, 1e36, 1e10, 1e-3, 1e-20, 1e-42])
@pytest.mark.parametrize("K", [64, 1000, 5120, 16392])
def test_equal_values_with_any_eps(sk, K, value, eps):
    g = gen(K)
    x = torch.full((2, K), value, device="cuda")
    equal_rows(sk, x, 1 + 0.3 * randn(g, K), randn(g, K), "f32", float(x[0, 0]), eps=eps)


@pytest.mark.parametrize("eps", [1e30, 1e36, 2e36, 1e38, 3.3e38])
@pytest.mark.parametrize("size", [1e-15, 1.0, 1e15, 1e19])
@pytest.mark.parametrize("K", [64, 2048, 16392])
def test_large_eps(sk, K, size, eps):
    """eps beyond the squares' range takes nothing from small values."""
    g = gen(K)
    x, w = size * randn(g, 3, K), 1 + 0.3 * randn(g, K)
    y, mean, rstd, _ = forward(sk, x, None, w, None, "f32", eps=eps)
    check_forward(y, mean, rstd, x, w, None, "f32", eps=eps)


@pytest.mark.parametrize("K", [64, 2048, 16392])
def test_equal_sums_of_any_size(sk, K):
    """The same where the values are sums that nothing keeps, and in the place of x."""
    g = gen(K)
    w, b = 1 + 0.3 * randn(g, K), randn(g, K)
    x, res = torch.full((2, K), 2e38, device="cuda"), torch.full((2, K), 1e38, device="cuda")
    y, z, total = (torch.full_like(x, float("nan")) for _ in range(3))
    sk.layernorm(x, w, b, y, 2, K, "f32", eps=EPS, residual=res)
    assert torch.equal(y, b.expand(2, K))
    h = x + res
    sk.layernorm(x, w, b, z, 2, K, "f32", eps=EPS, residual=res, sum_out=x)
    assert torch.equal(z, y) and torch.equal(x, h)
    sk.layernorm(x, w, b, total, 2, K, "f32", eps=EPS, sum_out=x)
    assert torch.equal(total, y) and torch.equal(x, h)


@pytest.mark.parametrize("value", [3e38, -1e36, 1.7e20, 1e10, 1e4])
@pytest.mark.parametrize("K", [64, 392, 1000, 2048, 5120, 16392])
def test_spread_of_a_few_steps(sk, K, value):
    """Values a few steps of F32 apart, a single one among equal values too: the differences
    from a mean that is right to a step are exact.  (Where they are taken from a mean that
    is off by the root of the variance at most, its rounding leaves c U of that in y.)"""
    g = gen(K)
    x = torch.full((4, K), value, device="cuda")
    bits = x.view(torch.int32)
    bits[:2] -= torch.randint(0, 4, (2, K), device="cuda", generator=g, dtype=torch.int32)
    bits[2, K // 2] -= 1
    bits[3, ::3] -= 1
    w, b = 1 + 0.3 * randn(g, K), randn(g, K)
    y, mean, rstd, _ = forward(sk, x, None, w, b, "f32")
    want, m, r, n = ref.layernorm(x, w, b, EPS)
    c = row_terms(K)
    within(y, want, 2 * U * (c * (1 + n.abs() + n.abs().mean(1, keepdim=True)) * w.double().abs() + b.double().abs()))
    within(mean, m, 2 * U * (m.abs() + c / r))
    within(rstd, r, (c + 8) * U * r)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", [(3, 72), (5, 1024), (4, 2048), (3, 8200), (2, 16392), (2, 50008)])
def test_the_input_in_its_own_place(sk, M, K, dtype):
    """`sum` without a residual receives x: as x itself, and elsewhere (guarded)."""
    g = gen(K)
    x, w = (2 * randn(g, M, K) + 3).to(DT[dtype]), (1 + 0.3 * randn(g, K)).to(DT[dtype])
    y, mean, rstd, _ = forward(sk, x, None, w, None, dtype)
    own, other = x.clone(), Guarded((M, K), DT[dtype])
    for place in (own, other.data):
        z, m, r, total = forward(sk, own, None, w, None, dtype, in_place=place)
        assert torch.equal(total, x) and torch.equal(z, y) and torch.equal(m, mean) and torch.equal(r, rstd)
    assert other.intact()

"""Layer norm of rows at the ends of F32's range, on the GPU against its definition in
64 bits.

Tolerances: those of the layer norm's other tests (U = 2^-24, c = K / 256 + 64 terms of
a sum one after another).  A row that is done again is multiplied by powers of two
alone, which round nothing where no square leaves F32's normal numbers."""
import pytest

torch = pytest.importorskip("torch")

from rows_reference import DT  # noqa: E402
from test_gpu_fp8_grouped import gen, randn, sk  # noqa: E402,F401
from test_gpu_layernorm import check_backward, check_forward, forward  # noqa: E402

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

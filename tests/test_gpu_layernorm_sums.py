"""The weight's and the bias's gradients within the roundings that their sums have.

U = 2^-24.  A row's n = (h - mean) rstd, of the mean and rstd as given, is rounded twice,
and each product joins its sum with one rounding.  Rows of up to 8192 values: a block takes
`side` rows side by side, so that a thread adds M / (parts side) rows, rounded up; then the
`side` sums are added, and the blocks' parts, an eighth of them one after another and the
eighths.  Longer rows stand alone.  (The parts' number is the workspace's.)"""
import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402
from rows_reference import DT, U, within  # noqa: E402
from test_gpu_fp8_grouped import gen, randn, sk  # noqa: E402,F401
from test_gpu_layernorm import backward, forward  # noqa: E402

pytestmark = pytest.mark.gpu


def roundings(parts, M, K):
    side = 1
    if K <= 8192:
        threads = (K // 8 + 1) // 2
        threads = 8 if threads <= 8 else 16 if threads <= 16 else (threads + 31) // 32 * 32
        side = 512 // threads
    rows = -(-M // (parts * side))
    return rows + side + -(-parts // 8) + 8


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 2048), (3, 264), (9, 1000), (150, 8), (151, 4096), (153, 5120), (1216, 1024), (4097, 264), (3000, 2056),
                                 (20001, 64), (7, 8200), (65, 16384), (129, 16392), (40, 400008)])
def test_weight_and_bias_gradients(sk, M, K, dtype):
    g = gen(M + K)
    h, w = (2 * randn(g, M, K) + 0.5).to(DT[dtype]), (1 + 0.3 * randn(g, K)).to(DT[dtype])
    dy = randn(g, M, K).to(DT[dtype])
    _, mean, rstd, _ = forward(sk, h, None, w, None, dtype)
    _, dw, db = backward(sk, dy, h, w, mean, rstd, None, dtype)
    _, ww, wb, _, sw, sb = ref.layernorm_grad(dy, h, w, mean, rstd, None)
    n = roundings(sk.layernorm_grad_workspace_bytes(M, K) // (8 * K), M, K)
    within(dw, ww, U * (n + 3) * sw)
    within(db, wb, U * n * sb)

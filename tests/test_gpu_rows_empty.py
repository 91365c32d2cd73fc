"""Calls without tokens whose empty tensors lie inside the other operands' buffers
(given as addresses: an empty slice of a torch tensor has none)."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_fp8_grouped import Guarded, sk  # noqa: E402,F401

pytestmark = pytest.mark.gpu
INT = torch.int32


def test_no_tokens_in_slices(sk):
    G, K, top = 8, 64, 2
    offsets = Guarded((G + 1,), INT)
    none = offsets.data.data_ptr() + 16
    sk.moe_sort(none, offsets.data, none, none, 0, top, G)
    assert offsets.data.eq(0).all() and offsets.intact()
    offsets.data.fill_(7)
    sk.moe_dispatch(none, none, offsets.data, none, None, none, 0, top, G, K, "f32")
    assert offsets.data.eq(0).all() and offsets.intact()


def test_no_rows_in_slices(sk):
    K = 264
    dw, db, w = Guarded((K,), torch.float32), Guarded((K,), torch.float32), torch.ones(K, device="cuda")
    rows = dw.data.data_ptr() + 32
    sk.layernorm_grad(rows, w.data_ptr() + 16, w, rows, rows, rows + 32, dw.data, db.data, None, 0, 0, K, "f32")
    assert dw.data.eq(0).all() and db.data.eq(0).all() and dw.intact() and db.intact()

"""The norm of as many gradients as a call takes, on the GPU against its exact value.

A thread adds at most 11 squares and sums in F32 one after another, then pairs of F32
numbers; a thread's number, a block's part and the sum of the parts are rounded once
each: 14 U (U = 2^-24), of which the root leaves half, and it and its power of two add
two.  The test's bound is twice that, whatever the number of launches."""
import math

import pytest

torch = pytest.importorskip("torch")

from rows_reference import U, within  # noqa: E402
from test_gpu_fp8_grouped import Guarded, sk  # noqa: E402,F401

pytestmark = pytest.mark.gpu
NORM = 18 * U
FIRST, MOST = 512, 65536   # tensors of the first launch, and of a call


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1, 33, 16384])
def test_small_parts_behind_large_ones(sk, size, dtype):
    """Each launch but the first adds 2^-24 of what is there."""
    large, small = torch.full((size,), 4096.0, device="cuda").to(dtype), torch.ones(size, device="cuda").to(dtype)
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm = Guarded((nbytes,), torch.uint8), Guarded((1,), torch.float32)
    for count in (FIRST + 1, 5 * FIRST, MOST):
        sk.grad_norm([large] * FIRST + [small] * (count - FIRST), norm.data, ws.data, nbytes)
        want = math.sqrt(size * (FIRST * 2 ** 24 + count - FIRST))
        within(norm.data, torch.tensor([want], dtype=torch.float64), torch.tensor([NORM * want], dtype=torch.float64))
        assert ws.intact() and norm.intact()


def test_the_most_tensors_clipped(sk):
    """65536 gradients of a few values each, in place and elsewhere, and twice the same bits."""
    flat = torch.zeros(MOST, 4, device="cuda")
    flat[:FIRST], flat[FIRST:] = 4096.0, 1.0
    out = torch.zeros_like(flat)
    sizes = [1 + i % 4 for i in range(MOST)]
    grads, outs = ([t[i, :n] for i, n in enumerate(sizes)] for t in (flat, out))
    there = torch.arange(4, device="cuda")[None] < torch.tensor(sizes, device="cuda")[:, None]
    want = math.sqrt(float(flat.double().square()[there].sum()))
    nbytes = sk.grad_norm_workspace_bytes()
    ws, norm, again = torch.empty(nbytes, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    kept = flat.clone()
    sk.grad_clip(grads, want / 4, norm, ws, nbytes, out=outs)
    within(norm, torch.tensor([want], dtype=torch.float64), torch.tensor([NORM * want], dtype=torch.float64))
    ref = torch.where(there, kept.double() / 4, 0.0)
    within(out, ref, (NORM + 2 * U) * ref)
    assert torch.equal(flat, kept)
    sk.grad_clip(grads, want / 4, again, ws, nbytes)
    assert torch.equal(norm, again) and torch.equal(torch.where(there, flat, 0.0), out)

"""A mixture-of-experts feed-forward block on libsplitk's 8-bit operators.

One block of a decoder, from the residual stream to what is added to it:

  residual addition + RMS norm -> 8 bits            rmsnorm_fp8
  router: the `top` best experts of each token      torch
  the tokens' rows sorted by expert                 torch
  gate and up projections, per expert               gemm_grouped_fp8_bt
  silu(gate) * up -> 8 bits                         torch, fp8_quantize
  down projection, per expert                       gemm_grouped_fp8_bt
  weighted sum of each token's experts              torch

Nothing waits for the GPU: the counts per expert stay on it.

    python examples/moe_block.py [--tokens 256] [--experts 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import split_bf16_gemm_gb300 as sk  # noqa: E402

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


class Experts:
    """Weights [experts, out, in] in 8 bits, prepared once."""

    def __init__(self, w):
        self.G, self.N, self.K = w.shape
        self.q = torch.empty(w.shape, dtype=E4M3, device=w.device)
        self.scales = torch.empty(self.G, blocks(self.N), blocks(self.K), device=w.device)
        sk.fp8_prepare_bt(w, self.q, self.scales, self.G, self.N, self.K, w.dtype)

    def __call__(self, q, scales, offsets):
        out = torch.empty(q.shape[0], self.N, dtype=torch.bfloat16, device=q.device)
        sk.gemm_grouped_fp8_bt(q, scales, self.q, self.scales, offsets, out, q.shape[0], self.G, self.N, self.K, "bf16")
        return out


class MoeBlock:
    def __init__(self, norm, router, gate_up, down, top):
        self.norm, self.router, self.top = norm, router, top
        self.gate_up, self.down = Experts(gate_up), Experts(down)

    def __call__(self, x, residual):
        """Returns the block's output and the new residual (written in place)."""
        M, K = x.shape
        G = self.gate_up.G
        q = torch.empty(M, K, dtype=E4M3, device=x.device)
        scales = torch.empty(M, blocks(K), device=x.device)
        y = torch.empty_like(x)
        sk.rmsnorm_fp8(x, self.norm, q, scales, M, K, x.dtype, residual=residual, sum_out=residual, y=y)

        share, expert = torch.topk(torch.softmax((y @ self.router).float(), -1), self.top)
        order = torch.argsort(expert.flatten(), stable=True)
        token = order // self.top
        counts = torch.zeros(G, dtype=torch.int32, device=x.device)
        counts.scatter_add_(0, expert.flatten(), torch.ones_like(expert.flatten(), dtype=torch.int32))
        offsets = torch.nn.functional.pad(torch.cumsum(counts, 0, dtype=torch.int32), (1, 0))

        gate, up = self.gate_up(q.view(torch.uint8)[token].view(E4M3), scales[token], offsets).chunk(2, -1)
        h = (torch.nn.functional.silu(gate.float()) * up.float()).bfloat16()
        hq = torch.empty(h.shape, dtype=E4M3, device=x.device)
        hs = torch.empty(h.shape[0], blocks(h.shape[1]), device=x.device)
        sk.fp8_quantize(h, hq, hs, h.shape[0], h.shape[1], h.dtype)
        out = self.down(hq, hs, offsets)
        return torch.zeros(M, K, device=x.device).index_add_(0, token, out.float() * share.flatten()[order, None]), residual


def plain(block, x, residual, gate_up, down):
    """The block in 32 bits, with the weights before their preparation."""
    h = (x.float() + residual.float()).to(x.dtype).float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * block.norm.float()
    share, expert = torch.topk(torch.softmax((y.to(x.dtype) @ block.router).float(), -1), block.top)
    out = torch.zeros_like(y)
    for e in range(gate_up.shape[0]):
        token, place = (expert == e).nonzero(as_tuple=True)
        gate, up = (y[token] @ gate_up[e].float().T).chunk(2, -1)
        out.index_add_(0, token, (torch.nn.functional.silu(gate) * up) @ down[e].float().T * share[token, place, None])
    return out


def main(tokens=256, experts=16, hidden=2048, inner=1024, top=2, seed=0):
    """Runs the block and returns its relative difference from 32 bits."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device=dev, generator=g) * scale).bfloat16()

    gate_up = randn(experts, 2 * inner, hidden, scale=hidden ** -0.5)
    down = randn(experts, hidden, inner, scale=inner ** -0.5)
    block = MoeBlock(1 + randn(hidden, scale=0.1), randn(hidden, experts, scale=hidden ** -0.5), gate_up, down, top)
    x, residual = randn(tokens, hidden), randn(tokens, hidden)
    want = plain(block, x, residual, gate_up, down)
    got, _ = block(x, residual)
    if sk.splitk_get_device_status() != 0:
        raise RuntimeError("a kernel's bounded wait ran out")
    return float((got - want).norm() / want.norm())


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--experts", type=int, default=16)
    a = p.parse_args()
    sk.build()
    print(f"difference from 32 bits: {main(a.tokens, a.experts):.3f} of the output's norm")

"""The definitions of routing, sorted rows, layer norm and the gradient norm in 64
bits, for the GPU tests; and the differences that their gradients are held to."""
import math

import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24                                                     # half a step of F32
HALF = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}            # half a step of the output's type, of |result|
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}   # half a step among its subnormals


def within(got, ref, tol, out="f32"):
    """Every value within tol of the reference (an error of the F32 result), and the
    rounding to the output's type."""
    got, ref, tol = (torch.as_tensor(t).double().cpu() for t in (got, ref, tol))
    tol = tol + HALF[out] * (ref.abs() + tol) + TINY[out]
    off = (got - ref).abs()
    bad = ~(off <= tol) & ~((got == ref) | (got.isnan() & ref.isnan()))
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[0].tolist(), float((off - tol)[bad].max()))


def route(logits, top, chosen_only):
    """experts, shares, p (the row's softmax) of logits in 64 bits (no NaN, no +inf)."""
    M, G = logits.shape
    l = logits.double()
    experts = torch.full((M, top), -1, dtype=torch.int64)
    shares = torch.zeros(M, top, dtype=torch.float64)
    p = torch.zeros(M, G, dtype=torch.float64)
    for m in range(M):
        row = l[m].tolist()
        order = sorted((g for g in range(G) if row[g] > -math.inf), key=lambda g: (-row[g], g))[:top]
        if not order:
            continue
        most = row[order[0]]
        among = order if chosen_only else [g for g in range(G) if row[g] > -math.inf]
        part = {g: math.exp(row[g] - most) for g in among}
        total = math.fsum(part.values())
        for g in among:
            p[m, g] = part[g] / total
        for j, g in enumerate(order):
            experts[m, j] = g
            shares[m, j] = part[g] / total
    return experts, shares, p


def route_grad(p, experts, d):
    """dlogits of the formula, with p the row's softmax."""
    G = p.shape[1]
    there = (experts >= 0) & (experts < G)
    at = torch.where(there, experts, 0)
    w = torch.where(there, p.gather(1, at), 0.0)
    both = torch.zeros_like(p).scatter_add(1, at, torch.where(there, d, 0.0))
    c = (w * d.double()).sum(1, keepdim=True)
    return p * (both - c)


def sort(experts, G):
    """offsets, slots, source of flat lists."""
    flat = experts.flatten().tolist()
    order = sorted((i for i, e in enumerate(flat) if 0 <= e < G), key=lambda i: (flat[i], i))
    slots, source, offsets = [-1] * len(flat), order + [-1] * (len(flat) - len(order)), [0] * (G + 1)
    for r, i in enumerate(order):
        slots[i] = r
    for i in order:
        offsets[flat[i] + 1] += 1
    for g in range(G):
        offsets[g + 1] += offsets[g]
    return offsets, slots, source


def combine(rows, slots, shares):
    """out and sum |shares rows| in 64 bits."""
    T, K = rows.shape
    there = (slots >= 0) & (slots < T)
    x = rows.double()[torch.where(there, slots, 0).long()]
    s = torch.ones(slots.shape, dtype=torch.float64, device=slots.device) if shares is None else shares.double()
    x = torch.where(there[..., None], x * s[..., None], 0.0)
    return x.sum(1), x.abs().sum(1)


def layernorm(h, w, b, eps):
    """y, mean, rstd, and n = (h - mean) rstd."""
    h = h.double()
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1 / (d.pow(2).mean(1) + eps).sqrt()
    n = d * rstd[:, None]
    y = n * w.double() + (0 if b is None else b.double())
    return y, mean, rstd, n


def layernorm_grad(dy, h, w, mean, rstd, dsum):
    """dx, dweight, dbias, and the magnitudes that their sums go through."""
    dy, h, w = dy.double(), h.double(), w.double()
    r = rstd.double()[:, None]
    n = (h - mean.double()[:, None]) * r
    g = dy * w
    dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    return dx, (dy * n).sum(0), dy.sum(0), size, (dy * n).abs().sum(0), dy.abs().sum(0)


def differences(f, x, step=1e-5):
    """The gradient of the scalar f at x (64 bits) by central differences."""
    x = x.double().clone()
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        kept = float(flat[i])
        flat[i] = kept + step
        up = float(f(x))
        flat[i] = kept - step
        out[i] = (up - float(f(x))) / (2 * step)
        flat[i] = kept
    return g

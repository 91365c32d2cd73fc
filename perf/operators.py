"""Cases for the 8-bit and grouped operators, and the same operators in elementary torch operations.

Five kinds of pass, named by a case's "op":

  norm     residual addition, root-mean-square norm, 8-bit output with a scale for each 128 values of a row
  fp8      out = A B^T, both in 8 bits; a scale for each 128 values of A's rows and each 128 x 128 block of B
  experts_fp8  the same product grouped by expert: A's rows lie in consecutive ragged runs, one run per weight of B
  experts  the grouped product on 16-bit operands
  train    the grouped product on 16-bit operands with the gradients of its activations and its weights

`own = False` computes them here in 32 bits; `own = True` calls this repository's library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128            # values that share a scale
E4M3_MAX = 448.0
SMALLEST_SCALE = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token's hidden state, the smallest call of a decoding step
        {"name": "norm_token", "op": "norm", "M": 1, "K": 2048, "dtype": "bf16", "residual": True, "y": False},
        # a ragged batch of prompts whose router also reads the norm in 16 bits
        {"name": "norm_ragged", "op": "norm", "M": 333, "K": 5120, "dtype": "f16", "residual": True, "y": True},
        # a long prompt
        {"name": "norm_prefill", "op": "norm", "M": 8192, "K": 8192, "dtype": "bf16", "residual": True, "y": False},
        # one token through a projection
        {"name": "fp8_token", "op": "fp8", "M": 1, "N": 1024, "K": 2048, "out": "bf16"},
        # the size of this repository's benchmark, with its F32 output
        {"name": "fp8_batch", "op": "fp8", "M": 256, "N": 1024, "K": 2048, "out": "f32"},
        # odd sizes, the last block of K only 16 wide
        {"name": "fp8_odd", "op": "fp8", "M": 1001, "N": 2107, "K": 5136, "out": "f16"},
        # a prompt through a feed-forward projection
        {"name": "fp8_prefill", "op": "fp8", "M": 4096, "N": 8192, "K": 4096, "out": "bf16"},
        # a decoding batch spread thinly over the experts, some of which get nothing
        {"name": "experts_fp8_decode", "op": "experts_fp8", "T": 64, "G": 32, "empty": 6, "N": 2048, "K": 4096, "out": "bf16"},
        # a prompt over a few experts
        {"name": "experts_fp8_prefill", "op": "experts_fp8", "T": 8192, "G": 16, "empty": 0, "N": 4096, "K": 2048, "out": "bf16"},
        # weights kept as [K, N], odd sizes
        {"name": "experts_ragged", "op": "experts", "T": 1003, "G": 24, "empty": 5, "N": 1000, "K": 1544, "dtype": "f16", "layout": "kn", "out": "f32"},
        # one training step of a small layer, and of a large one
        {"name": "train_small", "op": "train", "T": 512, "G": 8, "empty": 1, "N": 512, "K": 1024, "dtype": "bf16"},
        {"name": "train_large", "op": "train", "T": 8192, "G": 8, "empty": 0, "N": 2048, "K": 2048, "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number of steps between lo and hi, even over its logarithm; the one size that no case has is passed over."""
    v = step * max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "fp8", "fp8", "experts_fp8", "experts_fp8", "experts", "train"])
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 512, 8192, 16), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                "residual": rng.random() < 0.8, "y": rng.random() < 0.3}
    out = rng.choice(["bf16", "bf16", "f16", "f32"])
    while True:
        if op == "fp8":
            c = {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 8192), "K": _log(rng, 128, 8192, 16), "out": out}
            if c["M"] * c["N"] * c["K"] <= 4096 * 8192 * 4096:
                return c
            continue
        G = _log(rng, 2, 64)
        c = {"op": op, "T": _log(rng, 1, 8192), "G": G, "empty": rng.randrange(0, max(1, G // 4))}
        if op == "experts_fp8":
            c |= {"N": _log(rng, 128, 4096), "K": _log(rng, 256, 4096, 16), "out": out}
        elif op == "experts":
            c |= {"N": _log(rng, 128, 4096, 8), "K": _log(rng, 256, 4096, 8), "dtype": rng.choice(["bf16", "f16"]),
                  "layout": rng.choice(["nk", "kn"]), "out": rng.choice(["same", "f32"])}
            if c["out"] == "same":
                c["out"] = c["dtype"]
        else:
            c |= {"N": _log(rng, 128, 2048, 8), "K": _log(rng, 128, 2048, 8), "dtype": rng.choice(["bf16", "f16"])}
        if c["G"] * c["N"] * c["K"] <= 64 * 2048 * 2048 and c["T"] * c["N"] * c["K"] <= 8192 * 2048 * 2048:
            return c


def _blocks(k):
    return (k + BLOCK - 1) // BLOCK


def _quantized_rows(x):
    """Codes and scales of a matrix with a scale for each 128 values of a row (the last block of a row may be short)."""
    m, k = x.shape
    b = torch.nn.functional.pad(x.float(), (0, _blocks(k) * BLOCK - k)).view(m, -1, BLOCK)
    scales = (b.abs().amax(-1) / E4M3_MAX).clamp_min(SMALLEST_SCALE)
    q = (b / scales[..., None]).reshape(m, -1)[:, :k].contiguous().to(torch.float8_e4m3fn)
    return q, scales


def _quantized_weights(w):
    """Codes and scales of weights [G, N, K] with a scale for each 128 x 128 block."""
    g, n, k = w.shape
    b = torch.nn.functional.pad(w.float(), (0, _blocks(k) * BLOCK - k, 0, _blocks(n) * BLOCK - n))
    b = b.view(g, _blocks(n), BLOCK, _blocks(k), BLOCK)
    scales = (b.abs().amax((2, 4)) / E4M3_MAX).clamp_min(SMALLEST_SCALE)
    q = (b / scales[:, :, None, :, None]).reshape(g, _blocks(n) * BLOCK, -1)[:, :n, :k].contiguous()
    return q.to(torch.float8_e4m3fn), scales


def _counts(case, seed):
    """Rows of each expert: `empty` of them get none, the others at least one where the rows suffice, unevenly."""
    r = np.random.RandomState(seed % (1 << 32))
    T, G = case["T"], case["G"]
    active = min(T, G - case["empty"])
    p = np.exp(0.5 * r.standard_normal(active))
    some = 1 + r.multinomial(T - active, p / p.sum())
    counts = np.zeros(G, dtype=np.int64)
    counts[r.permutation(G)[:active]] = some
    return counts


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    def activations(m, k):  # a few channels are much larger than the others, as in a residual stream
        return normal(m, k) * torch.exp(0.7 * normal(1, k))

    def empty(shape, name):
        return torch.empty(shape, dtype=DTYPES[name], device=dev)

    s = dict(case)
    if case["op"] == "norm":
        M, K, dt = case["M"], case["K"], case["dtype"]
        s["x"] = activations(M, K).to(DTYPES[dt])
        s["residual_in"] = activations(M, K).to(DTYPES[dt]) if case["residual"] else None
        s["weight"] = (1 + 0.1 * normal(K)).to(DTYPES[dt])
        s["sum_out"] = empty((M, K), dt) if case["residual"] else None
        s["y_out"] = empty((M, K), dt) if case["y"] else None
        s["q_out"] = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
        s["scales_out"] = empty((M, _blocks(K)), "f32")
        return s
    K, N = case["K"], case["N"]
    if case["op"] == "fp8":
        s["a"], s["a_scales"] = _quantized_rows(activations(case["M"], K))
        b, b_scales = _quantized_weights(normal(1, N, K) / math.sqrt(K))
        s["b"], s["b_scales"] = b[0], b_scales[0]
        s["result"] = empty((case["M"], N), case["out"])
        return s
    T, G = case["T"], case["G"]
    counts = _counts(case, seed)
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
    s["most"] = int(counts.max())
    if case["op"] == "experts_fp8":
        s["a"], s["a_scales"] = _quantized_rows(activations(T, K))
        s["b"], s["b_scales"] = _quantized_weights(normal(G, N, K) / math.sqrt(K))
        s["result"] = empty((T, N), case["out"])
        return s
    dt = case["dtype"]
    s["a"] = activations(T, K).to(DTYPES[dt])
    if case["op"] == "experts":
        s["b"] = (normal(G, *((K, N) if case["layout"] == "kn" else (N, K))) / math.sqrt(K)).to(DTYPES[dt])
        s["result"] = empty((T, N), case["out"])
        return s
    s["b"] = (normal(G, N, K) / math.sqrt(K)).to(DTYPES[dt])
    s["d"] = (0.1 * normal(T, N)).to(DTYPES[dt])
    s["result"], s["da"], s["db"] = empty((T, N), dt), empty((T, K), dt), empty((G, N, K), "f32")
    return s


def _run_own(s):
    import split_bf16_gemm_gb300 as sk

    op = s["op"]
    if op == "norm":
        sk.rmsnorm_fp8(s["x"], s["weight"], s["q_out"], s["scales_out"], s["M"], s["K"], s["dtype"], eps=EPS,
                       residual=s["residual_in"], sum_out=s["sum_out"], y=s["y_out"])
        return {"q": s["q_out"], "scales": s["scales_out"], "sum": s["sum_out"], "y": s["y_out"]}
    N, K = s["N"], s["K"]
    if op == "fp8":
        sk.gemm_fp8_bt(s["a"], s["a_scales"], s["b"], s["b_scales"], s["result"], s["M"], N, K, s["out"])
        return {"out": s["result"]}
    T, G, offsets = s["T"], s["G"], s["offsets"]
    if op == "experts_fp8":
        sk.gemm_grouped_fp8_bt(s["a"], s["a_scales"], s["b"], s["b_scales"], offsets, s["result"], T, G, N, K, s["out"])
        return {"out": s["result"]}
    if op == "experts":
        product = sk.gemm_grouped_kn if s["layout"] == "kn" else sk.gemm_grouped_bt
        product(s["a"], s["b"], offsets, s["result"], T, G, N, K, s["dtype"], s["out"])
        return {"out": s["result"]}
    dt = s["dtype"]
    sk.gemm_grouped_bt(s["a"], s["b"], offsets, s["result"], T, G, N, K, dt, dt)
    sk.gemm_grouped_kn(s["d"], s["b"], offsets, s["da"], T, G, K, N, dt, dt)
    sk.gemm_grouped_dw(s["a"], s["d"], offsets, s["db"], T, G, N, K, dt, "f32")
    return {"out": s["result"], "da": s["da"], "db": s["db"]}


def _real_rows(q, scales):
    """The numbers that 8-bit rows stand for, in 32 bits."""
    return q.float() * scales.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _real_weights(q, scales):
    return q.float() * scales.repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)[..., :q.shape[-2], :q.shape[-1]]


def _places(offsets, T, most):
    """Where an expert's rows stand: row numbers [G, most], which of them exist, and each row's place in that table."""
    at = torch.arange(T, device=offsets.device)
    expert = torch.searchsorted(offsets[1:], at, right=True)
    rows = offsets[:-1, None] + torch.arange(most, device=offsets.device)
    return rows.clamp(max=T - 1), rows < offsets[1:, None], expert * most + at - offsets[expert]


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        h = s["x"]
        if s["residual_in"] is not None:
            h = (h.float() + s["residual_in"].float()).to(h.dtype)
        y = h.float() * torch.rsqrt(h.float().square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scales = _quantized_rows(y)
        return {"q": q, "scales": scales, "sum": h if s["residual_in"] is not None else None, "y": y.to(h.dtype) if s["y"] else None}
    if op == "fp8":
        return {"out": (_real_rows(s["a"], s["a_scales"]) @ _real_weights(s["b"], s["b_scales"]).mT).to(DTYPES[s["out"]])}
    T, G, N, K = s["T"], s["G"], s["N"], s["K"]
    rows, there, place = _places(s["offsets"].long(), T, s["most"])
    if op == "experts_fp8":
        a, b = _real_rows(s["a"], s["a_scales"]), _real_weights(s["b"], s["b_scales"])
        return {"out": (a[rows] @ b.mT).view(-1, N)[place].to(DTYPES[s["out"]])}
    a, b = s["a"].float(), s["b"].float()
    if op == "experts":
        return {"out": (a[rows] @ (b if s["layout"] == "kn" else b.mT)).view(-1, N)[place].to(DTYPES[s["out"]])}
    dt, d = DTYPES[s["dtype"]], s["d"].float()
    a, d = a[rows], d[rows] * there[..., None]
    return {"out": (a @ b.mT).view(-1, N)[place].to(dt), "da": (d @ b).view(-1, K)[place].to(dt), "db": d.mT @ a}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "norm":
        M, K, e = case["M"], case["K"], size[case["dtype"]]
        reads = M * K * e * (2 if case["residual"] else 1) + K * e
        writes = M * K + 4 * M * _blocks(K) + M * K * e * (case["residual"] + case["y"])
        return {"bytes": reads + writes, "flops": 6 * M * K}
    N, K = case["N"], case["K"]
    if case["op"] == "fp8":
        M = case["M"]
        return {"bytes": M * K + N * K + 4 * _blocks(K) * (M + _blocks(N)) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    T, G = case["T"], case["G"]
    active = min(T, G - case["empty"])
    if case["op"] == "experts_fp8":
        b = T * K + active * N * K + 4 * _blocks(K) * (T + active * _blocks(N)) + 4 * (G + 1) + T * N * size[case["out"]]
        return {"bytes": b, "flops": 2 * T * N * K}
    if case["op"] == "experts":
        return {"bytes": 2 * (T * K + active * N * K) + 4 * (G + 1) + T * N * size[case["out"]], "flops": 2 * T * N * K}
    # read once: activations, weights, the output's gradient; written once: output, both gradients
    b = 2 * (T * K + active * N * K + T * N) + 4 * (G + 1) + 2 * (T * N + T * K) + 4 * G * N * K
    return {"bytes": b, "flops": 6 * T * N * K}


def exact(case, seed):
    s = prepare(case, seed)

    def wide(q, scales, rows_too):
        w = q.double()
        for j in range(scales.shape[-1]):
            f = scales[..., j].double()
            if rows_too:  # one scale for 128 rows
                f = torch.cat([f[..., i:i + 1].expand(*f.shape[:-1], min(BLOCK, w.shape[-2] - i * BLOCK)) for i in range(f.shape[-1])], -1)
            w[..., j * BLOCK:(j + 1) * BLOCK] *= f[..., None]
        return w

    if case["op"] == "norm":
        h = s["x"].double()
        if case["residual"]:  # the sum is kept in the inputs' type, and the norm is of what is kept
            h = (h + s["residual_in"].double()).to(s["x"].dtype).double()
        y = h / (h.pow(2).sum(-1, keepdim=True) / case["K"] + EPS).sqrt() * s["weight"].double()
        scales = torch.stack([p.abs().max(-1).values for p in y.split(BLOCK, -1)], -1) / E4M3_MAX
        codes = torch.cat([p / scales[:, j:j + 1] for j, p in enumerate(y.split(BLOCK, -1))], -1)
        # the nearest number with four significant bits, steps no finer than 2^-9, ties to even
        step = torch.exp2((torch.frexp(codes).exponent - 4).clamp_min(-9).double())
        return {"q": (codes / step).round() * step, "scales": scales, "sum": h if case["residual"] else None, "y": y if case["y"] else None}
    if case["op"] == "fp8":
        return {"out": wide(s["a"], s["a_scales"], False) @ wide(s["b"], s["b_scales"], True).t()}
    o = s["offsets"].tolist()
    runs = [(g, slice(o[g], o[g + 1])) for g in range(case["G"])]
    if case["op"] == "experts_fp8":
        a = wide(s["a"], s["a_scales"], False)
        return {"out": torch.cat([a[r] @ wide(s["b"][g], s["b_scales"][g], True).t() for g, r in runs])}
    a = s["a"].double()
    if case["op"] == "experts":
        return {"out": torch.cat([a[r] @ (s["b"][g].double() if case["layout"] == "kn" else s["b"][g].double().t()) for g, r in runs])}
    d = s["d"].double()
    return {"out": torch.cat([a[r] @ s["b"][g].double().t() for g, r in runs]),
            "da": torch.cat([d[r] @ s["b"][g].double() for g, r in runs]),
            "db": torch.stack([d[r].t() @ a[r] for g, r in runs])}

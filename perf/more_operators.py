"""Cases for routing, rows sorted by expert and back, layer norm and the gradient norm, and the same operators in elementary torch operations.

Five kinds of pass, named by a case's "op":

  route     each token's `top` best experts and their softmax shares; with "train" the logits' gradient too
  dispatch  tokens sorted by expert: run offsets, where each token's rows went, and the rows (16 or 32 bits, or 8 bits with their scales)
  combine   the experts' rows back to their tokens, weighted by the shares; with "train" the gradients of the rows, of the shares and of the
            tokens that were sorted
  norm      residual addition and layer norm; with "train" the gradients of its input, weight and bias
  clip      the norm of all gradients of a model, and the gradients scaled to a largest norm

`own = False` computes them here in 32 bits; `own = True` calls this repository's library.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128            # 8-bit values that share a scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}
EPS = 1e-5
LARGEST = 1 << 27      # values in the largest operand of any case


def listed():
    return [
        # one decoding step's tokens, shares over the chosen experts alone
        {"name": "route_decode", "op": "route", "M": 64, "G": 32, "top": 4, "dtype": "bf16", "chosen_only": True, "masked": 0.0, "padded": 0, "train": False},
        # a training batch over many experts, shares of all of them, the end of the batch padded
        {"name": "route_train", "op": "route", "M": 8192, "G": 256, "top": 8, "dtype": "f32", "chosen_only": False, "masked": 0.1, "padded": 100, "train": True},
        # the decoding step's 8-bit rows on their way to the experts
        {"name": "dispatch_decode", "op": "dispatch", "M": 64, "top": 4, "G": 32, "K": 4096, "dtype": "fp8", "padded": 0},
        # a training batch, each token to eight of many experts
        {"name": "dispatch_train", "op": "dispatch", "M": 8192, "top": 8, "G": 256, "K": 2048, "dtype": "bf16", "padded": 100},
        # the decoding step's rows on their way back
        {"name": "combine_decode", "op": "combine", "M": 64, "top": 4, "K": 4096, "dtype": "bf16", "padded": 0, "train": False},
        # a ragged training batch of odd sizes, part of it padding
        {"name": "combine_ragged", "op": "combine", "M": 1003, "top": 3, "K": 1544, "dtype": "f16", "padded": 41, "train": True},
        # a training batch of the size of the one above that is sorted
        {"name": "combine_train", "op": "combine", "M": 8192, "top": 8, "K": 2048, "dtype": "bf16", "padded": 100, "train": True},
        # one token's hidden state, the smallest call of a decoding step
        {"name": "norm_token", "op": "norm", "M": 1, "K": 2048, "dtype": "bf16", "residual": True, "train": False},
        # a small ragged training batch
        {"name": "norm_ragged", "op": "norm", "M": 333, "K": 5120, "dtype": "f16", "residual": True, "train": True},
        # a large training batch
        {"name": "norm_train", "op": "norm", "M": 8192, "K": 8192, "dtype": "bf16", "residual": True, "train": True},
        # the gradients of one small layer, in 32 bits
        {"name": "clip_layer", "op": "clip", "tensors": 9, "largest": 1 << 18, "shapes": 1, "dtypes": "f32", "clips": True},
        # the gradients of a model of many layers, a few of them (norms, biases) in 32 bits
        {"name": "clip_model", "op": "clip", "tensors": 290, "largest": 1 << 23, "shapes": 2, "dtypes": "mixed", "clips": True},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number of steps between lo and hi, even over its logarithm."""
    return min(hi, step * max(1, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))


def draw(rng):
    op = rng.choice(["route", "dispatch", "dispatch", "combine", "combine", "norm", "norm", "clip"])
    if op == "route":
        G = _log(rng, 4, 512)
        M = _log(rng, 1, 8192)
        return {"op": op, "M": M, "G": G, "top": rng.randint(1, min(G, 8)), "dtype": rng.choice(["f32", "bf16", "f16"]), "chosen_only": rng.random() < 0.5,
                "masked": rng.choice([0.0, 0.1, 0.5]), "padded": rng.randint(0, M // 8), "train": rng.random() < 0.5}
    if op in ("dispatch", "combine"):
        while True:
            M = _log(rng, 1, 8192)
            c = {"op": op, "M": M, "top": rng.randint(1, 8)}
            if op == "dispatch":
                c |= {"G": _log(rng, max(2, c["top"]), 512), "K": _log(rng, 256, 8192, 16), "dtype": rng.choice(["fp8", "fp8", "bf16", "f16", "f32"])}
            else:
                c |= {"K": _log(rng, 256, 8192, 8), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "train": rng.random() < 0.5}
            c["padded"] = rng.randint(0, M // 8)
            if M * c["top"] * c["K"] * SIZE[c["dtype"]] <= 2 * LARGEST:
                return c
    if op == "norm":
        while True:
            c = {"op": op, "M": _log(rng, 1, 16384), "K": _log(rng, 64, 16384, 8), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
                 "residual": rng.random() < 0.7, "train": rng.random() < 0.7}
            if c["M"] * c["K"] * SIZE[c["dtype"]] <= LARGEST:
                return c
    return {"op": op, "tensors": _log(rng, 1, 290), "largest": _log(rng, 1 << 12, 1 << 23), "shapes": rng.randrange(1 << 20),
            "dtypes": rng.choice(["f32", "bf16", "mixed"]), "clips": rng.random() < 0.8}


def _blocks(k):
    return (k + BLOCK - 1) // BLOCK


def _sizes(case):
    """Values and type of each gradient of a model: some matrices of the largest size, smaller ones, and vectors; any size, odd ones among them."""
    r = np.random.RandomState(case["shapes"])
    top = case["largest"]
    many = [top if u < 0.3 else max(1, int(top ** (0.5 + 0.5 * u))) if u < 0.7 else max(1, int(top ** (0.5 * u))) for u in r.random_sample(case["tensors"] - 1)]
    sizes = [top, *many]
    kinds = {"f32": ["f32"] * 4, "bf16": ["bf16"] * 4, "mixed": ["bf16", "bf16", "f16", "f32"]}[case["dtypes"]]
    names = [("f32" if n < 1 << 14 else "bf16") if case["dtypes"] == "mixed" and u < 0.8 else kinds[int(4 * u)] for n, u in zip(sizes, r.random_sample(len(sizes)))]
    return sizes, names


def _flat(case):
    """The gradients as a trainer keeps them, views of one buffer a type: its length, and each view's place in it (16-byte steps)."""
    length, places = {}, []
    for n, name in zip(*_sizes(case)):
        at = length.get(name, 0)
        places.append((name, at, n))
        step = 16 // SIZE[name]
        length[name] = at + (n + step - 1) // step * step
    return length, places


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    def activations(m, k):  # a few channels are much larger than the others, as in a residual stream
        return normal(m, k) * torch.exp(0.7 * normal(1, k))

    def zeros(shape, name):
        return torch.zeros(shape, dtype=DTYPES[name], device=dev)

    def whole(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=dev)

    s = dict(case)
    op = case["op"]
    if op == "clip":
        length, places = _flat(case)
        s["flat"] = {name: zeros(n, name) for name, n in length.items()}
        s["flat_out"] = {name: zeros(n, name) for name, n in length.items()}
        s["grads"], s["out"] = ([flat[name][at:at + n] for name, at, n in places] for flat in (s["flat"], s["flat_out"]))
        spread = torch.exp(normal(len(places)) - 4).tolist()
        for g, scale in zip(s["grads"], spread):
            g.copy_(normal(g.numel()) * scale)
        total = math.sqrt(sum(g.numel() * scale ** 2 for g, scale in zip(s["grads"], spread)))
        s["max_norm"] = total * (0.3 if case["clips"] else 3.0)
        s["norm_out"] = zeros(1, "f32")
        if own:  # what a program keeps beside its gradients
            import split_bf16_gemm_gb300 as sk

            s["list"], s["out_list"] = sk.grad_list(s["grads"]), sk.grad_list(s["out"])
            s["nbytes"] = sk.grad_norm_workspace_bytes()
            s["workspace"] = torch.empty(s["nbytes"], dtype=torch.uint8, device=dev)
        return s
    M = case["M"]
    if op == "norm":
        K, dt = case["K"], case["dtype"]
        s["x"] = (activations(M, K) + 0.3 * normal(M, 1)).to(DTYPES[dt])
        s["residual_in"] = activations(M, K).to(DTYPES[dt]) if case["residual"] else None
        s["weight"], s["bias"] = (1 + 0.1 * normal(K)).to(DTYPES[dt]), (0.1 * normal(K)).to(DTYPES[dt])
        s["sum_out"] = zeros((M, K), dt) if case["residual"] else None
        s["y_out"] = zeros((M, K), dt)
        if case["train"]:
            s["mean_out"], s["rstd_out"] = zeros(M, "f32"), zeros(M, "f32")
            s["dy"] = (0.1 * normal(M, K)).to(DTYPES[dt])
            s["dsum"] = (0.1 * normal(M, K)).to(DTYPES[dt]) if case["residual"] else None
            s["dx_out"], s["dweight_out"], s["dbias_out"] = zeros((M, K), dt), zeros(K, "f32"), zeros(K, "f32")
            if own:
                import split_bf16_gemm_gb300 as sk

                s["nbytes"] = sk.layernorm_grad_workspace_bytes(M, K)
                s["workspace"] = torch.empty(s["nbytes"], dtype=torch.uint8, device=dev)
        return s
    top = case["top"]
    live = torch.arange(M, device=dev) < M - case["padded"]
    if op == "route":
        G, dt = case["G"], case["dtype"]
        logits = 2 * normal(M, G) + normal(1, G)  # some experts are preferred
        logits[torch.rand(M, G, device=dev, generator=gen) < case["masked"]] = -math.inf
        logits[~live] = -math.inf
        s["logits"] = logits.to(DTYPES[dt])
        s["experts_out"], s["shares_out"] = whole(M, top), zeros((M, top), "f32")
        if case["train"]:
            s["dshares"] = 0.1 * normal(M, top)
            s["dlogits_out"] = zeros((M, G), dt)
        return s
    K, dt, T = case["K"], case["dtype"], M * top
    if op == "dispatch":
        G = case["G"]
        experts = (normal(M, G) + normal(1, G)).argsort(-1)[:, :top]
        s["experts"] = torch.where(live[:, None], experts, -1).int().contiguous()
        if dt == "fp8":
            s["x"] = (60 * normal(M, K)).clamp(-448, 448).to(DTYPES[dt])
            s["scales"] = torch.exp(normal(M, _blocks(K)) - 4)
            s["row_scales_out"] = zeros((T, _blocks(K)), "f32")
        else:
            s["x"] = activations(M, K).to(DTYPES[dt])
        s["rows_out"] = zeros((T, K), dt)
        s["offsets_out"], s["slots_out"], s["source_out"] = whole(G + 1), whole(M, top), whole(T)
        return s
    # sorted rows of live tokens, in any order that a sort can give
    used = (M - case["padded"]) * top
    slots = torch.full((M, top), -1, device=dev)
    slots[live] = torch.rand(used, device=dev, generator=gen).argsort().view(-1, top)
    s["slots"] = slots.int()
    s["shares"] = torch.softmax(normal(M, top), -1)
    s["rows"] = activations(T, K).to(DTYPES[dt])
    s["out"] = zeros((M, K), dt)
    if case["train"]:
        s["dout"], s["drows"] = (0.1 * normal(M, K)).to(DTYPES[dt]), (0.1 * normal(T, K)).to(DTYPES[dt])
        s["drows_out"], s["dshares_out"], s["dx_out"] = zeros((T, K), dt), zeros((M, top), "f32"), zeros((M, K), dt)
    return s


def _run_own(s):
    import split_bf16_gemm_gb300 as sk

    op = s["op"]
    if op == "clip":
        sk.grad_clip(s["list"], s["max_norm"], s["norm_out"], s["workspace"], s["nbytes"], out=s["out_list"])
        return {"norm": s["norm_out"], "grads": s["flat_out"]}
    M = s["M"]
    if op == "norm":
        K, dt = s["K"], s["dtype"]
        if not s["train"]:
            sk.layernorm(s["x"], s["weight"], s["bias"], s["y_out"], M, K, dt, eps=EPS, residual=s["residual_in"], sum_out=s["sum_out"])
            return {"sum": s["sum_out"], "y": s["y_out"]}
        sk.layernorm(s["x"], s["weight"], s["bias"], s["y_out"], M, K, dt, eps=EPS, residual=s["residual_in"], sum_out=s["sum_out"],
                     mean=s["mean_out"], rstd=s["rstd_out"])
        h = s["x"] if s["sum_out"] is None else s["sum_out"]
        sk.layernorm_grad(s["dy"], h, s["weight"], s["mean_out"], s["rstd_out"], s["dx_out"], s["dweight_out"], s["dbias_out"],
                          s["workspace"], s["nbytes"], M, K, dt, dsum=s["dsum"])
        return {"sum": s["sum_out"], "y": s["y_out"], "mean": s["mean_out"], "rstd": s["rstd_out"],
                "dx": s["dx_out"], "dweight": s["dweight_out"], "dbias": s["dbias_out"]}
    top, dt = s["top"], s["dtype"]
    if op == "route":
        G = s["G"]
        sk.moe_route(s["logits"], s["experts_out"], s["shares_out"], M, G, top, dt, chosen_only=s["chosen_only"])
        out = {"experts": s["experts_out"], "shares": s["shares_out"]}
        if s["train"]:
            sk.moe_route_grad(s["logits"], s["experts_out"], s["dshares"], s["dlogits_out"], M, G, top, dt, chosen_only=s["chosen_only"])
            out["dlogits"] = s["dlogits_out"]
        return out
    K = s["K"]
    if op == "dispatch":
        out = {"offsets": s["offsets_out"], "slots": s["slots_out"], "source": s["source_out"], "rows": s["rows_out"]}
        if dt == "fp8":
            sk.moe_dispatch_fp8(s["experts"], s["x"], s["scales"], s["offsets_out"], s["slots_out"], s["source_out"], s["rows_out"],
                                s["row_scales_out"], M, top, s["G"], K)
            out["scales"] = s["row_scales_out"]
        else:
            sk.moe_dispatch(s["experts"], s["x"], s["offsets_out"], s["slots_out"], s["source_out"], s["rows_out"], M, top, s["G"], K, dt)
        return out
    sk.moe_combine(s["rows"], s["slots"], s["shares"], s["out"], M, top, K, dt, dt)
    out = {"out": s["out"]}
    if s["train"]:
        sk.moe_combine_grad(s["dout"], s["rows"], s["slots"], s["shares"], s["drows_out"], s["dshares_out"], M, top, K, dt)
        sk.moe_combine(s["drows"], s["slots"], None, s["dx_out"], M, top, K, dt, dt)
        out |= {"drows": s["drows_out"], "dshares": s["dshares_out"], "dx": s["dx_out"]}
    return out


def _plain_clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).double().sum().sqrt()
    factor = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    return {"norm": norm.float().view(1), "grads": {name: (flat.float() * factor).to(flat.dtype) for name, flat in s["flat"].items()}}


def _plain_norm(s):
    h = s["x"]
    if s["residual_in"] is not None:
        h = (h.float() + s["residual_in"].float()).to(h.dtype)
    mean = h.float().mean(-1, keepdim=True)
    rstd = torch.rsqrt((h.float() - mean).square().mean(-1, keepdim=True) + EPS)
    xhat = (h.float() - mean) * rstd
    out = {"sum": None if s["residual_in"] is None else h, "y": (xhat * s["weight"].float() + s["bias"].float()).to(h.dtype)}
    if s["train"]:
        dy = s["dy"].float()
        g = dy * s["weight"].float()
        dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        out |= {"mean": mean.view(-1), "rstd": rstd.view(-1), "dx": dx.to(h.dtype), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}
    return out


def _plain_route(s):
    logits, top, chosen_only = s["logits"].float(), s["top"], s["chosen_only"]
    value, expert = (t[:, :top] for t in torch.sort(logits, dim=-1, descending=True, stable=True))
    there = value > -math.inf
    most = torch.where(there[:, :1], value[:, :1], 0.0)
    part = torch.exp(value - most)
    total = (part if chosen_only else torch.exp(logits - most)).sum(-1, keepdim=True)
    total = torch.where(total > 0, total, 1.0)
    shares = part / total
    out = {"experts": torch.where(there, expert, -1).int(), "shares": shares}
    if s["train"]:
        d = s["dshares"]
        mean = (d * shares).sum(-1, keepdim=True)
        p = torch.zeros_like(logits) if chosen_only else torch.exp(logits - most) / total
        out["dlogits"] = (-p * mean).scatter(-1, expert, shares * (d - mean)).to(s["logits"].dtype)
    return out


def _plain_dispatch(s):
    flat, T, top = s["experts"].flatten().long(), s["M"] * s["top"], s["top"]
    key, source = torch.sort(torch.where(flat < 0, s["G"], flat), stable=True)
    offsets = torch.searchsorted(key, torch.arange(s["G"] + 1, device=key.device))
    there = key < s["G"]
    at = torch.arange(T, device=key.device)
    slots = torch.zeros_like(flat).scatter(0, source, torch.where(there, at, -1))
    raw = s["x"].view(torch.uint8) if s["dtype"] == "fp8" else s["x"]
    rows = torch.where(there[:, None], raw[source // top], 0).view(s["x"].dtype)
    out = {"offsets": offsets.int(), "slots": slots.view(-1, top).int(), "source": torch.where(there, source, -1).int(), "rows": rows}
    if s["dtype"] == "fp8":
        out["scales"] = torch.where(there[:, None], s["scales"][source // top], 0.0)
    return out


def _plain_combine(s):
    slots, rows, there = s["slots"].long().clamp(min=0), s["rows"].float(), (s["slots"] >= 0)[..., None]
    mine = torch.where(there, rows[slots], 0.0)
    out = {"out": (mine * s["shares"][..., None]).sum(1).to(s["rows"].dtype)}
    if s["train"]:
        d = s["dout"].float()[:, None]
        part = (d * s["shares"][..., None]).to(s["rows"].dtype)
        at = torch.where(there[..., 0], slots, rows.shape[0]).flatten()  # one row more, for what goes nowhere
        drows = rows.new_zeros(rows.shape[0] + 1, rows.shape[1], dtype=part.dtype).index_copy(0, at, part.flatten(0, 1))[:-1]
        dx = torch.where(there, s["drows"].float()[slots], 0.0).sum(1)
        out |= {"drows": drows, "dshares": (mine * d).sum(-1), "dx": dx.to(s["rows"].dtype)}
    return out


def _run_plain(s):
    return {"clip": _plain_clip, "norm": _plain_norm, "route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine}[s["op"]](s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "clip":
        sizes, names = _sizes(case)
        return {"bytes": 2 * sum(n * SIZE[name] for n, name in zip(sizes, names)) + 4, "flops": 3 * sum(sizes)}
    M, e = case["M"], SIZE[case["dtype"]]
    if op == "norm":
        K = case["K"]
        values = M * K * (2 + 2 * case["residual"]) + 2 * K
        if not case["train"]:
            return {"bytes": values * e, "flops": 8 * M * K}
        values += M * K * (2 + case["residual"])  # the output's and the sum's gradients in, the input's out
        return {"bytes": values * e + 8 * M + 8 * K, "flops": 24 * M * K}
    top = case["top"]
    if op == "route":
        G = case["G"]
        train = case["train"]
        return {"bytes": M * G * e * (1 + train) + M * top * 4 * (2 + train), "flops": M * G * (4 + 3 * train)}
    K, T, rows = case["K"], M * top, (M - case["padded"]) * top
    if op == "dispatch":
        row = K + 4 * _blocks(K) if case["dtype"] == "fp8" else K * e
        return {"bytes": 12 * T + 4 * (case["G"] + 1) + (M - case["padded"]) * row + rows * row, "flops": T}
    if not case["train"]:
        return {"bytes": rows * K * e + M * K * e + 8 * T, "flops": 2 * rows * K}
    # in: the rows, the rows' gradient from the experts, the output's gradient; out: the output, the tokens' gradient, the rows' gradient
    return {"bytes": 3 * rows * K * e + 3 * M * K * e + 12 * T, "flops": 6 * rows * K}


def exact(case, seed):
    global own
    kept, own = own, False  # its inputs alone
    s = prepare(case, seed)
    own = kept
    op = case["op"]
    if op == "clip":
        norm = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in s["grads"]))
        return {"norm": torch.tensor([norm], dtype=torch.float64), "grads": {k: v.double() * min(1.0, s["max_norm"] / norm) for k, v in s["flat"].items()}}
    if op == "norm":
        h = s["x"].double()
        if case["residual"]:  # the sum is kept in the inputs' type, and the norm is of what is kept
            h = (h + s["residual_in"].double()).to(s["x"].dtype).double()
        K = case["K"]
        mean = h.sum(1) / K
        off = h - mean[:, None]
        rstd = 1 / (off.pow(2).sum(1) / K + EPS).sqrt()
        w = s["weight"].double()
        out = {"sum": h if case["residual"] else None, "y": off * rstd[:, None] * w + s["bias"].double()}
        if case["train"]:
            dy = s["dy"].double()
            # the derivative of (h_k - mean) rstd by h_i is rstd (delta_ik - 1 / K) - off_k off_i rstd^3 / K
            a, b = (dy @ w) / K, ((dy * off) @ w) / K
            dx = rstd[:, None] * (dy * w - a[:, None]) - off * (b * rstd.pow(3))[:, None]
            out |= {"mean": mean, "rstd": rstd, "dx": dx + s["dsum"].double() if case["residual"] else dx,
                    "dweight": torch.einsum("mk,m->k", dy * off, rstd), "dbias": dy.sum(0)}
        return out
    M, top = case["M"], case["top"]
    if op == "route":
        logits = s["logits"].double()
        G, dev = case["G"], logits.device
        # the number of experts before each one: larger logits, and equal ones of a lower index
        before = torch.zeros(M, G, dtype=torch.long, device=dev)
        for g in range(G):
            before[:, g] = (logits > logits[:, g:g + 1]).sum(1) + (logits[:, :g] == logits[:, g:g + 1]).sum(1)
        chosen = (before < top) & (logits > -math.inf)
        among = logits if not case["chosen_only"] else torch.where(chosen, logits, -math.inf)
        p = torch.nan_to_num(torch.softmax(among, -1))  # a row without any expert has shares of 0
        place = torch.where(chosen, before, top)
        shares = torch.zeros(M, top + 1, dtype=torch.float64, device=dev).scatter_add(1, place, torch.where(chosen, p, 0.0))[:, :top]
        experts = torch.full((M, top + 1), -1, device=dev).scatter(1, place, torch.arange(G, device=dev).expand(M, G))
        experts[:, top] = -1
        out = {"experts": experts[:, :top].int(), "shares": shares}
        if case["train"]:
            d = torch.cat([s["dshares"].double(), torch.zeros(M, 1, dtype=torch.float64, device=dev)], 1).gather(1, place)
            out["dlogits"] = p * (d - (p * d).sum(1, keepdim=True))
        return out
    if op == "dispatch":
        flat = s["experts"].flatten().tolist()
        order = sorted((t for t in range(len(flat)) if flat[t] >= 0), key=lambda t: (flat[t], t))
        counts, slots = [0] * (case["G"] + 1), [-1] * len(flat)
        for r, t in enumerate(order):
            counts[flat[t] + 1] += 1
            slots[t] = r
        source = torch.tensor(order + [-1] * (len(flat) - len(order)), dtype=torch.int32)
        token = source[:len(order)].long().to(s["x"].device) // top
        out = {"offsets": torch.tensor(counts).cumsum(0).int(), "slots": torch.tensor(slots, dtype=torch.int32).view(M, top), "source": source}
        for name, x in (("rows", s["x"]), ("scales", s.get("scales"))):
            if x is not None:  # rows that nothing was sorted into stay as they were, zeros
                out[name] = torch.cat([x.double()[token], torch.zeros(len(flat) - len(order), x.shape[1], dtype=torch.float64, device=x.device)])
        return out
    mine = s["slots"].cpu().numpy()
    rows, shares = s["rows"].double(), s["shares"].double()
    m, j = (torch.from_numpy(v).to(rows.device) for v in np.nonzero(mine >= 0))
    at = s["slots"][m, j].long()
    out = torch.zeros(M, case["K"], dtype=torch.float64, device=rows.device)
    r = {"out": out.index_add(0, m, rows[at] * shares[m, j, None])}
    if case["train"]:
        d = s["dout"].double()[m]
        r["drows"] = torch.zeros_like(rows)
        r["drows"][at] = d * shares[m, j, None]
        r["dshares"] = torch.zeros_like(shares)
        r["dshares"][m, j] = torch.einsum("rk,rk->r", d, rows[at])
        r["dx"] = out.index_add(0, m, s["drows"].double()[at])
    return r

"""More tests of the 8-bit and grouped operators on the GPU: pairs of thread
blocks that leave, long contractions, rows at the ends of F32's range, every
plan, broken offsets over many runs, streams, threads and captured chains.

Tolerances are those of test_gpu_fp8_grouped.py unless a test states its own.
"""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_fp8_grouped import (BLOCK, DT, E4M3, HALF_UNIT, Guarded, c_16, c_fp8, check, check_rows,  # noqa: E402
                                  fp8_rows, fp8_weights, gen, nblk, offsets_of, randn, real_rows,
                                  real_weights, runs, sk, spread)  # noqa: F401

pytestmark = pytest.mark.gpu


def whole(g, dtype, *shape, most=3):
    """Whole numbers of at most `most`: products and sums of fewer than 2^24 are exact."""
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).float().to(dtype)


# ------------------------------------------------------------------ pairs of thread blocks

@pytest.mark.parametrize("kblocks", [1, 2, 3, 4, 5, 6, 7, 9])
@pytest.mark.parametrize("form", ["fp8", "bt", "dw"])
def test_pairs_leave_after_their_last_stages(sk, form, kblocks):
    """Launches of pairs (this many tiles take them) with fewer k-blocks than the
    ring has stages, as many and more, one behind the other: the next launch's
    blocks take over the shared memory that the last one's arrivals went to."""
    g = gen(kblocks)
    M = N = 4096
    outs = [Guarded((M, N), torch.float32) for _ in range(2)]
    if form == "fp8":
        K = 128 * kblocks - 16
        a, b = whole(g, E4M3, M, K), whole(g, E4M3, N, K)
        ones = [torch.ones(r, kblocks, device="cuda") for r in (M, (N + 127) // 128)]
        for i in range(24):
            sk.gemm_fp8_bt(a, ones[0], b, ones[1], outs[i % 2].data, M, N, K, "f32")
        want = a.double() @ b.double().T
    elif form == "bt":
        K = 64 * kblocks - 8
        a, b = whole(g, torch.bfloat16, M, K), whole(g, torch.bfloat16, N, K)
        _, offs = offsets_of([M])
        for i in range(24):
            sk.gemm_grouped_bt(a, b, offs, outs[i % 2].data, M, 1, N, K, "bf16", "f32")
        want = a.double() @ b.double().T
    else:
        T = 64 * kblocks - 5                      # the last k-block ends inside a step of 16
        a, d = whole(g, torch.bfloat16, T, M), whole(g, torch.bfloat16, T, N)
        _, offs = offsets_of([T])
        for i in range(24):
            sk.gemm_grouped_dw(a, d, offs, outs[i % 2].data, T, 1, N, M, "bf16", "f32")
        want = d.double().T @ a.double()
    assert sk.splitk_get_device_status() == 0
    for out in outs:
        assert torch.equal(out.data.double(), want) and out.intact()


# ------------------------------------------------------------------ long contractions

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form", ["bt", "kn", "dw"])
def test_long_contraction_with_16_bit_output(sk, form, dt):
    """131072 products of one sign a value: the output is rounded from an F32 sum,
    so the error that goes with the length is that of its additions (every 512
    products), not of a tensor-core accumulator (every 16, cut off): c_16 of an
    F32 output, and half a unit of the output's last place."""
    L = 131072
    g = gen(21)

    def positive(*shape):
        return (torch.rand(*shape, device="cuda", generator=g) * 0.5 + 0.25).to(DT[dt])

    if form == "dw":
        counts, N, K = [L, 0, 70], 136, 72
        T, G = sum(counts), len(counts)
        a, d = positive(T, K), positive(T, N)
        o, offs = offsets_of(counts)
        res = Guarded((G, N, K), DT[dt])
        sk.gemm_grouped_dw(a, d, offs, res.data, T, G, N, K, dt, dt)
        got = [(res.data[e], d[r].double().T @ a[r].double()) for e, r in runs(o)]
        assert not res.data[1].any()
    else:
        T, N = 1100, 1104
        a = positive(T, L)
        w = positive(1, *((L, N) if form == "kn" else (N, L)))
        _, offs = offsets_of([T])
        res = Guarded((T, N), DT[dt])
        (sk.gemm_grouped_kn if form == "kn" else sk.gemm_grouped_bt)(a, w, offs, res.data, T, 1, N, L, dt, dt)
        rows = torch.arange(0, T, 17, device="cuda")
        got = [(res.data[rows], a[rows].double() @ (w[0] if form == "kn" else w[0].T).double())]
    assert sk.splitk_get_device_status() == 0
    for out, ref in got:
        check(out, ref, ref, c_16(L, "f32"), dt)       # all terms are positive
    assert res.intact()


# ------------------------------------------------------------------ scales and codes to the last bit

def scales_of(m):
    """max(m / 448, 2^-126) in F32 from the largest magnitudes m: a quotient of F32
    numbers in 64 bits is far enough from a tie to be rounded to F32 once more."""
    return (m.double() / 448).clamp_min(2.0 ** -126).float()


def largest(x):
    M, K = x.shape
    return torch.nn.functional.pad(x.float(), (0, nblk(K) * BLOCK - K)).view(M, -1, BLOCK).abs().amax(-1)


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (300, 400), (64, 4096), (3, 30000)])
def test_quantized_rows_to_the_last_bit(sk, M, K, dt):
    x = (randn(gen(K + M), M, K) * 3).to(DT[dt])
    q, s = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32)
    sk.fp8_quantize(x, q.data, s.data, M, K, dt)
    assert torch.equal(s.data, scales_of(largest(x)))
    assert same_bits(q.data, (x.float() / spread(s.data, K, 1)).to(E4M3))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (3, 130, 272), (2, 500, 2064)])
def test_prepared_weights_to_the_last_bit(sk, G, N, K, dt):
    b = randn(gen(N + K), G, N, K).to(DT[dt])
    q, s = Guarded((G, N, K), E4M3), Guarded((G, nblk(N), nblk(K)), torch.float32)
    sk.fp8_prepare_bt(b, q.data, s.data, G, N, K, dt)
    pad = torch.nn.functional.pad(b.float(), (0, nblk(K) * BLOCK - K, 0, nblk(N) * BLOCK - N))
    assert torch.equal(s.data, scales_of(pad.view(G, nblk(N), BLOCK, nblk(K), BLOCK).abs().amax((2, 4))))
    assert same_bits(q.data, (b.float() / spread(spread(s.data, N, 1), K, 2)).to(E4M3))


@pytest.mark.parametrize("M,K", [(300, 400), (64, 4096), (3, 30000)])
def test_norm_codes_follow_from_its_output(sk, M, K):
    """With F32 inputs y is what the scales and codes are made of."""
    g = gen(K)
    x, w = randn(g, M, K), 1 + 0.2 * randn(g, K)
    q, s, y = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32), Guarded((M, K), torch.float32)
    sk.rmsnorm_fp8(x, w, q.data, s.data, M, K, "f32", eps=1e-5, y=y.data)
    assert torch.equal(s.data, scales_of(largest(y.data)))
    assert same_bits(q.data, (y.data / spread(s.data, K, 1)).to(E4M3))


@pytest.mark.parametrize("eps", [0.0, 0.5])
def test_norm_root_is_one_operation(sk, eps):
    """Rows of one value c of 10 significant bits: squares, their sum, the mean and
    the sum with eps are exact, so y = c / sqrt(c^2 + eps) is off by what the
    reciprocal root may be (two units, 2^-22) and the product's rounding, 2^-24."""
    K, M = 512, 512
    c = torch.arange(512, 512 + M, device="cuda").float() / 512
    x = c[:, None].expand(M, K).contiguous()
    q, s, y = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32), Guarded((M, K), torch.float32)
    sk.rmsnorm_fp8(x, torch.ones(K, device="cuda"), q.data, s.data, M, K, "f32", eps=eps, y=y.data)
    ref = x.double() / (x.double().square() + eps).sqrt()
    assert bool(((y.data.double() - ref).abs() <= 5 * 2.0 ** -24 * ref).all())


# ------------------------------------------------------------------ rows whose squares leave F32's range

@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [16, 400, 1008, 2048, 4096, 8208, 20000])
def test_norm_of_rows_at_the_ends_of_the_range(sk, K, dt, eps):
    """Rows of one launch (several share a block) from 3e38 down to the smallest
    numbers, beside ordinary ones, against 64 bits; the relative error of the
    root is test_norm's, whatever the row's size."""
    scale = [1.0, 1e30, 5e19, 3e37, 1e-18, 1e-20, 1e-25, 1e-38, 1.0, 1e-3] + ([1e-43] if dt == "f32" else [])
    M = len(scale)
    g = gen(K)
    x = (randn(g, M, K).clamp(-4, 4).double() * torch.tensor(scale, device="cuda").double()[:, None]).to(DT[dt])
    x[8, 3] = 3e38                                        # one value decides
    w = (1 + 0.2 * randn(g, K)).to(DT[dt])
    q, s, y = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32), Guarded((M, K), DT[dt])
    sk.rmsnorm_fp8(x, w, q.data, s.data, M, K, dt, eps=eps, y=y.data)
    H = x.double()
    ref = H / (H.square().mean(-1, keepdim=True) + torch.tensor(eps, dtype=torch.float32).double().item()).sqrt() * w.double()
    rel = (8 * (K // 4096 + 1) * 4 + 10 + 6) * 2.0 ** -24
    check_rows(ref, q.data, s.data, rel)
    # below 2^-126 the output's step is 2^-149 (BF16: 2^-133)
    tol = (rel + HALF_UNIT[dt]) * ref.abs() + (2.0 ** -133 if dt == "bf16" else 2.0 ** -148)
    assert bool(((y.data.double() - ref).abs() <= tol).all())
    assert q.intact() and s.intact() and y.intact()


@pytest.mark.parametrize("K", [400, 1008, 2048, 20000])
@pytest.mark.parametrize("kept", ["x", "residual", "new", "none"])
def test_norm_of_large_sums(sk, K, kept):
    """The same through the residual's addition, the sum kept in place, elsewhere or not at all."""
    M = 4
    g = gen(K + 1)
    x, r, w = randn(g, M, K) * 1e25, randn(g, M, K) * 1e25, torch.ones(K, device="cuda")
    h = x + r
    q, s = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32)
    out = {"x": x, "residual": r, "new": torch.empty_like(x), "none": None}[kept]
    sk.rmsnorm_fp8(x, w, q.data, s.data, M, K, "f32", residual=r, sum_out=out)
    assert out is None or torch.equal(out, h)
    ref = h.double() / h.double().square().mean(-1, keepdim=True).sqrt()
    check_rows(ref, q.data, s.data, (8 * (K // 4096 + 1) * 4 + 10 + 6) * 2.0 ** -24)


@pytest.mark.parametrize("K", [400, 1008, 20000])
def test_norm_of_zeros_without_eps_and_of_infinities(sk, K):
    """0 / 0 is NaN; beside it an infinity's block is NaN and its row's others 0."""
    x, w = torch.ones(3, K, device="cuda"), torch.ones(K, device="cuda")
    x[0] = 0
    x[1, 200] = -float("inf")
    q, s = Guarded((3, K), E4M3), Guarded((3, nblk(K)), torch.float32)
    sk.rmsnorm_fp8(x, w, q.data, s.data, 3, K, "f32", eps=0.0)
    assert torch.isnan(s.data[0]).all() and torch.isnan(q.data[0].float()).all()
    assert torch.isnan(s.data[1, 1]) and torch.isnan(q.data[1, 200].float())
    assert not q.data[1, :128].float().any() and not q.data[1, 256:].float().any()
    assert bool((q.data[2].float() == 448).all())


# ------------------------------------------------------------------ every plan

PLANS = [(c, s) for c in (32, 64, 128) for s in (1, 2, 4, 8)] + [(256, 1)]
PLAN_IDS = [f"{c}x{s}" for c, s in PLANS]
# counts, N, rows before the first run and after the last: rows that are whole boxes
# of the outputs' stores and not, whole 16 bytes and not, runs that end inside a
# tile, and more tiles than an SM or a pair of them takes at once
PLAN_SETS = {
    "ragged": ([130, 0, 1, 255, 64, 129], 264, 2, 3),
    "rows8": ([700], 1000, 0, 0),
    "odd": ([333, 31, 0, 512], 1001, 1, 0),
    "few": ([0, 3, 1, 0, 16, 33], 520, 0, 1),
    "many": ([2500, 0, 300], 5200, 0, 0),
    "wide": ([4, 60], 5188, 0, 0),
}


@pytest.fixture
def planned(sk):
    yield sk.splitk_set_grouped_override
    sk.splitk_set_grouped_override(0, 0)


_operands = {}


def operands(form, name):
    """Operands of a set and their products in 64 bits, kept while the same set is asked for."""
    if (form, name) not in _operands:
        _operands.clear()
        counts, N, before, after = PLAN_SETS[name]
        if form in ("kn", "dw"):
            N = N // 8 * 8
        K = {"fp8": 2064, "dw": 392}.get(form, 1032)          # 17 k-blocks, the last a short one
        G, T = len(counts), sum(counts) + before + after
        g = gen(T + N)
        o, offs = offsets_of(counts, before)
        if form == "fp8":
            a, b = fp8_rows(g, T, K), fp8_weights(g, G, N, K)
            A, B = real_rows(*a), real_weights(*b)
            refs = [(r, A[r] @ B[e].T, A[r].abs() @ B[e].abs().T) for e, r in runs(o)]
        else:
            a = randn(g, T, K).bfloat16()
            b = randn(g, *{"bt": (G, N, K), "kn": (G, K, N), "dw": (T, N)}[form]).bfloat16()
            A, B = a.double(), b.double()
            if form == "dw":
                refs = [(e, B[r].T @ A[r], B[r].abs().T @ A[r].abs()) for e, r in runs(o)]
            else:
                W = B if form == "kn" else B.mT
                refs = [(r, A[r] @ W[e], A[r].abs() @ W[e].abs()) for e, r in runs(o)]
        _operands[form, name] = (a, b, o, offs, T, G, N, K, refs)
    return _operands[form, name]


def planned_product(sk, form, name, out):
    a, b, o, offs, T, G, N, K, refs = operands(form, name)
    res = Guarded((G, N, K) if form == "dw" else (T, N), DT[out])
    if form == "fp8":
        sk.gemm_grouped_fp8_bt(*a, *b, offs, res.data, T, G, N, K, out)
    else:
        call = {"bt": sk.gemm_grouped_bt, "kn": sk.gemm_grouped_kn, "dw": sk.gemm_grouped_dw}[form]
        call(a, b, offs, res.data, T, G, N, K, "bf16", out)
    return res


def check_planned(sk, form, name, out, plan):
    a, b, o, offs, T, G, N, K, refs = operands(form, name)
    # the same call twice, with another plan's between
    first = planned_product(sk, form, name, out)
    sk.splitk_set_grouped_override(256 if plan[0] == 128 else 128, 1)
    planned_product(sk, form, name, out)
    sk.splitk_set_grouped_override(*plan)
    res = planned_product(sk, form, name, out)
    assert sk.splitk_get_device_status() == 0
    assert torch.equal(first.raw, res.raw)
    # a sum over splits adds one rounding a split
    L = max(o[e + 1] - o[e] for e in range(G)) if form == "dw" else K
    c = (c_fp8(K) if form == "fp8" else c_16(L, out)) + plan[1]
    for at, ref, mag in refs:
        check(res.data[at], ref, mag, c, out)
    if form == "dw":
        for e in range(G):
            assert o[e + 1] > o[e] or not res.data[e].any()
    else:
        assert torch.isnan(res.data[:o[0]].float()).all() and torch.isnan(res.data[o[-1]:].float()).all()
    assert res.intact()


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("plan", PLANS, ids=PLAN_IDS)
@pytest.mark.parametrize("name", PLAN_SETS)
@pytest.mark.parametrize("form", ["fp8", "bt", "kn"])
def test_every_plan(sk, planned, form, name, plan, out):
    planned(*plan)
    check_planned(sk, form, name, out, plan)


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("columns", [128, 256])
@pytest.mark.parametrize("name", PLAN_SETS)
def test_every_plan_of_the_weight_gradient(sk, planned, name, columns, out):
    planned(columns, 1)
    check_planned(sk, "dw", name, out, (columns, 1))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("plan", PLANS, ids=PLAN_IDS)
@pytest.mark.parametrize("M,N", [(1, 64), (33, 1160), (300, 136), (2000, 2600)])
def test_every_plan_of_the_plain_product(sk, planned, M, N, plan, out):
    K = 2064
    g = gen(M)
    a, b = fp8_rows(g, M, K), fp8_weights(g, 1, N, K)
    res = Guarded((M, N), DT[out])
    planned(*plan)
    sk.gemm_fp8_bt(*a, b[0][0], b[1][0], res.data, M, N, K, out)
    assert sk.splitk_get_device_status() == 0
    A, B = real_rows(*a), real_weights(*b)[0]
    check(res.data, A @ B.T, A.abs() @ B.abs().T, c_fp8(K) + plan[1], out)
    assert res.intact()


@pytest.mark.parametrize("plan", [(128, 1), (256, 1)], ids=["128x1", "256x1"])
@pytest.mark.parametrize("form", ["bt", "kn", "dw"])
def test_sums_in_registers_for_16_bit_outputs(sk, planned, form, plan):
    """Past 8192 products 16-bit outputs take the sums in registers, in each form."""
    L = 8200 + 56
    g = gen(7)
    planned(*plan)
    T, N, K = (L - 3, 264, 136) if form == "dw" else (333, 264, L)
    a = randn(g, T, K).bfloat16()
    b = randn(g, *{"bt": (1, N, K), "kn": (1, K, N), "dw": (T, N)}[form]).bfloat16()
    _, offs = offsets_of([T])
    res = Guarded((1, N, K) if form == "dw" else (T, N), DT["f16"])
    call = {"bt": sk.gemm_grouped_bt, "kn": sk.gemm_grouped_kn, "dw": sk.gemm_grouped_dw}[form]
    call(a, b, offs, res.data, T, 1, N, K, "bf16", "f16")
    assert sk.splitk_get_device_status() == 0
    A, B = a.double(), b.double()
    left, right = {"bt": (A, B.mT), "kn": (A, B), "dw": (B.mT, A)}[form]
    got, right = (res.data[0], right) if form == "dw" else (res.data, right[0])
    check(got, left @ right, left.abs() @ right.abs(), c_16(L, "f32"), "f16")
    assert res.intact()


# ------------------------------------------------------------------ scales at the ends of the range

@pytest.mark.parametrize("M", [5, 130, 300])
def test_products_of_scales_at_the_ends_of_the_range(sk, M):
    """The two scales' product is formed in F32 first.  Where it is an ordinary
    number the result is as exact as ever, however large one scale and small the
    other; below 2^-126 it is within half of F32's smallest step, 2^-150; beyond
    the range it is infinite, and NaN against a sum of 0."""
    N, K = 200, 400
    g = gen(M)
    a, _ = fp8_rows(g, M, K)
    b, _ = fp8_weights(g, 1, N, K)
    b = b[0]
    a[0, 128:256] = 0
    pairs = [(1e30, 1e-30), (1e-37, 1e30), (2.0 ** -120, 2.0 ** -20), (2.0 ** -100, 2.0 ** -60), (1e25, 1e14)]
    for left, right in pairs:
        sa = (torch.rand(M, nblk(K), device="cuda", generator=g) + 0.5) * left
        sb = (torch.rand(nblk(N), nblk(K), device="cuda", generator=g) + 0.5) * right
        res = Guarded((M, N), torch.float32)
        sk.gemm_fp8_bt(a, sa, b, sb, res.data, M, N, K, "f32")
        A, B = real_rows(a, sa), real_weights(b, sb)
        if left * right > 3.5e38:
            assert not torch.isfinite(res.data).any() and torch.isnan(res.data[0]).all()
            continue
        codes = a.double().abs() @ b.double().abs().T
        tol = c_fp8(K) * 2.0 ** -23 * (A.abs() @ B.abs().T) + 2.0 ** -150 * codes + 2.0 ** -148
        assert bool(((res.data.double() - A @ B.T).abs() <= tol).all()), (left, right)
    assert sk.splitk_get_device_status() == 0


# ------------------------------------------------------------------ broken offsets over many runs

@pytest.mark.parametrize("form", ["bt", "fp8", "dw"])
@pytest.mark.parametrize("G", [33, 70, 129])
def test_broken_offsets_over_many_runs(sk, G, form):
    """Offsets that fall and leave [0, T], also across the 32 runs that a warp takes
    at a time: the runs are those of the clamped, rising sequence, rows outside
    them stay as they were, and the gradients of empty runs are zero."""
    T, N, K = 300, 136, 144
    g = gen(G)
    bad = torch.randint(0, 7, (G + 1,), generator=torch.Generator().manual_seed(G)).cumsum(0).tolist()
    bad[0] = 9
    bad[5] = -1000
    for i, v in ((30, 150), (31, 2 ** 31 - 1 if G == 33 else 160), (32, 20), (33, -2 ** 31), (63, 190), (64, 30), (128, 5)):
        if i < G:
            bad[i] = v
    offs = torch.tensor(bad, dtype=torch.int32, device="cuda")
    o = [min(max(x, 0), T) for x in bad]
    for i in range(1, len(o)):
        o[i] = max(o[i], o[i - 1])
    if form == "fp8":
        a, sa = fp8_rows(g, T, K)
        b, sb = fp8_weights(g, G, N, K)
        res = Guarded((T, N), torch.float32)
        sk.gemm_grouped_fp8_bt(a, sa, b, sb, offs, res.data, T, G, N, K, "f32")
        A, B = real_rows(a, sa), real_weights(b, sb)
    else:
        a, b, d = (randn(g, *s).bfloat16() for s in ((T, K), (G, N, K), (T, N)))
        A, B, D = a.double(), b.double(), d.double()
        if form == "bt":
            res = Guarded((T, N), torch.float32)
            sk.gemm_grouped_bt(a, b, offs, res.data, T, G, N, K, "bf16", "f32")
        else:
            res = Guarded((G, N, K), torch.float32)
            sk.gemm_grouped_dw(a, d, offs, res.data, T, G, N, K, "bf16", "f32")
    assert sk.splitk_get_device_status() == 0
    assert 0 < o[0] and len(runs(o)) >= 3
    for e, r in runs(o):
        if form == "dw":
            check(res.data[e], D[r].T @ A[r], D[r].abs().T @ A[r].abs(), c_16(T, "f32"), "f32")
        else:
            check(res.data[r], A[r] @ B[e].T, A[r].abs() @ B[e].abs().T, c_fp8(K) + 48, "f32")
    if form == "dw":
        for e in set(range(G)) - {e for e, _ in runs(o)}:
            assert not res.data[e].any()
    else:
        assert torch.isnan(res.data[:o[0]]).all() and torch.isnan(res.data[o[-1]:]).all()
    assert res.intact()


# ------------------------------------------------------------------ beside the split-K calls, streams, threads

class Chain:
    """Split-K product -> norm to 8 bits -> 8-bit product -> split-K product ->
    rows to 8 bits -> grouped product: each reads what the one before wrote."""

    M, D = 128, 512
    COUNTS = [50, 0, 78]

    def __init__(self, sk, seed):
        g = gen(seed)
        M, D = self.M, self.D
        self.sk = sk
        self.x = randn(g, M, D).bfloat16()
        self.b1, self.b2 = ((randn(g, D, D) * D ** -0.5).bfloat16() for _ in range(2))
        self.w = (1 + 0.1 * randn(g, D))
        self.b3, self.s3 = fp8_weights(g, 1, D, D)
        self.b4, self.s4 = fp8_weights(g, len(self.COUNTS), D, D)
        _, self.offs = offsets_of(self.COUNTS)
        self.nbytes = sk.gemm_bt_workspace_bytes(M, D, D, 2, D // 2)
        self.ws = torch.empty(self.nbytes // 4, device="cuda")
        sk.gemm_bt_workspace_init(self.ws, self.nbytes)
        self.mid = [torch.empty(M, D, device="cuda"), torch.empty(M, D, dtype=E4M3, device="cuda"),
                    torch.empty(M, nblk(D), device="cuda"), torch.empty(M, D, dtype=torch.bfloat16, device="cuda")]
        self.out = torch.empty(M, D, device="cuda")

    def run(self, fused=1, wait=lambda: None, stream=None):
        sk, M, D = self.sk, self.M, self.D
        c, q, s, h = self.mid
        steps = (
            lambda: sk.gemm_bt(self.x, self.b1, c, self.ws, self.nbytes, M, D, D, 2, D // 2, "bf16", fused=fused, stream=stream),
            lambda: sk.rmsnorm_fp8(c, self.w, q, s, M, D, "f32", stream=stream),
            lambda: sk.gemm_fp8_bt(q, s, self.b3, self.s3, h, M, D, D, "bf16", stream=stream),
            lambda: sk.gemm_bt(h, self.b2, c, self.ws, self.nbytes, M, D, D, 2, D // 2, "bf16", fused=fused, stream=stream),
            lambda: sk.fp8_quantize(c, q, s, M, D, "f32", stream=stream),
            lambda: sk.gemm_grouped_fp8_bt(q, s, self.b4, self.s4, self.offs, self.out, M, len(self.COUNTS), D, D, "f32",
                                           stream=stream),
        )
        for step in steps:
            step()
            wait()

    def poison(self):
        for t in (*self.mid, self.out):
            t.view(torch.uint8).fill_(0xFF)


@pytest.mark.parametrize("fused", [0, 1, 3])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_split_k_and_8_bit_calls_feed_one_another(sk, mode, fused):
    """Every buffer is written and read again within the capture, so a launch that
    started before its input was there, or wrote over what was still read, shows."""
    chain = Chain(sk, 31)
    chain.poison()
    chain.run(fused, wait=torch.cuda.synchronize)
    want = chain.out.clone()
    assert torch.isfinite(want).all()
    sk.splitk_set_overlap(mode)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                chain.run(fused)
    finally:
        sk.splitk_set_overlap(2)
    for _ in range(5):
        chain.poison()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(chain.out, want)
    chain.poison()
    for _ in range(3):
        chain.run(fused)
    torch.cuda.synchronize()
    assert torch.equal(chain.out, want)
    assert sk.splitk_get_device_status() == 0


def test_streams_side_by_side(sk):
    chains = [Chain(sk, 40 + i) for i in range(3)]
    want = []
    for c in chains:
        c.run(wait=torch.cuda.synchronize)
        want.append(c.out.clone())
        c.poison()
    streams = [torch.cuda.Stream() for _ in chains]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(chains, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        assert torch.equal(c.out, w)
    assert sk.splitk_get_device_status() == 0


def test_threads_side_by_side(sk):
    import threading

    chains = [Chain(sk, 50 + i) for i in range(4)]
    want, errors = [], []
    for c in chains:
        c.run(wait=torch.cuda.synchronize)
        want.append(c.out.clone())
        c.poison()
    torch.cuda.synchronize()

    def work(c):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                c.run(stream=stream)
            stream.synchronize()
        except BaseException as e:   # noqa: B036 -- reported by the test
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in chains]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for c, w in zip(chains, want):
        assert torch.equal(c.out, w)
    assert sk.splitk_get_device_status() == 0

"""The 8-bit and grouped operators on the GPU against their definitions in 64 bits.

Tolerances.  The tensor cores form products exactly and may drop the bits of a
step's terms below the F32 sum's last place: per step of 16 or 32 values at
most one unit, 2^-23 of the magnitudes summed so far, plus as much for each of
the step's terms.  A unit of k-blocks (8 of them, 32 steps; one of 4 steps with
8-bit operands) goes to F32 sums rounded to nearest.  So an F32 output is within
c 2^-23 sum|a b|, c = 32 + 16 + K / 512 (16 bits) or 4 + 32 + K / 128 + 2 (8 bits: the
scales' product and the scaled addition round too); a 16-bit output of 16-bit
operands (one accumulator) c = K / 16 + 16.  A 16-bit output adds half a unit of
its last place.  Integer operands whose sums stay below 2^24 are exact.
"""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BLOCK = 128
E4M3 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}     # of |result|, with room for a tie
TINY = {"f32": 0.0, "f16": 2.0 ** -24, "bf16": 0.0}                # F16's subnormal step


@pytest.fixture(scope="module", autouse=True)
def sk():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import split_bf16_gemm_gb300 as sk

    sk.build()
    yield sk


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


class Guarded:
    """An output of `shape` between guard bytes, poisoned with NaN patterns."""

    def __init__(self, shape, dtype):
        n = 1
        for d in shape:
            n *= d
        size = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((n * size + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        self.raw[:256] = 0xA5
        self.raw[256 + n * size:] = 0xA5
        self.end = 256 + n * size
        self.data = self.raw[256:self.end].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:256] == 0xA5).all() and (self.raw[self.end:] == 0xA5).all())


def nblk(n):
    return (n + BLOCK - 1) // BLOCK


def spread(scales, n, dim):
    return scales.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def fp8_rows(g, m, k):
    q = (randn(g, m, k) * 60).clamp(-448, 448).to(E4M3)
    return q, (torch.rand(m, nblk(k), device="cuda", generator=g) + 0.5) * 0.01


def fp8_weights(g, e, n, k):
    q = (randn(g, e, n, k) * 60).clamp(-448, 448).to(E4M3)
    return q, (torch.rand(e, nblk(n), nblk(k), device="cuda", generator=g) + 0.5) * 0.01


def real_rows(q, s):
    return q.double() * spread(s.double(), q.shape[-1], -1)


def real_weights(q, s):
    return q.double() * spread(spread(s.double(), q.shape[-2], -2), q.shape[-1], -1)


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return o, torch.tensor(o, dtype=torch.int32, device="cuda")


def check(got, ref, mag, c, out):
    """Every element within c 2^-23 mag, plus the output type's rounding."""
    tol = c * 2.0 ** -23 * mag * (1 + HALF_UNIT[out]) + HALF_UNIT[out] * ref.abs() + TINY[out]
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(((got.double() - ref).abs() - tol).max()))


def c_fp8(K):
    return 4 + 32 + K / 128 + 2


def c_16(K, out):
    return 32 + 16 + K / 512 if out == "f32" else K / 16 + 16


# ------------------------------------------------------------------ the product in 8 bits

FP8_SHAPES = [(1, 1, 16), (1, 64, 128), (1, 1024, 2048), (3, 129, 144), (16, 130, 272), (17, 257, 400), (31, 64, 16),
              (33, 200, 1040), (64, 512, 2048), (65, 127, 640), (127, 384, 160), (128, 128, 128), (129, 129, 129 * 16),
              (200, 1000, 528), (257, 255, 1024), (300, 640, 7168), (513, 1025, 272), (1000, 2112, 5136),
              (2049, 520, 656), (2049, 2600, 656), (4100, 1300, 144), (1300, 4105, 1040)]


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", FP8_SHAPES)
def test_fp8_product(sk, M, N, K, out):
    g = gen(M * 7 + N * 3 + K)
    a, sa = fp8_rows(g, M, K)
    b, sb = fp8_weights(g, 1, N, K)
    b, sb = b[0], sb[0]
    res = Guarded((M, N), DT[out])
    sk.gemm_fp8_bt(a, sa, b, sb, res.data, M, N, K, out)
    assert sk.splitk_get_device_status() == 0
    A, B = real_rows(a, sa), real_weights(b, sb)
    check(res.data, A @ B.T, A.abs() @ B.abs().T, c_fp8(K), out)
    assert res.intact()


@pytest.mark.parametrize("M,N,K", [(5, 300, 528), (150, 300, 528), (400, 700, 1040)])
def test_fp8_integers_are_exact(sk, M, N, K):
    g = gen(3)
    a = torch.randint(-8, 9, (M, K), device="cuda", generator=g).float().to(E4M3)
    b = torch.randint(-8, 9, (N, K), device="cuda", generator=g).float().to(E4M3)
    sa = torch.randint(1, 3, (M, nblk(K)), device="cuda", generator=g).float()
    sb = torch.randint(1, 3, (nblk(N), nblk(K)), device="cuda", generator=g).float()
    res = Guarded((M, N), torch.float32)
    sk.gemm_fp8_bt(a, sa, b, sb, res.data, M, N, K, "f32")
    assert torch.equal(res.data.double(), real_rows(a, sa) @ real_weights(b, sb).T)


@pytest.mark.parametrize("M", [4, 200, 300])
def test_fp8_nan_stays_in_its_row(sk, M):
    N, K = 300, 528
    g = gen(8)
    a, sa = fp8_rows(g, M, K)
    b, sb = fp8_weights(g, 1, N, K)
    clean, dirty = Guarded((M, N), torch.float32), Guarded((M, N), torch.float32)
    sk.gemm_fp8_bt(a, sa, b, sb, clean.data, M, N, K, "f32")
    a.view(torch.uint8)[1, 5] = 0x7F                      # NaN
    sa[2, 1] = float("inf")
    sk.gemm_fp8_bt(a, sa, b, sb, dirty.data, M, N, K, "f32")
    assert torch.isnan(dirty.data[1]).all()
    assert not torch.isfinite(dirty.data[2]).any()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(dirty.data[keep], clean.data[keep])


# ------------------------------------------------------------------ grouped products

GROUPED = [  # counts, N, K, rows before the first run and after the last
    ([1], 8, 8, 0, 0),
    ([5], 136, 72, 0, 0),
    ([0, 3, 0, 0, 1, 17, 0], 200, 264, 0, 0),
    ([1] * 40, 72, 520, 0, 0),
    ([0, 0, 0], 64, 64, 0, 0),
    ([16, 32, 48, 15, 31, 33], 256, 512, 3, 5),
    ([130, 0, 1, 255, 64, 129], 264, 200, 0, 7),
    ([300], 1000, 1544, 11, 0),
    ([700, 1, 0, 40, 513], 392, 648, 1, 2),
    ([129] * 9, 512, 1032, 0, 0),
    ([1500, 600], 1160, 2056, 0, 0),
    ([1500, 0, 700, 257, 1, 640], 1800, 264, 4, 3),
    ([500, 900, 333], 2600, 2056, 0, 0),
    ([0] * 500 + [7] + [0] * 300 + [50] + [2] * 222, 72, 136, 0, 0),
]
GROUPED_IDS = [f"G{len(c)}T{sum(c)}N{n}K{k}" for c, n, k, _, _ in GROUPED]


def runs(o):
    return [(g, slice(o[g], o[g + 1])) for g in range(len(o) - 1) if o[g + 1] > o[g]]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,N,K,before,after", GROUPED, ids=GROUPED_IDS)
def test_grouped_fp8(sk, counts, N, K, before, after, out):
    K = K // 16 * 16 + 16
    N = N + 1
    G, T = len(counts), sum(counts) + before + after
    g = gen(T + N + K)
    a, sa = fp8_rows(g, max(T, 1), K)
    b, sb = fp8_weights(g, G, N, K)
    o, offs = offsets_of(counts, before)
    res = Guarded((T, N), DT[out])
    sk.gemm_grouped_fp8_bt(a, sa, b, sb, offs, res.data, T, G, N, K, out)
    assert sk.splitk_get_device_status() == 0
    A, B = real_rows(a, sa), real_weights(b, sb)
    for e, r in runs(o):
        check(res.data[r], A[r] @ B[e].T, A[r].abs() @ B[e].abs().T, c_fp8(K), out)
    assert torch.isnan(res.data[:o[0]]).all() and torch.isnan(res.data[o[-1]:]).all()   # left as they were
    assert res.intact()


@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("layout", ["bt", "kn"])
@pytest.mark.parametrize("counts,N,K,before,after", GROUPED, ids=GROUPED_IDS)
def test_grouped_16(sk, counts, N, K, before, after, layout, dt, out):
    if layout == "bt":
        N = N + 3
    G, T = len(counts), sum(counts) + before + after
    g = gen(T + N + K)
    a = randn(g, T, K).to(DT[dt])
    w = randn(g, G, *((N, K) if layout == "bt" else (K, N))).to(DT[dt])
    o, offs = offsets_of(counts, before)
    res = Guarded((T, N), DT[out])
    call = sk.gemm_grouped_bt if layout == "bt" else sk.gemm_grouped_kn
    call(a, w, offs, res.data, T, G, N, K, dt, out)
    assert sk.splitk_get_device_status() == 0
    A, W = a.double(), (w if layout == "kn" else w.mT).double()
    for e, r in runs(o):
        check(res.data[r], A[r] @ W[e], A[r].abs() @ W[e].abs(), c_16(K, out), out)
    assert torch.isnan(res.data[:o[0]].float()).all() and torch.isnan(res.data[o[-1]:].float()).all()
    assert res.intact()


@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("counts,N,K,before,after", GROUPED, ids=GROUPED_IDS)
def test_grouped_weight_gradient(sk, counts, N, K, before, after, dt, out):
    G, T = len(counts), sum(counts) + before + after
    g = gen(T + N + K)
    a, d = randn(g, max(T, 1), K).to(DT[dt]), randn(g, max(T, 1), N).to(DT[dt])
    a[:before], d[:before] = float("nan"), float("inf")      # rows outside the runs take no part
    a[T - after:T], d[T - after:T] = float("inf"), float("nan")
    o, offs = offsets_of(counts, before)
    res = Guarded((G, N, K), DT[out])
    sk.gemm_grouped_dw(a, d, offs, res.data, T, G, N, K, dt, out)
    assert sk.splitk_get_device_status() == 0
    A, D = a.double(), d.double()
    there = {e for e, _ in runs(o)}
    for e, r in runs(o):
        check(res.data[e], D[r].T @ A[r], D[r].abs().T @ A[r].abs(), c_16(counts[e], out), out)
    for e in set(range(G)) - there:
        assert not res.data[e].any()
    assert res.intact()


@pytest.mark.parametrize("counts", [[3, 0, 14], [40, 7, 0, 150]])
def test_weight_gradient_takes_nothing_from_the_next_run(sk, counts):
    N, K, G, T = 136, 200, len(counts), sum(counts)
    g = gen(1)
    a, d = randn(g, T, K).bfloat16(), randn(g, T, N).bfloat16()
    o, offs = offsets_of(counts)
    clean, dirty = Guarded((G, N, K), torch.float32), Guarded((G, N, K), torch.float32)
    sk.gemm_grouped_dw(a, d, offs, clean.data, T, G, N, K, "bf16", "f32")
    a[o[-2]:], d[o[-2]:] = float("nan"), float("inf")
    sk.gemm_grouped_dw(a, d, offs, dirty.data, T, G, N, K, "bf16", "f32")
    assert torch.equal(dirty.data[:-1], clean.data[:-1])
    assert torch.isnan(dirty.data[-1]).all()


def test_gradients_against_differences(sk):
    """L = sum(out * D) is linear in A and in B: with small whole numbers every
    sum is exact, so (L(B + E) - L(B - E)) / 2 equals <dB, E> to the last bit."""
    counts, N, K = [9, 0, 70, 33], 72, 136
    G, T = len(counts), sum(counts)
    g = gen(4)

    def ints(*shape):
        return torch.randint(-3, 4, shape, device="cuda", generator=g).bfloat16()

    a, b, d, ea, eb = ints(T, K), ints(G, N, K), ints(T, N), ints(T, K), ints(G, N, K)
    _, offs = offsets_of(counts)

    def loss(a, b):
        out = torch.empty(T, N, device="cuda")
        sk.gemm_grouped_bt(a, b, offs, out, T, G, N, K, "bf16", "f32")
        return float((out.double() * d.double()).sum())

    da, db = torch.empty(T, K, device="cuda"), torch.empty(G, N, K, device="cuda")
    sk.gemm_grouped_kn(d, b, offs, da, T, G, K, N, "bf16", "f32")
    sk.gemm_grouped_dw(a, d, offs, db, T, G, N, K, "bf16", "f32")
    assert (loss(a, b + eb) - loss(a, b - eb)) / 2 == float((db.double() * eb.double()).sum())
    assert (loss(a + ea, b) - loss(a - ea, b)) / 2 == float((da.double() * ea.double()).sum())


@pytest.mark.parametrize("bad", [[0, 50, 20, 60], [-5, 10, 90, 1000], [70, 60, 50, 40], [2 ** 31 - 1, -2 ** 31, 5, 64]])
@pytest.mark.parametrize("form", ["bt", "fp8", "dw"])
def test_broken_offsets_stay_in_bounds(sk, bad, form):
    # clamped to a rising sequence within [0, T]
    T, G, N, K = 64, 3, 136, 144
    g = gen(2)
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
    for e, r in runs(o):
        if form == "dw":
            check(res.data[e], D[r].T @ A[r], D[r].abs().T @ A[r].abs(), c_16(T, "f32"), "f32")
        else:
            check(res.data[r], A[r] @ B[e].T, A[r].abs() @ B[e].abs().T, c_fp8(K) + 48, "f32")
    assert res.intact()


def test_weight_gradient_without_rows(sk):
    res = Guarded((3, 72, 136), torch.float32)
    a, d = (torch.empty(0, n, device="cuda", dtype=torch.bfloat16) for n in (136, 72))
    sk.gemm_grouped_dw(a, d, torch.zeros(4, dtype=torch.int32, device="cuda"), res.data, 0, 3, 72, 136, "bf16", "f32")
    assert not res.data.any() and res.intact()


# ------------------------------------------------------------------ rows and weights to 8 bits

def e4m3_step(x):
    """Spacing of E4M3 around |x| (steps no finer than 2^-9)."""
    return torch.exp2((torch.frexp(x).exponent - 4).clamp_min(-9).double())


def check_rows(y, q, s, rel):
    """q and s stand for y [M,K] (64 bits), whose F32 values are within `rel`."""
    M, K = y.shape
    pad = torch.nn.functional.pad(y, (0, nblk(K) * BLOCK - K)).view(M, -1, BLOCK)
    ref = (pad.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    assert bool(((s.double() - ref).abs() <= (rel + 2.0 ** -23) * ref).all())
    want = y / spread(ref, K, -1)
    off = (q.double() - want).abs()
    assert bool((off <= e4m3_step(want) / 2 + (2 * rel + 2.0 ** -22) * want.abs()).all())


NORMS = [(1, 16), (1, 128), (3, 144), (5, 1024), (7, 1040), (2, 2048), (333, 4096), (9, 4112), (4, 8192), (3, 8208),
         (2, 16384), (2, 16400), (3, 40000), (1, 100000)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual,y", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("M,K", NORMS)
def test_norm(sk, M, K, dt, residual, y):
    g = gen(M + K)
    x, r = (randn(g, M, K) * 2).to(DT[dt]), randn(g, M, K).to(DT[dt])
    w = (1 + 0.2 * randn(g, K)).to(DT[dt])
    q, s = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32)
    out, h = Guarded((M, K), DT[dt]), Guarded((M, K), DT[dt])
    sk.rmsnorm_fp8(x, w, q.data, s.data, M, K, dt, eps=1e-5, residual=r if residual else None,
                   sum_out=h.data if residual else None, y=out.data if y else None)
    want = (x.float() + r.float()).to(DT[dt]) if residual else x
    if residual:
        assert torch.equal(h.data, want)
    H = want.double()
    ref = H / (H.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w.double()
    # the sum of squares: at most 8 * turns + 10 roundings of positive terms, halved by the root
    rel = (8 * (K // 4096 + 1) * 4 + 10 + 6) * 2.0 ** -24
    check_rows(ref, q.data, s.data, rel)
    if y:
        tol = (rel + HALF_UNIT[dt]) * ref.abs() + TINY[dt]
        assert bool(((out.data.double() - ref).abs() <= tol).all())
    assert q.intact() and s.intact() and out.intact() and h.intact()


@pytest.mark.parametrize("K", [256, 20000])
@pytest.mark.parametrize("where", ["x", "residual"])
def test_norm_in_place(sk, K, where):
    M = 6
    g = gen(K)
    x, r, w = randn(g, M, K).bfloat16(), randn(g, M, K).bfloat16(), randn(g, K).bfloat16()
    outs = [(Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32)) for _ in range(2)]
    h = torch.empty_like(x)
    sk.rmsnorm_fp8(x, w, outs[0][0].data, outs[0][1].data, M, K, "bf16", residual=r, sum_out=h)
    kept = x if where == "x" else r
    sk.rmsnorm_fp8(x, w, outs[1][0].data, outs[1][1].data, M, K, "bf16", residual=r, sum_out=kept)
    assert torch.equal(kept, h)
    assert torch.equal(outs[0][0].data.view(torch.uint8), outs[1][0].data.view(torch.uint8))
    assert torch.equal(outs[0][1].data, outs[1][1].data)


def test_norm_of_zeros_and_non_finite_rows(sk):
    M, K = 5, 512
    g = gen(6)
    x, w = randn(g, M, K), torch.ones(K, device="cuda")
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 300] = float("inf")
    x[3] = 1e-30                                          # eps decides
    q, s = Guarded((M, K), E4M3), Guarded((M, 4), torch.float32)
    sk.rmsnorm_fp8(x, w, q.data, s.data, M, K, "f32", eps=1e-6)
    assert not q.data[0].float().any() and bool((s.data[0] == 2.0 ** -126).all())
    for i in (1, 2):
        product = q.data[i].float() * spread(s.data[i], K, 0)
        assert torch.isnan(product[128 * (0 if i == 1 else 2):][:128]).all()
    ref = x[3:].double() / (x[3:].double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
    check_rows(ref, q.data[3:], s.data[3:], 64 * 2.0 ** -24)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (4, 400), (37, 2048), (2, 30000)])
def test_quantize_rows(sk, M, K, dt):
    x = (randn(gen(K), M, K) * 3).to(DT[dt])
    x[0, :16] = 0
    q, s = Guarded((M, K), E4M3), Guarded((M, nblk(K)), torch.float32)
    sk.fp8_quantize(x, q.data, s.data, M, K, dt)
    check_rows(x.double(), q.data, s.data, 0.0)
    assert q.intact() and s.intact()


def test_quantize_keeps_codes_that_fit(sk):
    # values that are E4M3 numbers times a power of two, the largest 448 of them: exact
    K = 256
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(E4M3).float()
    codes = torch.nan_to_num(codes, nan=448.0)
    x = torch.stack([codes * 2.0 ** e for e in (-20, 0, 13)])
    q, s = Guarded((3, K), E4M3), Guarded((3, 2), torch.float32)
    sk.fp8_quantize(x, q.data, s.data, 3, K, "f32")
    assert torch.equal(q.data.float() * spread(s.data, K, 1), x)


def test_quantize_non_finite(sk):
    x = torch.ones(2, 256, device="cuda")
    x[0, 3], x[1, 200] = float("nan"), float("inf")
    q, s = Guarded((2, 256), E4M3), Guarded((2, 2), torch.float32)
    sk.fp8_quantize(x, q.data, s.data, 2, 256, "f32")
    assert torch.isnan(s.data[0, 0]) and torch.isnan(q.data[0, :128].float()).all()
    assert torch.isinf(s.data[1, 1]) and torch.isnan(q.data[1, 200].float())
    assert bool((s.data[0, 1] == s.data[1, 0]).all()) and bool((q.data[1, :128].float() == 448).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (1, 128, 128), (3, 130, 272), (2, 500, 1040)])
def test_prepare_weights(sk, G, N, K, dt):
    b = randn(gen(N), G, N, K).to(DT[dt])
    q, s = Guarded((G, N, K), E4M3), Guarded((G, nblk(N), nblk(K)), torch.float32)
    sk.fp8_prepare_bt(b, q.data, s.data, G, N, K, dt)
    B = b.double()
    pad = torch.nn.functional.pad(B, (0, nblk(K) * BLOCK - K, 0, nblk(N) * BLOCK - N))
    ref = pad.view(G, nblk(N), BLOCK, nblk(K), BLOCK).abs().amax((2, 4)) / 448
    assert bool(((s.data.double() - ref).abs() <= 2.0 ** -23 * ref).all())
    want = B / spread(spread(ref, N, 1), K, 2)
    assert bool(((q.data.double() - want).abs() <= e4m3_step(want) / 2 + 2.0 ** -22 * want.abs()).all())
    assert q.intact() and s.intact()


# ------------------------------------------------------------------ streams, graphs, repetition

def chain(sk, x, r, w, b, sb, offs, bufs, T, G, N, K, stream=None):
    h, q, s, out = bufs
    sk.rmsnorm_fp8(x, w, q, s, T, K, "bf16", residual=r, sum_out=h, stream=stream)
    sk.gemm_grouped_fp8_bt(q, s, b, sb, offs, out, T, G, N, K, "f32", stream=stream)


@pytest.mark.parametrize("counts,N,K", [([3, 0, 9], 520, 1024), ([200, 90, 0, 130], 520, 1024)])
def test_chain_on_a_stream_in_a_graph_and_again(sk, counts, N, K):
    """Norm then product: dependent launches give the same bits eagerly, on another
    stream, and replayed from a graph."""
    G, T = len(counts), sum(counts)
    g = gen(12)
    x, r, w = randn(g, T, K).bfloat16(), randn(g, T, K).bfloat16(), randn(g, K).bfloat16()
    b, sb = fp8_weights(g, G, N, K)
    _, offs = offsets_of(counts)

    def bufs():
        return (torch.empty_like(x), torch.empty(T, K, dtype=E4M3, device="cuda"),
                torch.empty(T, nblk(K), device="cuda"), torch.full((T, N), float("nan"), device="cuda"))

    one = bufs()
    chain(sk, x, r, w, b, sb, offs, one, T, G, N, K)
    torch.cuda.synchronize()
    assert torch.isfinite(one[3]).all()
    side = torch.cuda.Stream()
    two = bufs()
    torch.cuda.synchronize()
    for _ in range(5):
        chain(sk, x, r, w, b, sb, offs, two, T, G, N, K, stream=side)
    side.synchronize()
    assert torch.equal(one[3], two[3])
    three = bufs()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain(sk, x, r, w, b, sb, offs, three, T, G, N, K)
        chain(sk, x, r, w, b, sb, offs, three, T, G, N, K)
    for _ in range(3):
        three[3].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(one[3], three[3])
    assert sk.splitk_get_device_status() == 0


def test_beside_the_split_k_product(sk):
    """Launches of both kinds alternate on one stream, eagerly and captured."""
    M, N, K, S, kps = 256, 1024, 2048, 2, 1024
    g = gen(5)
    A, B = randn(g, M, K).bfloat16(), randn(g, N, K).bfloat16()
    a, sa = fp8_rows(g, M, K)
    b, sb = fp8_weights(g, 1, N, K)
    nbytes = sk.gemm_bt_workspace_bytes(M, N, K, S, kps)
    ws = torch.empty(nbytes // 4, device="cuda")

    def both(o1, o2):
        for _ in range(4):
            sk.gemm_bt(A, B, o1, ws, nbytes, M, N, K, S, kps, "bf16", fused=1)
            sk.gemm_fp8_bt(a, sa, b, sb, o2, M, N, K, "f32")

    e1, e2, c1, c2 = (torch.empty(M, N, device="cuda") for _ in range(4))
    sk.gemm_bt(A, B, e1, ws, nbytes, M, N, K, S, kps, "bf16", fused=1)
    torch.cuda.synchronize()
    sk.gemm_fp8_bt(a, sa, b, sb, e2, M, N, K, "f32")
    torch.cuda.synchronize()
    both(c1, c2)
    torch.cuda.synchronize()
    assert torch.equal(e1, c1) and torch.equal(e2, c2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(c1, c2)
    c1.zero_(), c2.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(e1, c1) and torch.equal(e2, c2)
    assert sk.splitk_get_device_status() == 0


@pytest.mark.parametrize("tokens,experts", [(1, 8), (37, 16), (700, 4)])
def test_example_block(sk, tokens, experts):
    """The example against the same block in 32 bits.  E4M3 keeps four significant
    bits: a value is off by at most 2^-4 of itself, 2^-4 / sqrt(3) on average, and
    four such errors (activations and weights of two products; the gated product
    passes its first factor's error on about twice) add to about 0.1."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(tokens, experts, hidden=1024, inner=512) < 0.1

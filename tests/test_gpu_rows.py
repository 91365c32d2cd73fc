"""Routing and rows sorted by expert and back, on the GPU against their definitions
in 64 bits.  Whole numbers and copies are equal; the tolerances of the others stand
with each test: U = 2^-24 is half a step of F32, and sums of n terms in F32 are
within (n - 1) U of the terms' magnitudes."""
import importlib.util
import math
import os
import threading

import pytest

torch = pytest.importorskip("torch")

import rows_reference as ref  # noqa: E402
from rows_reference import DT, U, within  # noqa: E402
from test_gpu_fp8_grouped import E4M3, Guarded, gen, nblk, randn, sk  # noqa: E402,F401

pytestmark = pytest.mark.gpu
INT = torch.int32


def guarded(shape, dtype, fill=None):
    g = Guarded(shape, dtype)
    if fill is not None:
        g.data.fill_(fill)
    return g


# ------------------------------------------------------------------ the router's choice

def route_tolerance(logits, p, experts=None):
    """exp within 2 units (4 U) of its rounded argument l - m, off by U |l - m|; a sum
    of at most 32 + 5 terms in a row, the quotient 3 U."""
    l = logits.double().cpu()
    m = torch.where(l.isinf(), -math.inf, l).amax(1, keepdim=True)
    far = torch.where(l > -math.inf, m - l, 0.0)
    worst = (p * far).sum(1, keepdim=True)
    return U * (64 + far + worst)


ROUTES = [(1, 1, 1), (1, 2, 1), (3, 8, 8), (5, 31, 4), (64, 32, 4), (33, 33, 2), (7, 64, 6), (130, 100, 3), (9, 128, 8), (257, 160, 8),
          (12, 256, 8), (6, 257, 32), (5, 500, 7), (4, 512, 32), (3, 1000, 5), (2, 1024, 32), (40, 16, 16), (11, 24, 9), (11, 48, 12), (6, 65, 17)]


@pytest.mark.parametrize("chosen_only", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,G,top", ROUTES)
def test_route_and_its_gradient(sk, M, G, top, dtype, chosen_only):
    g = gen(M * 31 + G)
    logits = 3 * randn(g, M, G)
    if G > 4:
        logits[torch.rand(M, G, device="cuda", generator=g) < 0.2] = -math.inf
    if M > 2:
        logits[1] = -math.inf                       # a padded token
        logits[2] = logits[2].round()               # many equal logits
    logits = logits.to(DT[dtype]).contiguous()
    e, s, d = guarded((M, top), INT), guarded((M, top), torch.float32), guarded((M, G), DT[dtype])
    sk.moe_route(logits, e.data, s.data, M, G, top, dtype, chosen_only=chosen_only)
    experts, shares, p = ref.route(logits.cpu(), top, chosen_only)
    assert torch.equal(e.data.cpu().long(), experts)
    at = experts.clamp(min=0)
    tol = route_tolerance(logits, p)
    within(s.data, shares, shares * tol.gather(1, at))
    ds = randn(g, M, top)
    sk.moe_route_grad(logits, e.data, ds, d.data, M, G, top, dtype, chosen_only=chosen_only)
    grad = ref.route_grad(p, experts, ds.cpu().double())
    # p, the products p d (as many as choices, added), and the difference
    size = ds.cpu().double().abs()
    inner = (p.gather(1, at) * (experts >= 0) * size).sum(1, keepdim=True)
    own = torch.zeros_like(p).scatter_add(1, at, size * (experts >= 0))
    within(d.data, grad, p * (own + inner) * (2 * tol.amax(1, keepdim=True) + 16 * U), dtype)
    assert e.intact() and s.intact() and d.intact()


def test_route_gradient_by_differences(sk):
    M, G, top = 3, 13, 4
    g = gen(5)
    logits, d = randn(g, M, G), randn(g, M, top)
    e, s, dl = (torch.empty(M, top, dtype=INT, device="cuda"), torch.empty(M, top, device="cuda"), torch.empty(M, G, device="cuda"))
    for chosen_only in (False, True):
        sk.moe_route(logits, e, s, M, G, top, "f32", chosen_only=chosen_only)
        sk.moe_route_grad(logits, e, d, dl, M, G, top, "f32", chosen_only=chosen_only)
        at = e.cpu().long()

        def loss(l):
            p = torch.softmax(l.gather(1, at) if chosen_only else l, 1)
            return ((p if chosen_only else p.gather(1, at)) * d.cpu().double()).sum()

        # shares have third derivatives of at most 6 |d|: 6 * 4 * 3 * 1e-10 / 6; rounding 1e-15 / 1e-5
        want = ref.differences(loss, logits.cpu())
        within(dl, want, torch.full_like(want, 1e-8) + 256 * U * float(d.abs().sum()))


def test_route_ties_zeros_and_types(sk):
    for dtype in ("f32", "f16", "bf16"):
        logits = torch.tensor([[0.0, -0.0, 0.0, -0.0, -1.0, 0.0], [-0.0, 0.0, 5.0, 5.0, -math.inf, 5.0]], device="cuda").to(DT[dtype])
        e, s = torch.empty(2, 4, dtype=INT, device="cuda"), torch.empty(2, 4, device="cuda")
        sk.moe_route(logits, e, s, 2, 6, 4, dtype)
        assert e.tolist() == [[0, 1, 2, 3], [2, 3, 5, 0]]
        sk.moe_route(logits, e, s, 2, 6, 4, dtype, chosen_only=True)
        assert s[0].tolist() == [0.25] * 4


@pytest.mark.parametrize("G", [8, 40, 64, 100, 256, 500, 1024])
def test_route_of_equal_logits(sk, G):
    """As a router whose weights are zeros gives them; and groups of equal ones."""
    M = 5
    for top in (1, 4, 8, min(G, 32)):
        logits = torch.zeros(M, G, device="cuda")
        logits[1] = (torch.arange(G, device="cuda") % 3).float()
        logits[2, G // 2:] = -math.inf
        logits[3] = torch.arange(G, device="cuda") // 40
        logits[4, ::2] = -0.0
        e, s = torch.empty(M, top, dtype=INT, device="cuda"), torch.empty(M, top, device="cuda")
        sk.moe_route(logits, e, s, M, G, top, "f32")
        experts, shares, p = ref.route(logits.cpu(), top, False)
        assert torch.equal(e.cpu().long(), experts)
        within(s, shares, shares * route_tolerance(logits, p).gather(1, experts.clamp(min=0)))


def test_route_extremes(sk):
    inf, nan = math.inf, math.nan
    rows = [[nan, 1.0, 2.0, inf], [1.0, inf, 0.0, inf], [3e38, -3e38, 0.0, -inf], [-inf, -inf, -3e38, -inf], [1e-45, 0.0, -1e-45, -inf]]
    logits = torch.tensor(rows, device="cuda")
    M, G, top = len(rows), 4, 3
    e, s, d = torch.empty(M, top, dtype=INT, device="cuda"), torch.empty(M, top, device="cuda"), torch.empty(M, G, device="cuda")
    sk.moe_route(logits, e, s, M, G, top, "f32")
    assert e.tolist() == [[0, 3, 2], [1, 3, 0], [0, 2, 1], [2, -1, -1], [0, 1, 2]]
    assert s[:2].isnan().all()
    assert s[2].tolist() == [1.0, 0.0, 0.0] and s[3].tolist() == [1.0, 0.0, 0.0]
    within(s[4], torch.full((3,), 1 / 3.0, dtype=torch.float64), torch.full((3,), 8 * U / 3))
    sk.moe_route_grad(logits, e, torch.ones_like(s), d, M, G, top, "f32")
    assert d[:2].isnan().all() and d[2:4].eq(0).all() and d[4].abs().max() < 16 * U


@pytest.mark.parametrize("dtype,bits", [("f32", (0x7fc00000, -0x400000, 0x7f800001, -1)), ("f16", (0x7e00, -0x200, 0x7c01, -1)), ("bf16", (0x7fc0, -0x40, 0x7f81, -1))])
@pytest.mark.parametrize("G", [9, 200])
def test_route_takes_any_nan_for_the_largest(sk, G, dtype, bits):
    whole = {"f32": torch.int32, "f16": torch.int16, "bf16": torch.int16}[dtype]
    for b in bits:
        logits = randn(gen(1), 3, G).to(DT[dtype])
        logits[:, 3] = math.inf
        logits.view(whole)[1, 7] = b
        e, s = torch.empty(3, 4, dtype=INT, device="cuda"), torch.empty(3, 4, device="cuda")
        sk.moe_route(logits, e, s, 3, G, 4, dtype)
        assert e[:, 0].tolist() == [3, 7, 3] and e[1, 1] == 3 and s.isnan().all()


def test_route_gradient_of_repeated_and_foreign_experts(sk):
    """An expert that is there twice counts twice; one outside [0, G) is passed over."""
    M, G, top = 2, 6, 5
    logits, d = randn(gen(1), M, G), randn(gen(2), M, top)
    e = torch.tensor([[3, 3, 1, 3, 1], [7, -5, 2, 2, 2 ** 31 - 1]], dtype=INT, device="cuda")
    dl = torch.empty(M, G, device="cuda")
    for chosen_only in (False, True):
        sk.moe_route_grad(logits, e, d, dl, M, G, top, "f32", chosen_only=chosen_only)
        l, at = logits.double().cpu().requires_grad_(), e.cpu().long()
        there = (at >= 0) & (at < G)
        safe = torch.where(there, at, 0)
        if chosen_only:
            p = torch.softmax(torch.where(there, l.gather(1, safe), -math.inf), 1)
        else:
            p = torch.softmax(l, 1).gather(1, safe) * there
        (p * d.double().cpu()).sum().backward()
        within(dl, l.grad, torch.full((M, G), 128 * U * float(d.abs().sum())))


# ------------------------------------------------------------------ sorted rows

SORTS = [(1, 1, 1, 0), (1, 8, 8, 0), (5, 3, 2, 1), (64, 4, 32, 0), (33, 3, 1000, 7), (255, 4, 16, 9), (256, 4, 256, 0), (257, 4, 7, 11),
         (1000, 1, 1024, 0), (1025, 2, 64, 100), (4099, 8, 256, 31), (8192, 8, 256, 100), (20000, 6, 60, 5), (4096, 4, 100, 0), (16385, 1, 16, 0), (131, 32, 40, 3), (3, 32, 1024, 0)]


def choose(g, M, top, G, padded):
    """top distinct experts of a token where there are as many; the last tokens none."""
    e = (randn(g, M, max(G, top)) + randn(g, 1, max(G, top))).argsort(-1)[:, :top].int()
    e[e >= G] = -1
    if padded:
        e[M - padded:] = -1
    return e.contiguous()


def check_sort(e, G, offsets, slots, source):
    o, s, src = ref.sort(e.cpu(), G)
    assert offsets.tolist() == o
    assert slots.flatten().tolist() == s
    if source is not None:
        assert source.tolist() == src
    return o, src


@pytest.mark.parametrize("M,top,G,padded", SORTS)
def test_sort(sk, M, top, G, padded):
    e = choose(gen(M + G), M, top, G, padded)
    o, s, src = guarded((G + 1,), INT), guarded((M, top), INT), guarded((M * top,), INT)
    sk.moe_sort(e, o.data, s.data, src.data, M, top, G)
    check_sort(e, G, o.data, s.data, src.data)
    assert o.intact() and s.intact() and src.intact()
    sk.moe_sort(e, o.data, s.data, None, M, top, G)     # without `source`
    check_sort(e, G, o.data, s.data, None)


@pytest.mark.parametrize("T,G", [(300, 5), (1024, 16), (5000, 1024), (70000, 3)])
def test_sort_of_any_entries(sk, T, G):
    """Entries outside [0, G), all in one expert, or none at all."""
    g = gen(T)
    wild = torch.randint(-3, G + 3, (T, 1), device="cuda", generator=g).int()
    wild[::7] = 2 ** 31 - 1
    wild[3::11] = -2 ** 31
    for e in (wild, torch.full((T, 1), G - 1, device="cuda").int(), torch.full((T, 1), -1, device="cuda").int()):
        o, s, src = guarded((G + 1,), INT), guarded((T, 1), INT), guarded((T,), INT)
        sk.moe_sort(e, o.data, s.data, src.data, T, 1, G)
        check_sort(e, G, o.data, s.data, src.data)
        assert o.intact() and s.intact() and src.intact()


@pytest.mark.parametrize("G", [15, 16, 17, 63, 64, 65, 255, 256, 257, 293, 301, 302, 341, 353, *range(357, 364), 511, 512, 513, 1023])
def test_sort_with_any_number_of_experts(sk, G):
    """The ends of what a launch takes shared memory and bits for."""
    for T in (900, 2500, 17000):
        e = torch.randint(0, G, (T, 1), device="cuda", generator=gen(G)).int()
        o, s, src = guarded((G + 1,), INT), guarded((T, 1), INT), guarded((T,), INT)
        sk.moe_sort(e, o.data, s.data, src.data, T, 1, G)
        check_sort(e, G, o.data, s.data, src.data)
        assert o.intact() and s.intact() and src.intact()


def test_sort_of_no_tokens_gives_empty_runs(sk):
    for G in (1, 33, 1024):
        o = guarded((G + 1,), INT)
        sk.moe_sort(None, o.data, None, None, 0, 2, G)
        assert o.data.eq(0).all() and o.intact()
        o.data.fill_(9)
        sk.moe_dispatch(None, None, o.data, None, None, None, 0, 2, G, 64, "bf16")
        assert o.data.eq(0).all() and o.intact()


def test_sort_of_the_largest_count(sk):
    T, G = 1 << 22, 1000
    g = gen(4)
    e = torch.randint(-1, G, (T // 4, 4), device="cuda", generator=g).int()
    o, s, src = guarded((G + 1,), INT), guarded((T // 4, 4), INT), guarded((T,), INT)
    sk.moe_sort(e, o.data, s.data, src.data, T // 4, 4, G)
    flat = torch.where(e.flatten() < 0, G, e.flatten())
    key, order = torch.sort(flat, stable=True)
    there = key < G
    assert torch.equal(src.data.long(), torch.where(there, order, -1))
    assert torch.equal(o.data.long(), torch.searchsorted(key, torch.arange(G + 1, device="cuda", dtype=INT)))
    want = torch.empty(T, dtype=torch.int64, device="cuda").scatter(0, order, torch.where(there, torch.arange(T, device="cuda"), -1))
    assert torch.equal(s.data.flatten().long(), want)
    assert o.intact() and s.intact() and src.intact()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "fp8"])
@pytest.mark.parametrize("M,top,G,padded", [c for c in SORTS if c[0] * c[1] < 9000] + [(300, 3, 40, 2), (300, 4, 40, 2)])
def test_dispatch(sk, M, top, G, padded, dtype):
    K = {0: 16, 1: 144, 2: 1040, 3: 4112}[(M + G) % 4]
    g, T = gen(M * top), M * top
    e = choose(g, M, top, G, padded)
    o, s, src = guarded((G + 1,), INT), guarded((M, top), INT), guarded((T,), INT)
    if dtype == "fp8":
        x = (60 * randn(g, M, K)).clamp(-448, 448).to(E4M3)
        sc = randn(g, M, nblk(K))
        rows, rs = guarded((T, K), E4M3), guarded((T, nblk(K)), torch.float32, 7.0)
        rows.data.view(torch.uint8).fill_(7)
        sk.moe_dispatch_fp8(e, x, sc, o.data, s.data, src.data, rows.data, rs.data, M, top, G, K)
        pairs = [(x.view(torch.uint8), rows.data.view(torch.uint8)), (sc, rs.data)]
        assert rs.intact()
    else:
        x = randn(g, M, K).to(DT[dtype])
        rows = guarded((T, K), DT[dtype], 7.0)
        sk.moe_dispatch(e, x, o.data, s.data, src.data, rows.data, M, top, G, K, dtype)
        pairs = [(x, rows.data)]
    offsets, source = check_sort(e, G, o.data, s.data, src.data)
    n = offsets[-1]
    token = torch.tensor(source[:n], device="cuda", dtype=torch.long) // top
    for have, got in pairs:
        assert torch.equal(got[:n], have[token])
        assert got[n:].eq(7).all()                       # rows behind the last run
    assert o.intact() and s.intact() and src.intact() and rows.intact()


BACKS = [(1, 1, 8), (1, 8, 2048), (3, 2, 72), (64, 4, 4096), (33, 3, 1544), (65, 5, 264), (17, 32, 520), (200, 9, 1032), (128, 7, 16400), (1003, 3, 1544)]


def sums_in_a_row(K):
    """The terms that a thread adds in a row, a warp's lanes over K at the least, and
    the lanes' and warps' after them."""
    return K / 32 + 24


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,top,K", BACKS)
def test_combine_and_its_gradient(sk, M, top, K, dtype):
    g, T = gen(M + K), M * top
    slots = torch.randperm(T, device="cuda", generator=g).view(M, top).int()
    shares, rows, dout = randn(g, M, top), randn(g, T, K).to(DT[dtype]), randn(g, M, K).to(DT[dtype])
    if M > 2:
        rows[slots[2, top - 1].long()] = math.nan        # a row that nobody takes
        slots[2, top - 1] = -1
        slots[1] = torch.tensor([[-1, T, -2 ** 31, 2 ** 31 - 1, T + 1][j % 5] for j in range(top)], dtype=INT)
    for out_dtype in ("f32", dtype):
        for w in (shares, None):
            out = guarded((M, K), DT[out_dtype])
            sk.moe_combine(rows, slots, w, out.data, M, top, K, dtype, out_dtype)
            want, size = ref.combine(rows, slots, w)
            within(out.data, want, top * U * size, out_dtype)
            assert out.intact()
    there = (slots >= 0) & (slots < T)
    at = slots[there].long()
    m = there.nonzero()[:, 0]
    drows, ds = guarded((T, K), DT[dtype], 5.0), guarded((M, top), torch.float32)
    sk.moe_combine_grad(dout, rows, slots, shares, drows.data, ds.data, M, top, K, dtype)
    want = torch.full((T, K), 5.0, dtype=torch.float64, device="cuda")
    want[at] = dout.double()[m] * shares.double()[there][:, None]
    within(drows.data, want, U * want.abs(), dtype)
    x = torch.where(there[..., None], rows.double()[slots.clamp(0, T - 1).long()], 0.0)
    dots = x * dout.double()[:, None]
    within(ds.data, dots.sum(-1), sums_in_a_row(K) * U * dots.abs().sum(-1))
    assert drows.intact() and ds.intact()
    # each of the two alone, without shares, and the rows' gradient in the rows' place
    one, alone = guarded((T, K), DT[dtype], 5.0), guarded((M, top), torch.float32)
    sk.moe_combine_grad(dout, None, slots, None, one.data, None, M, top, K, dtype)
    want[at] = dout.double()[m]
    assert torch.equal(one.data.double(), want)
    sk.moe_combine_grad(dout, rows, slots, shares, None, alone.data, M, top, K, dtype)
    assert torch.equal(alone.data, ds.data)
    place = rows.clone()
    sk.moe_combine_grad(dout, place, slots, shares, place, alone.data, M, top, K, dtype)
    assert torch.equal(alone.data, ds.data) and torch.equal(place[at], drows.data[at])
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[at] = False
    assert torch.equal(place[others].nan_to_num(9), rows[others].nan_to_num(9))


def test_combine_gradient_by_differences(sk):
    """Integers: the sums and their central differences are exact."""
    M, top, K = 3, 2, 8
    g = gen(9)
    rows = torch.randint(-4, 5, (M * top, K), device="cuda", generator=g).float()
    shares = torch.randint(-3, 4, (M, top), device="cuda", generator=g).float()
    dout = torch.randint(-4, 5, (M, K), device="cuda", generator=g).float()
    slots = torch.randperm(M * top, device="cuda", generator=g).view(M, top).int()
    out, drows, ds = torch.empty(M, K, device="cuda"), torch.empty(M * top, K, device="cuda"), torch.empty(M, top, device="cuda")

    def loss(r, s):
        sk.moe_combine(r.float().cuda(), slots, s.float().cuda(), out, M, top, K, "f32", "f32")
        return (out.double() * dout.double()).sum()

    sk.moe_combine_grad(dout, rows, slots, shares, drows, ds, M, top, K, "f32")
    assert torch.equal(drows.cpu().double(), ref.differences(lambda r: loss(r, shares), rows.cpu(), 1.0))
    assert torch.equal(ds.cpu().double(), ref.differences(lambda s: loss(rows, s), shares.cpu(), 1.0))


def test_rows_beyond_32_bits(sk):
    """Rows whose values count past 2^31, and whose bytes past 2^32."""
    M, top, K, G = 75000, 8, 4096, 64
    T = M * top
    assert T * K > 1 << 31
    g = gen(0)
    e = choose(g, M, top, G, 0)
    x = torch.randint(-8, 9, (M, K), device="cuda", generator=g).half()
    o, s = torch.empty(G + 1, dtype=INT, device="cuda"), torch.empty(M, top, dtype=INT, device="cuda")
    rows = torch.empty(T, K, dtype=torch.float16, device="cuda")
    sk.moe_dispatch(e, x, o, s, None, rows, M, top, G, K, "f16")
    assert s.max() == T - 1
    at = torch.cat([s.flatten().argmax()[None], torch.randint(0, T, (300,), device="cuda", generator=g)])
    assert torch.equal(rows[s.flatten()[at].long()], x[at // top])
    out = torch.empty(M, K, device="cuda", dtype=torch.float16)
    sk.moe_combine(rows, s, None, out, M, top, K, "f16", "f16")
    assert torch.equal(out, 8 * x)
    ds = torch.empty(M, top, device="cuda")
    drows = rows
    sk.moe_combine_grad(x, rows, s, torch.full((M, top), 2.0, device="cuda"), drows, ds, M, top, K, "f16")
    assert torch.equal(ds, x.double().square().sum(1, keepdim=True).expand(M, top).float())
    assert torch.equal(drows[s.flatten()[at].long()], 2 * x[at // top])


def test_the_most_tokens(sk):
    """2^22 tokens of one entry each, short rows: through route, dispatch and back."""
    M, G, K = 1 << 22, 3, 8
    g = gen(2)
    logits = randn(g, M, G)
    e, s, dl = torch.empty(M, 1, dtype=INT, device="cuda"), torch.empty(M, 1, device="cuda"), torch.empty(M, G, device="cuda")
    sk.moe_route(logits, e, s, M, G, 1, "f32")
    p = torch.softmax(logits.double(), 1)
    assert torch.equal(e[:, 0].long(), logits.argmax(1))
    within(s, p.amax(1, keepdim=True), 96 * U * p.amax(1, keepdim=True))
    ones = torch.ones(M, 1, device="cuda")
    sk.moe_route_grad(logits, e, ones, dl, M, G, 1, "f32")
    top = p.gather(1, e.long())
    want = -p * top
    want.scatter_add_(1, e.long(), top)
    within(dl, want, 256 * U * (p * top).clamp(min=0) + 256 * U * top * torch.zeros_like(p).scatter(1, e.long(), 1.0))
    x = randn(g, M, K).half()
    o, sl, src = torch.empty(G + 1, dtype=INT, device="cuda"), torch.empty(M, 1, dtype=INT, device="cuda"), torch.empty(M, dtype=INT, device="cuda")
    rows, back, ds = torch.empty_like(x), torch.empty_like(x), torch.empty(M, 1, device="cuda")
    sk.moe_dispatch(e, x, o, sl, src, rows, M, 1, G, K, "f16")
    assert torch.equal(rows, x[src.long()]) and o.tolist() == [0, *torch.bincount(e.flatten(), minlength=G).cumsum(0).tolist()]
    sk.moe_combine(rows, sl, None, back, M, 1, K, "f16", "f16")
    assert torch.equal(back, x)
    sk.moe_combine_grad(x, rows, sl, None, None, ds, M, 1, K, "f16")
    size = x.double().square().sum(1, keepdim=True)
    within(ds, size, 16 * U * size)


# ------------------------------------------------------------------ together

class Layer:
    """A layer of experts in 16 bits, forward and backward through the library alone."""

    def __init__(self, sk, M, G, top, K, N, seed=0, dtype="bf16"):
        g = gen(seed)
        self.sk, self.M, self.G, self.top, self.K, self.N, self.dt = sk, M, G, top, K, N, dtype
        t, T = DT[dtype], M * top
        self.x, self.res = randn(g, M, K).to(t), randn(g, M, K).to(t)
        self.w, self.b = (1 + 0.1 * randn(g, K)).to(t), (0.1 * randn(g, K)).to(t)
        self.router = (randn(g, K, G) / K ** 0.5).to(t)
        self.up, self.down = (randn(g, G, N, K) / K ** 0.5).to(t), (randn(g, G, K, N) / N ** 0.5).to(t)
        self.dout, self.dsum = (0.1 * randn(g, M, K)).to(t), (0.1 * randn(g, M, K)).to(t)

        def e(*shape, dtype=t):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        f = torch.float32
        self.sum, self.y, self.mean, self.rstd = e(M, K), e(M, K), e(M, dtype=f), e(M, dtype=f)
        self.logits, self.experts, self.shares = e(M, G), e(M, top, dtype=INT), e(M, top, dtype=f)
        self.offsets, self.slots = e(G + 1, dtype=INT), e(M, top, dtype=INT)
        self.rows, self.mid, self.back, self.out = (torch.zeros(T, K, dtype=t, device="cuda"), torch.zeros(T, N, dtype=t, device="cuda"),
                                                    torch.zeros(T, K, dtype=t, device="cuda"), e(M, K))
        self.dback, self.dshares, self.dlogits = torch.zeros(T, K, dtype=t, device="cuda"), e(M, top, dtype=f), e(M, G)
        self.dmid, self.drows, self.dy = torch.zeros(T, N, dtype=t, device="cuda"), torch.zeros(T, K, dtype=t, device="cuda"), e(M, K)
        self.dup, self.ddown, self.drouter = e(G, N, K, dtype=f), e(G, K, N, dtype=f), e(K, G)
        self.dx, self.dw, self.db, self.norm = e(M, K), e(K, dtype=f), e(K, dtype=f), e(1, dtype=f)
        self.nbytes = sk.layernorm_grad_workspace_bytes(M, K)
        self.ws, self.gws = e(self.nbytes, dtype=torch.uint8), e(sk.grad_norm_workspace_bytes(), dtype=torch.uint8)
        self.grads = sk.grad_list([self.dup, self.ddown, self.drouter, self.dw, self.db])

    def step(self):
        sk, M, G, top, K, N, dt = self.sk, self.M, self.G, self.top, self.K, self.N, self.dt
        T = M * top
        sk.layernorm(self.x, self.w, self.b, self.y, M, K, dt, residual=self.res, sum_out=self.sum, mean=self.mean, rstd=self.rstd)
        torch.mm(self.y, self.router, out=self.logits)
        sk.moe_route(self.logits, self.experts, self.shares, M, G, top, dt)
        sk.moe_dispatch(self.experts, self.y, self.offsets, self.slots, None, self.rows, M, top, G, K, dt)
        sk.gemm_grouped_bt(self.rows, self.up, self.offsets, self.mid, T, G, N, K, dt, dt)
        sk.gemm_grouped_bt(self.mid, self.down, self.offsets, self.back, T, G, K, N, dt, dt)
        sk.moe_combine(self.back, self.slots, self.shares, self.out, M, top, K, dt, dt)
        # and back
        sk.moe_combine_grad(self.dout, self.back, self.slots, self.shares, self.dback, self.dshares, M, top, K, dt)
        sk.gemm_grouped_kn(self.dback, self.down, self.offsets, self.dmid, T, G, N, K, dt, dt)
        sk.gemm_grouped_dw(self.mid, self.dback, self.offsets, self.ddown, T, G, K, N, dt, "f32")
        sk.gemm_grouped_kn(self.dmid, self.up, self.offsets, self.drows, T, G, K, N, dt, dt)
        sk.gemm_grouped_dw(self.rows, self.dmid, self.offsets, self.dup, T, G, N, K, dt, "f32")
        sk.moe_combine(self.drows, self.slots, None, self.dy, M, top, K, dt, dt)
        sk.moe_route_grad(self.logits, self.experts, self.dshares, self.dlogits, M, G, top, dt)
        torch.mm(self.y.t(), self.dlogits, out=self.drouter)
        torch.addmm(self.dy, self.dlogits, self.router.t(), out=self.dx)
        sk.layernorm_grad(self.dx, self.sum, self.w, self.mean, self.rstd, self.dx, self.dw, self.db, self.ws, self.nbytes, M, K, dt,
                          dsum=self.dsum)
        sk.grad_clip(self.grads, 0.5, self.norm, self.gws, sk.grad_norm_workspace_bytes())

    OUTPUTS = ("sum", "y", "out", "dx", "dup", "ddown", "drouter", "dw", "db", "norm", "experts", "shares", "offsets", "slots")

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.OUTPUTS}


@pytest.mark.parametrize("M", [1, 96, 1500])
def test_a_training_step_of_a_layer_of_experts(sk, M):
    """Against the same layer in 64 bits with the library's choice of experts, by
    autograd.  Values pass through about ten roundings to BF16 (2^-8 at worst, 2^-9.8
    rms) on the way to a gradient: 2% of the norm leaves twice what they add up to."""
    layer = Layer(sk, M, 8, 2, 264, 136)
    layer.step()
    assert sk.splitk_get_device_status() == 0
    leaves = {n: getattr(layer, n).double().requires_grad_() for n in ("w", "b", "router", "up", "down")}
    h = layer.sum.double().requires_grad_()
    mean = h.mean(1, keepdim=True)
    y = (h - mean) / ((h - mean).square().mean(1, keepdim=True) + 1e-5).sqrt() * leaves["w"] + leaves["b"]
    shares = torch.softmax(y @ leaves["router"], -1).gather(1, layer.experts.long())
    out = torch.zeros_like(h)
    for j in range(layer.top):
        e = layer.experts[:, j].long()
        mid = torch.einsum("mk,mnk->mn", y, leaves["up"][e])
        out = out + shares[:, j, None] * torch.einsum("mn,mkn->mk", mid, leaves["down"][e])
    (out * layer.dout.double()).sum().add((h * layer.dsum.double()).sum()).backward()
    got = {"up": layer.dup, "down": layer.ddown, "router": layer.drouter, "w": layer.dw, "b": layer.db}
    norm = math.sqrt(sum(float(leaves[n].grad.square().sum()) for n in got))
    assert abs(float(layer.norm) / norm - 1) < 0.02
    factor = min(1.0, 0.5 / norm)
    assert torch.linalg.norm(layer.out.double() - out) < 0.02 * torch.linalg.norm(out)
    assert torch.linalg.norm(layer.dx.double() - h.grad) < 0.02 * torch.linalg.norm(h.grad)
    for n, t in got.items():
        want = leaves[n].grad * factor
        assert torch.linalg.norm(t.double() - want) < 0.04 * torch.linalg.norm(want), n


@pytest.mark.parametrize("M", [5, 700])
def test_a_captured_step_gives_the_eager_bits(sk, M):
    layer = Layer(sk, M, 8, 2, 264, 136, seed=3)
    layer.step()
    torch.cuda.synchronize()
    want = layer.outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    for seed in (3, 4, 3):
        other = Layer(sk, M, 8, 2, 264, 136, seed=seed)
        for n in ("x", "res", "router", "dout"):
            getattr(layer, n).copy_(getattr(other, n))
        for n in Layer.OUTPUTS:
            getattr(layer, n).fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        if seed == 3:
            for n, t in want.items():
                assert torch.equal(t, getattr(layer, n)), n
    assert sk.splitk_get_device_status() == 0


def test_streams_and_threads(sk):
    """Four threads, each with its own stream and tensors: the bits of a single one."""
    layers = [Layer(sk, 200 + 70 * i, 8, 2, 264, 136, seed=i) for i in range(4)]
    want = []
    for layer in layers:
        layer.step()
        want.append(layer.outputs())
    torch.cuda.synchronize()
    failed = []

    def work(layer):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    layer.step()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(layer,)) for layer in layers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for layer, w in zip(layers, want):
        for n, t in w.items():
            assert torch.equal(t, getattr(layer, n)), n


def test_large_calls_at_once(sk):
    """Clusters of 16 blocks, rings that fill an SM and grids over all SMs, from four
    threads on their own streams: the bits of a single one."""
    class Work:
        def __init__(self, i):
            g = gen(40 + i)
            self.M, self.top, self.G, self.K = 6000 + 700 * i, 4, 300 + i, 520
            M, K, T = self.M, self.K, self.M * 4
            self.e, self.x = choose(g, M, 4, self.G, 17), randn(g, M, K).bfloat16()
            self.o, self.s, self.src = (torch.empty(n, dtype=INT, device="cuda") for n in (self.G + 1, T, T))
            self.rows, self.back = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda"), torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
            self.w, self.mean, self.rstd = torch.ones(K, device="cuda").bfloat16(), torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
            self.dx, self.dw, self.db = torch.empty_like(self.back), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
            self.nbytes = sk.layernorm_grad_workspace_bytes(M, K)
            self.ws, self.gws = torch.empty(self.nbytes, dtype=torch.uint8, device="cuda"), torch.empty(sk.grad_norm_workspace_bytes(), dtype=torch.uint8, device="cuda")
            self.norm, self.out = torch.empty(1, device="cuda"), [torch.empty_like(self.rows), torch.empty_like(self.dw)]

        def step(self):
            M, top, K = self.M, self.top, self.K
            sk.moe_sort(self.e, self.o, self.s, self.src, M, top, self.G)
            sk.moe_dispatch(self.e, self.x, self.o, self.s, self.src, self.rows, M, top, self.G, K, "bf16")
            sk.moe_combine(self.rows, self.s, None, self.back, M, top, K, "bf16", "bf16")
            sk.layernorm_grad(self.back, self.x, self.w, self.mean, self.rstd, self.dx, self.dw, self.db, self.ws, self.nbytes, M, K, "bf16")
            sk.grad_clip([self.rows, self.dw], 3.0, self.norm, self.gws, sk.grad_norm_workspace_bytes(), out=self.out)

        def outputs(self):
            return [t.clone() for t in (self.o, self.s, self.src, self.rows, self.back, self.dx, self.dw, self.db, self.norm, *self.out)]

    works, want, failed = [Work(i) for i in range(4)], [], []
    for w in works:
        w.step()
        want.append(w.outputs())
    torch.cuda.synchronize()

    def run(w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    w.step()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for w, kept in zip(works, want):
        assert all(torch.equal(a, b) for a, b in zip(kept, w.outputs()))


def test_captured_beside_the_split_k_product(sk):
    """Layer norm, a split-K product of its output, route of the product's rows, and back
    through the norm, captured in one graph: the eager bits."""
    M, K, G = 64, 1024, 64
    g = gen(12)
    x, w, router = randn(g, M, K).half(), randn(g, K).half(), randn(g, G, K).half()
    nbytes = sk.gemm_bt_workspace_bytes(M, G, K, 2, 512)
    ws = torch.empty(nbytes // 4, device="cuda")
    y, logits, e, s = torch.empty_like(x), torch.empty(M, G, device="cuda"), torch.empty(M, 4, dtype=INT, device="cuda"), torch.empty(M, 4, device="cuda")
    o, sl, rows, out = (torch.empty(G + 1, dtype=INT, device="cuda"), torch.empty(M, 4, dtype=INT, device="cuda"),
                        torch.empty(4 * M, K, dtype=torch.float16, device="cuda"), torch.empty(M, K, device="cuda"))

    def step():
        for fused in (0, 1):
            sk.layernorm(x, w, None, y, M, K, "f16")
            sk.gemm_bt(y, router, logits, ws, nbytes, M, G, K, 2, 512, "f16", fused=fused)
            sk.moe_route(logits, e, s, M, G, 4, "f32")
            sk.moe_dispatch(e, y, o, sl, None, rows, M, 4, G, K, "f16")
            sk.moe_combine(rows, sl, s, out, M, 4, K, "f16", "f32")
            x.copy_(out)

    kept = x.clone()
    step()
    want = [t.clone() for t in (logits, e, s, o, sl, rows, out)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.copy_(kept)
        for t in (logits, e, s, o, sl, rows, out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (logits, e, s, o, sl, rows, out)))
    assert sk.splitk_get_device_status() == 0


FIRST = """
import sys
sys.path.insert(0, {root!r})
import torch
import split_bf16_gemm_gb300 as sk
M, top, G, K = 5000, 4, 500, 264
e = torch.arange(M * top, device="cuda").mul(7).remainder(G).int().view(M, top)
x = torch.arange(M, device="cuda").float()[:, None].expand(M, K).contiguous()
o, s = torch.zeros(G + 1, dtype=torch.int32, device="cuda"), torch.zeros(M, top, dtype=torch.int32, device="cuda")
src, rows, back = torch.zeros(M * top, dtype=torch.int32, device="cuda"), torch.zeros(M * top, K, device="cuda"), torch.zeros(M, K, device="cuda")
dw, db, one = torch.zeros(K, device="cuda"), torch.zeros(K, device="cuda"), torch.ones(M, device="cuda")
nb = sk.layernorm_grad_workspace_bytes(M, K)
ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    sk.moe_dispatch(e, x, o, s, src, rows, M, top, G, K, "f32")
    sk.moe_sort(e, o, s, src, M, top, G)
    sk.moe_combine(rows, s, None, back, M, top, K, "f32", "f32")
    sk.layernorm_grad(back, x, one[:K].contiguous(), one, one, rows[:M], dw, db, ws, nb, M, K, "f32")
graph.replay()
torch.cuda.synchronize()
assert torch.equal(back, top * x), "rows"
key, order = torch.sort(e.flatten(), stable=True)
assert torch.equal(src.long(), order), "source"
assert torch.equal(db, torch.full_like(db, float(top * M * (M - 1) // 2))) or (db / (top * M * (M - 1) / 2) - 1).abs().max() < 1e-5
print("first calls captured")
"""


def test_first_calls_of_a_process_may_be_captured(sk):
    """Kernels that need more shared memory or wider clusters than the default set
    that up in any call."""
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=200)
    assert "first calls captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("M", [4, 300])
def test_example_block_on_sorted_rows(sk, M):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block_rows", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # eight-bit operands: four significant bits, as in the example's own test
    assert example.main(M, 24, hidden=512, inner=256, top=3) < 0.1

"""Expert products where a CTA or a pair of them works through many units, so
that every ring of buffers, plans and row lists is used again and again; very
uneven experts; and NaN and infinities in rows that count.  Against 64 bits
with the tolerances of the arithmetic (u = 2^-24: exact products, 128
additions in a block, one product and addition a block, twice u for
truncation; a bf16 output lies between the roundings of the tolerance's ends)."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    return load_ep()


def cast_blocks(x, rows_per_scale):
    """e4m3 codes and scales of [N, K] in blocks of rows_per_scale x 128 (N a multiple of rows_per_scale)."""
    N, K = x.shape
    b = x.view(N // rows_per_scale, rows_per_scale, K // 128, 128)
    amax = b.abs().amax((1, 3))
    q = (b * (448.0 / amax.clamp_min(1e-30))[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(N, K), amax / 448.0


def case(m, R, Tr, E, k, N, K, counts, seed=0):
    """Problem and operands; the rows that do not count hold NaN codes with NaN scales."""
    T = R * Tr
    p = m.problem(T, K, k, E, R)
    counts = torch.as_tensor(counts, dtype=torch.int32, device=DEV)
    gen = torch.Generator(DEV).manual_seed(seed)
    live = (torch.arange(Tr, device=DEV) < counts.t()[..., None]).reshape(-1)
    a = torch.full((E * T, K), 0x7F, dtype=torch.uint8, device=DEV)
    s = torch.full((E * T, K // 128), math.nan, device=DEV)
    a[live], s[live] = cast_blocks(torch.randn(int(live.sum()), K, generator=gen, device=DEV), 1)
    w = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    ws = torch.empty(E, N // 128, K // 128, device=DEV)
    for e in range(E):
        w[e], ws[e] = cast_blocks(torch.randn(N, K, generator=gen, device=DEV) * K ** -0.5, 128)
    return p, counts, live, a, s, w, ws


def products(live, a, s, w, ws):
    """(rows, c, sum of |terms|) of each expert that has rows, in 64 bits."""
    per = live.numel() // w.shape[0]
    for e in range(w.shape[0]):
        at = e * per + torch.nonzero(live[e * per:(e + 1) * per])[:, 0]
        if at.numel() == 0:
            continue
        av = a[at].view(torch.float8_e4m3fn).double() * s[at].double().repeat_interleave(128, 1)
        wv = w[e].view(torch.float8_e4m3fn).double()
        wv *= ws[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        yield at, av @ wv.t(), av.abs() @ wv.abs().t()


def run_gemm(m, p, counts, a, s, w, ws):
    y = torch.full((a.shape[0], w.shape[1]), -5.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_expert_gemm(p, a, s, w, ws, counts, y, st)
    assert int(st.item()) == 0
    return y


def run_swiglu(m, p, counts, a, s, w, ws):
    I = w.shape[1] // 2
    q = torch.full((a.shape[0], I), 0x55, dtype=torch.uint8, device=DEV)
    qs = torch.full((a.shape[0], I // 128), -5.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_expert_swiglu(p, a, s, w, ws, counts, q, qs, st)
    assert int(st.item()) == 0
    return q, qs


def check_gemm(m, p, counts, live, a, s, w, ws):
    K = a.shape[1]
    y = run_gemm(m, p, counts, a, s, w, ws)
    for at, c, mag in products(live, a, s, w, ws):
        tol = (128 + K / 128 + 8) * 2 * U * mag + 1e-30
        lo, hi = (c - tol).float().bfloat16(), (c + tol).float().bfloat16()
        assert bool(((lo <= y[at]) & (y[at] <= hi)).all())
    assert bool((y[~live] == -5).all())
    for _ in range(3):
        assert torch.equal(run_gemm(m, p, counts, a, s, w, ws), y)


def check_swiglu(m, p, counts, live, a, s, w, ws):
    K, I = a.shape[1], w.shape[1] // 2
    q, qs = run_swiglu(m, p, counts, a, s, w, ws)
    assert bool((q[~live] == 0x55).all()) and bool((qs[~live] == -5).all())
    for at, c, mag in products(live, a, s, w, ws):
        err = (128 + K / 128 + 8) * 2 * U * mag
        g, up, eg, eu = c[:, :I], c[:, I:], err[:, :I], err[:, I:]
        sil = g / (1 + torch.exp(-g))
        h = sil * up
        # |silu'| <= 1.1; exp, quotient and products: a dozen roundings and that of the exponent's argument
        eh = 1.1 * eg * (up.abs() + eu) + sil.abs() * eu + (16 + 2 * g.abs()) * U * h.abs()
        top, etop = h.view(-1, I // 128, 128).abs().amax(2), eh.view(-1, I // 128, 128).amax(2)
        scale = qs[at].double()
        assert bool(((scale - top / 448).abs() <= etop / 448 + 4 * U * top / 448 + 1e-45).all())
        wide = scale.repeat_interleave(128, 1)
        step = torch.maximum(2.0 ** -4 * h.abs(), 2.0 ** -10 * wide)     # half a step of e4m3
        dec = q[at].view(torch.float8_e4m3fn).double() * wide
        assert bool(((dec - h).abs() <= step * (1 + 2.0 ** -10) + 1.1 * eh).all())
    for _ in range(3):
        q2, qs2 = run_swiglu(m, p, counts, a, s, w, ws)
        assert torch.equal(q, q2) and torch.equal(qs, qs2)


def spread(R, Tr, E, rows, seed):
    """Counts [R, E] with about `rows` rows an expert, uneven, some experts and segments empty."""
    rng = np.random.default_rng(seed)
    c = rng.binomial(Tr, min(1.0, rows / (R * Tr)), (R, E))
    c[rng.random((R, E)) < 0.1] = 0
    c[:, rng.random(E) < 0.1] = 0
    return c


# Few rows an expert (tokens * k <= 48 experts).  64 experts x 64 column tiles are 27 units for each of 152 CTAs: with
# one step a unit (K = 128) the ring of 16 row lists and the 4 to 7 operand buffers go around most often for their
# work; K = 2048 has several units and 16 steps each.
FEW = [(2, 16, 64, 4, 8192, 128, 8), (4, 24, 64, 32, 8192, 128, 40), (8, 6, 64, 32, 4096, 256, 20),
       (1, 96, 64, 8, 4096, 384, 70), (2, 16, 64, 4, 8192, 2048, 8)]


@pytest.mark.parametrize("R,Tr,E,k,N,K,rows", FEW)
def test_few_rows_many_units(m, R, Tr, E, k, N, K, rows):
    assert R * Tr * k <= 48 * E
    c = case(m, R, Tr, E, k, N, K, spread(R, Tr, E, rows, N + K + rows))
    check_gemm(m, *c)
    check_swiglu(m, *c)


@pytest.mark.parametrize("K", [128, 640])
def test_few_rows_rule_with_uneven_experts(m, K):
    """Two experts of 64 take every token: many row tiles each, in the kernel that the average chooses."""
    R, Tr, E, k, N = 4, 128, 64, 2, 2048
    counts = np.zeros((R, E), np.int32)
    counts[:, 5] = counts[:, 40] = Tr
    counts[1, 40] = Tr - 3
    counts[2, 63] = 1
    c = case(m, R, Tr, E, k, N, K, counts)
    check_gemm(m, *c)
    check_swiglu(m, *c)


def broken_rows(m, R, Tr, E, k, N, K, rows):
    """Operands with a NaN code, a NaN scale and an infinite scale in three rows that count, and a clean copy."""
    p, counts, live, a, s, w, ws = case(m, R, Tr, E, k, N, K, spread(R, Tr, E, rows, 11), 3)
    at = torch.nonzero(live)[:, 0][[0, 7, 20]]
    a2, s2 = a.clone(), s.clone()
    a2[at[0], K - 3] = 0x7F
    s2[at[1], 0] = math.nan
    s2[at[2], K // 128 - 1] = math.inf
    return p, counts, live, a, s, w, ws, a2, s2, at


def bad_operands(m, R, Tr, E, k, N, K, rows):
    p, counts, live, a, s, w, ws, a2, s2, at = broken_rows(m, R, Tr, E, k, N, K, rows)
    per = live.numel() // E
    others = live.clone()
    others[at] = False
    # rows
    clean, y = run_gemm(m, p, counts, a, s, w, ws), run_gemm(m, p, counts, a2, s2, w, ws)
    assert torch.equal(y[others], clean[others])
    assert bool(y[at[:2]].isnan().all()) and bool((~y[at[2]].isfinite()).all()) and bool(y[at[2]].isinf().any())
    e = int(at[2]) // per
    last = (a[at[2], -128:].view(torch.float8_e4m3fn).double() *
            w[e, :, -128:].view(torch.float8_e4m3fn).double()).sum(1)
    assert bool((last != 0).all())
    assert bool((y[at[2]].double() == torch.where(last > 0, math.inf, -math.inf)).all())
    I = N // 2
    (q, qs), (q2, qs2) = run_swiglu(m, p, counts, a, s, w, ws), run_swiglu(m, p, counts, a2, s2, w, ws)
    assert torch.equal(q2[others], q[others]) and torch.equal(qs2[others], qs[others])
    assert bool(qs2[at[:2]].isnan().all()) and bool(((q2[at[:2]] & 0x7F) == 0x7F).all())
    # a gate of -inf has no value (-inf / inf), one of +inf is infinite: no finite scale either way
    assert bool((~qs2[at[2]].isfinite()).all()) and bool(((q2[at[2]] & 0x7F) == 0x7F).all())
    # matrices: a NaN code in one row of one expert
    e = int(at[0]) // per
    mine = torch.zeros_like(live)
    mine[e * per:(e + 1) * per] = live[e * per:(e + 1) * per]
    w2 = w.clone()
    w2[e, 130, 5] = 0xFF
    y = run_gemm(m, p, counts, a, s, w2, ws)
    assert torch.equal(y[~mine], clean[~mine]) and bool(y[mine][:, 130].isnan().all())
    keep = torch.arange(N, device=DEV) != 130
    assert torch.equal(y[mine][:, keep], clean[mine][:, keep])
    for col in (130, I + 130):                    # a gate row, an up row: its block of 128 has no scale
        w2 = w.clone()
        w2[e, col, 5] = 0x7F
        q2, qs2 = run_swiglu(m, p, counts, a, s, w2, ws)
        assert torch.equal(q2[~mine], q[~mine]) and torch.equal(qs2[~mine], qs[~mine])
        assert bool(qs2[mine][:, 1].isnan().all()) and bool(((q2[mine][:, 130] & 0x7F) == 0x7F).all())
        rest = [b for b in range(I // 128) if b != 1]
        assert torch.equal(qs2[mine][:, rest], qs[mine][:, rest])
        assert torch.equal(q2[mine].view(-1, I // 128, 128)[:, rest], q[mine].view(-1, I // 128, 128)[:, rest])


def test_few_rows_nan_and_infinities(m):
    bad_operands(m, 2, 30, 8, 4, 768, 384, 20)


# Many rows an expert: 16 experts of about 300 rows and 32 or 16 column tiles are 7 to 13 units for each of 76 pairs, so
# that the ring of 4 plans goes around two or three times.  One or two long segments come in boxes, 16 short ones by threads.
MANY = [(2, 600, 16, 4, 8192, 128, 300), (16, 80, 16, 4, 8192, 128, 320), (2, 600, 16, 4, 4096, 1024, 300),
        (16, 80, 16, 4, 4096, 1024, 320), (4, 160, 16, 2, 8192, 256, 90), (1, 1200, 16, 4, 8192, 384, 600)]


@pytest.mark.parametrize("R,Tr,E,k,N,K,rows", MANY)
def test_many_rows_many_units(m, R, Tr, E, k, N, K, rows):
    assert R * Tr * k > 48 * E
    c = case(m, R, Tr, E, k, N, K, spread(R, Tr, E, rows, N + K + rows))
    check_gemm(m, *c)
    check_swiglu(m, *c)


@pytest.mark.parametrize("K", [128, 640])
def test_many_rows_rule_with_uneven_experts(m, K):
    """One expert of 8 takes every token, the others none to three: tiles of one row, in the kernel for many rows."""
    R, Tr, E, k, N = 4, 256, 8, 2, 4096
    counts = np.zeros((R, E), np.int32)
    counts[:, 6] = Tr
    counts[0, 0] = counts[3, 7] = 1
    counts[:3, 3] = 1
    assert R * Tr * k > 48 * E
    c = case(m, R, Tr, E, k, N, K, counts)
    check_gemm(m, *c)
    check_swiglu(m, *c)


@pytest.mark.parametrize("R,Tr,E", [(2, 200, 4), (8, 50, 8)])
def test_many_rows_nan_and_infinities(m, R, Tr, E):
    bad_operands(m, R, Tr, E, 4, 768, 384, 180)


@pytest.mark.parametrize("R,Tr", [(2, 320), (16, 40)])       # rows in boxes, and copied by threads
@pytest.mark.parametrize("kernel", ["EP_EXPERT_FEW_ROWS", "EP_EXPERT_MANY_ROWS"])
def test_waits_that_give_up(m, kernel, R, Tr):
    """A launch whose waits run out says so, comes back with nothing in flight, and the next one is right."""
    E, N, K = 16, 2048, 1024
    p, counts, live, a, s, w, ws = case(m, R, Tr, E, 4, N, K, spread(R, Tr, E, 200, 5))
    rows = a.shape[0]

    def run(clocks, gemm):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        y = torch.full((rows, N), -5.0, dtype=torch.bfloat16, device=DEV) if gemm else None
        q = None if gemm else torch.full((rows, N // 2), 0x55, dtype=torch.uint8, device=DEV)
        qs = None if gemm else torch.full((rows, N // 256), -5.0, device=DEV)
        m.ep_selftest_expert_timeout(p, getattr(m, kernel), a, s, w, ws, counts, y, q, qs, clocks, st)
        return int(st.item()), (y,) if gemm else (q, qs)

    for gemm in (True, False):
        code, want = run(1 << 32, gemm)
        assert code == 0
        # the first wait that is not over at once gives up; longer limits run out further in, or not at all
        assert run(1, gemm)[0] == m.EP_STATUS_TIMEOUT
        for clocks in (200, 1000, 1800, 2500, 3500, 5000, 8000, 20000, 10 ** 9):
            code, out = run(clocks, gemm)
            assert code in (0, m.EP_STATUS_TIMEOUT) and (code == 0 or clocks < 10 ** 9)
            for o, right in zip(out, want):
                assert bool((o[~live] == right[~live]).all())          # never a row that does not count
                assert code != 0 or torch.equal(o, right)
            code, out = run(1 << 32, gemm)
            assert code == 0 and all(torch.equal(o, right) for o, right in zip(out, want))
    check_gemm(m, p, counts, live, a, s, w, ws)
    check_swiglu(m, p, counts, live, a, s, w, ws)

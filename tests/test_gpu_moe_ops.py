"""The routing, combine-backward and expert-product operators against their
definitions in 64 bits.

Tolerances follow from the arithmetic: u = 2^-24 is fp32's unit roundoff,
2^-4 e4m3's.  A bf16 output has to be the rounding of a value within the fp32
tolerance: it lies between the roundings of the tolerance's two ends.  Selections are compared exactly: inputs in which two
different keys are closer than their own rounding are drawn again.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from combine_ep_layout_05_gb300 import inputs
from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def rounds_to(got, want, tol):
    """Every bf16 in got is the nearest-even rounding of a value in want +- tol (rounding is monotone)."""
    lo, hi = (want - tol).float().bfloat16(), (want + tol).float().bfloat16()
    return bool(((lo <= got) & (got <= hi)).all())


@pytest.fixture(scope="module")
def m():
    return load_ep()


# --------------------------------------------------------------------------------------------------------------
# routing
# --------------------------------------------------------------------------------------------------------------

def ref_keys(x, bias, scoring):
    x = x.astype(np.float64)
    with np.errstate(over="ignore"):
        key = x if scoring == "softmax" else 1.0 / (1.0 + np.exp(-x))
    key = key + (0 if bias is None else bias.astype(np.float64))
    fit = (x > -np.inf) & (key > -np.inf)
    return np.where(fit, key, -np.inf)


def ref_select(key, k, groups, keep, best):
    """Ids of one row's choice by the definition: best first, lowest id among equals, -1 for none."""
    E = key.size
    per = E // groups
    if groups > 1:
        score = []
        for g in range(groups):
            v = [z for z in sorted(key[g * per:(g + 1) * per], reverse=True)[:best] if z > -np.inf]
            score.append(sum(v) if v else -np.inf)
        order = sorted((g for g in range(groups) if score[g] > -np.inf), key=lambda g: (-score[g], g))[:keep]
        key = np.array([key[e] if e // per in order else -np.inf for e in range(E)])
    ids = sorted((e for e in range(E) if key[e] > -np.inf), key=lambda e: (-key[e], e))[:k]
    return ids + [-1] * (k - len(ids))


def ref_scores(x, scoring):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), np.finfo(np.float32).max))
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def ref_weights(x, idx, scoring, renorm, scale):
    s = np.where(idx >= 0, np.take_along_axis(ref_scores(x, scoring), np.maximum(idx, 0), 1), 0.0)
    if renorm:
        tot = s.sum(1, keepdims=True)
        s = np.where(tot > 0, s / np.where(tot > 0, tot, 1), 0.0)
    return s * scale


def apart(key, k, groups, best):
    """Rows in which no two different keys, or different group scores, are nearer than 1e-6."""
    def ok(v):
        with np.errstate(invalid="ignore"):
            d = np.abs(np.diff(np.sort(v, 1), axis=1))
        return ~((d > 0) & (d < 1e-6)).any(1)
    good = ok(key)
    if groups > 1:
        v = -np.sort(-key.reshape(key.shape[0], groups, -1), 2)[:, :, :best]
        good &= ok(np.where(v > -np.inf, v, 0).sum(2))
    return good


def make_logits(T, E, dtype, seed, bias, scoring, groups, best, k, spread=1.0, masked=0.0):
    rng = np.random.default_rng(seed)
    draw = lambda n: torch.from_numpy((rng.standard_normal((n, E)) * spread).astype(np.float32)).to(dtype)
    x = draw(T)
    off = rng.random((T, E)) < masked
    x[torch.from_numpy(off)] = -math.inf
    for _ in range(40):
        bad = ~apart(ref_keys(x.float().numpy(), bias, scoring), k, groups, best)
        if not bad.any():
            return x
        new = draw(int(bad.sum()))
        new[torch.from_numpy(off[bad])] = -math.inf
        x[torch.from_numpy(bad)] = new
    raise AssertionError("no inputs without near ties")


def run_route(m, p, r, x, bias, status=None):
    idx = torch.full((p.num_tokens, p.num_topk), -7, dtype=torch.int64, device=DEV)
    w = torch.full((p.num_tokens, p.num_topk), -7.0, device=DEV)
    m.ep_route(p, r, x, bias, idx, w, status)
    return idx, w


ROUTE = [
    # T, E, k, dtype, scoring, bias, groups, keep, best, renorm, scale, spread, masked
    (1, 8, 2, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 1.0, 0.0),
    (1, 256, 8, "fp32", "sigmoid", True, 8, 4, 2, True, 2.5, 1.0, 0.0),
    (33, 256, 8, "bf16", "sigmoid", True, 8, 4, 2, True, 2.5, 1.0, 0.1),
    (64, 160, 6, "fp32", "softmax", False, 8, 3, 1, False, 16.0, 1.0, 0.0),
    (37, 1, 1, "fp32", "sigmoid", False, 1, 1, 1, False, 1.0, 1.0, 0.2),
    (129, 60, 4, "bf16", "softmax", True, 5, 2, 2, True, 1.0, 1.0, 0.3),
    (50, 100, 32, "fp32", "sigmoid", False, 4, 1, 1, True, 1.0, 1.0, 0.0),     # k above what the groups leave: -1
    (40, 384, 8, "fp32", "sigmoid", True, 3, 2, 2, False, 1.0, 1.0, 0.9),
    (70, 1024, 32, "fp32", "softmax", False, 64, 40, 2, True, 1.0, 3.0, 0.5),
    (20, 1023, 7, "bf16", "softmax", False, 1, 1, 1, False, 1.0, 1.0, 0.0),
    (17, 36, 5, "fp32", "softmax", True, 36, 9, 2, True, 1.0, 1.0, 0.0),       # groups of one expert
    (300, 128, 8, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 8.0, 0.0),
    (16, 512, 8, "bf16", "sigmoid", True, 16, 4, 2, True, 1.0, 0.5, 0.98),     # rows left with nothing
    (45, 120, 8, "fp32", "sigmoid", True, 24, 7, 2, True, 1.0, 1.0, 0.1),      # groups that leave lanes over
    (31, 352, 9, "bf16", "sigmoid", False, 11, 5, 1, True, 1.0, 1.0, 0.2),
    (23, 999, 9, "fp32", "softmax", False, 3, 2, 2, True, 1.0, 1.0, 0.0),      # groups too large for lanes of their own
    (30, 66, 3, "fp32", "softmax", True, 2, 1, 2, False, 1.0, 1.0, 0.4),       # a group's last lanes empty
]


@pytest.mark.parametrize("T,E,k,dtype,scoring,with_bias,groups,keep,best,renorm,scale,spread,masked", ROUTE)
def test_route(m, T, E, k, dtype, scoring, with_bias, groups, keep, best, renorm, scale, spread, masked):
    rng = np.random.default_rng(T + E)
    bias = (np.round(rng.standard_normal(E) * 30) * 1e-3).astype(np.float32) if with_bias else None
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = make_logits(T, E, dt, 3 * T + E, bias, scoring, groups, best, k, spread, masked)
    p = m.problem(T, 128, k, E, 1)
    r = m.router(scoring, groups, keep, best, renorm, scale)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    # rows at a stride, starting at an odd element
    wide = torch.full((T, E + 5), 9.0, dtype=dt, device=DEV)
    wide[:, 3:3 + E] = x.to(DEV)
    bd = None if bias is None else torch.from_numpy(bias).to(DEV)
    idx, w = run_route(m, p, r, x.to(DEV), bd, status)
    idx2, w2 = run_route(m, p, r, wide[:, 3:3 + E], bd, status)
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    assert int(status.item()) == 0
    xf = x.float().numpy()
    key = ref_keys(xf, bias, scoring)
    want = np.array([ref_select(key[t], k, groups, keep, best) for t in range(T)])
    assert np.array_equal(idx.cpu().numpy(), want)
    ww = ref_weights(xf, want, scoring, renorm, scale)
    fin = np.where(np.isfinite(xf), xf, 0)
    # exp: 2 ulp and the rounding of x - max; sums over lanes, quotient, scale
    tol = (32 + 2 * np.ptp(fin)) * U * np.abs(ww)
    got = w.cpu().numpy()
    assert np.all(np.abs(got - ww) <= tol), float(np.max(np.abs(got - ww) / np.maximum(tol, 1e-30)))
    assert np.all(got[want < 0] == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_ties_go_to_the_lowest_index(m, dtype):
    T, E, k = 4, 64, 6
    p = m.problem(T, 128, k, E, 1)
    x = torch.zeros(T, E, dtype=dtype)
    x[1, 40:] = 1.0
    x[2, ::7] = 2.0
    x[3] = torch.arange(E) // 2 % 5
    for scoring in ("softmax", "sigmoid"):
        for groups, keep, best in ((1, 1, 1), (8, 2, 1), (8, 3, 2)):
            idx, _ = run_route(m, p, m.router(scoring, groups, keep, best), x.to(DEV), None)
            key = ref_keys(x.float().numpy(), None, scoring)
            assert idx.tolist() == [ref_select(key[t], k, groups, keep, best) for t in range(T)]


def test_route_infinities_nan_and_extremes(m):
    inf, nan, big = math.inf, math.nan, float(np.finfo(np.float32).max)
    rows = [
        [-inf] * 8,                                   # a padding token
        [nan] * 8,
        [-inf, 1, -inf, nan, -inf, -inf, -inf, -inf],  # one expert left
        [inf, 0, inf, 1, 2, 3, 4, 5],
        [-big, -big, -big, -big, -big, -big, -big, big],
        [-200, -201, -202, -203, -204, -205, -206, -207],   # sigmoids that all round to zero or nearly
    ]
    x = torch.tensor(rows, device=DEV)
    T, E, k = len(rows), 8, 3
    p = m.problem(T, 128, k, E, 1)
    for scoring in ("softmax", "sigmoid"):
        for renorm in (True, False):
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            idx, w = run_route(m, p, m.router(scoring, renormalize=renorm), x, None, st)
            assert int(st.item()) == m.EP_STATUS_BAD_LOGIT
            idx, w = idx.cpu().numpy(), w.cpu().numpy()
            assert np.isfinite(w).all()
            assert (idx[:2] == -1).all() and (w[:2] == 0).all()
            assert idx[2].tolist() == [1, -1, -1] and (w[2, 1:] == 0).all()
            if scoring == "softmax" or renorm:
                assert w[2, 0] == 1
            assert idx[3].tolist() == [0, 2, 7]
            if scoring == "softmax":
                assert w[3].tolist() == [0.5, 0.5, 0]
                assert idx[4, 0] == 7 and w[4].tolist() == [1, 0, 0]
                assert idx[5].tolist() == [0, 1, 2]
            gx = torch.full_like(x, 7.0)
            m.ep_route_backward(p, m.router(scoring, renormalize=renorm), x, torch.from_numpy(idx).to(DEV),
                                torch.ones(T, k, device=DEV), gx, st)
            assert bool(torch.isfinite(gx).all())
            assert bool((gx[:2] == 0).all()) and bool((gx[2, [0, 2, 3, 4, 5, 6, 7]] == 0).all())


def test_route_bias_can_take_an_expert_out(m):
    x = torch.tensor([[3.0, 2.0, 1.0, 0.0]], device=DEV)
    p = m.problem(1, 128, 2, 4, 1)
    bias = torch.tensor([-math.inf, 0.0, 0.0, 2.0], device=DEV)
    for scoring in ("softmax", "sigmoid"):
        idx, w = run_route(m, p, m.router(scoring, renormalize=False), x, bias)
        assert idx.tolist() == [[3, 1]] if scoring == "sigmoid" else sorted(idx.tolist()[0]) == [1, 3]
        want = ref_weights(x.cpu().numpy(), idx.cpu().numpy(), scoring, False, 1.0)
        assert np.all(np.abs(w.cpu().numpy() - want) <= 40 * U * want)   # the bias is not in the weights


def ref_route_grad(x, idx, g, scoring, renorm, scale):
    """The formula in 64 bits, and the size of the terms it sums (for the tolerance)."""
    s = ref_scores(x, scoring)
    T, E = s.shape
    sel = np.zeros((T, E))
    gd = np.zeros((T, E))
    for t in range(T):
        for j, e in enumerate(idx[t]):
            if e >= 0 and x[t, e] > -np.inf:
                sel[t, e] = 1
                gd[t, e] = g[t, j] * scale
    ds, mag = gd, np.abs(gd)
    if renorm:
        tot = (s * sel).sum(1, keepdims=True)
        tot = np.where(tot > 0, tot, np.inf)
        ds = sel * (gd - (gd * s).sum(1, keepdims=True) / tot) / tot
        mag = sel * (np.abs(gd) + (np.abs(gd) * s).sum(1, keepdims=True) / tot) / tot
    if scoring == "sigmoid":
        return ds * s * (1 - s), mag * s
    return s * (ds - (ds * s).sum(1, keepdims=True)), s * (mag + (mag * s).sum(1, keepdims=True))


def ref_loss(x, idx, g, scoring, renorm, scale):
    return (ref_weights(x, idx, scoring, renorm, scale) * g).sum()


@pytest.mark.parametrize("T,E,k,dtype,scoring,renorm,scale,spread", [
    (1, 8, 2, "fp32", "softmax", True, 1.0, 1.0), (5, 40, 8, "fp32", "softmax", False, 2.5, 1.0),
    (33, 256, 8, "bf16", "softmax", False, 1.0, 1.0), (65, 160, 6, "fp32", "sigmoid", True, 2.5, 1.0),
    (7, 1024, 32, "fp32", "softmax", False, 1.0, 3.0), (9, 1001, 5, "bf16", "sigmoid", False, 1.0, 4.0),
    (40, 64, 1, "bf16", "sigmoid", True, 1.0, 1.0), (3, 1, 1, "fp32", "softmax", True, 1.0, 1.0),
    (130, 128, 8, "bf16", "softmax", True, 1.0, 6.0)])
def test_route_backward(m, T, E, k, dtype, scoring, renorm, scale, spread):
    rng = np.random.default_rng(T * E)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32)).to(dt)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int64)
    idx[rng.random((T, k)) < 0.1] = -1
    if T > 4:
        x[2, :] = -math.inf              # a padding token: no entries, no gradient
        idx[2] = -1
        x[3, 0] = -math.inf
    g = rng.standard_normal((T, k)).astype(np.float32)
    p = m.problem(T, 128, k, E, 1)
    r = m.router(scoring, renormalize=renorm, scale=scale)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    wide = torch.zeros((T, E + 3), dtype=dt, device=DEV)
    wide[:, 1:1 + E] = x.to(DEV)
    gx = torch.full((T, E), 7.0, dtype=dt, device=DEV)
    gwide = torch.full((T, E + 7), 7.0, dtype=dt, device=DEV)
    args = (torch.from_numpy(idx).to(DEV), torch.from_numpy(g).to(DEV))
    m.ep_route_backward(p, r, x.to(DEV), *args, gx, st)
    m.ep_route_backward(p, r, wide[:, 1:1 + E], *args, gwide[:, 2:2 + E], st)
    assert torch.equal(gx, gwide[:, 2:2 + E])
    assert bool((gwide[:, :2] == 7).all()) and bool((gwide[:, 2 + E:] == 7).all())
    assert int(st.item()) == 0
    xf = x.float().numpy()
    want, mag = ref_route_grad(xf, idx, g.astype(np.float64), scoring, renorm, scale)
    fin = np.where(np.isfinite(xf), xf, 0)
    tol = (64 + 4 * np.ptp(fin)) * U * mag + 1e-38
    got = gx.float().cpu().numpy()
    if dtype == "bf16":
        assert rounds_to(gx.cpu(), torch.from_numpy(want), torch.from_numpy(tol))
        return
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
    # against central differences of the weights themselves (64 bits, step 1e-5: error below 1e-9 of the terms)
    for t in range(min(T, 6)):
        row = xf[t:t + 1].astype(np.float64)
        for e in range(0, E, max(1, E // 12)):
            if not np.isfinite(row[0, e]):
                continue
            hi, lo = row.copy(), row.copy()
            hi[0, e] += 1e-5
            lo[0, e] -= 1e-5
            a = (idx[t:t + 1], g[t:t + 1].astype(np.float64), scoring, renorm, scale)
            fd = (ref_loss(hi, *a) - ref_loss(lo, *a)) / 2e-5
            assert abs(got[t, e] - fd) <= tol[t, e] + 1e-8 * max(1.0, np.abs(a[1]).sum() * scale)


def test_route_backward_flags_bad_entries(m):
    x = torch.randn(4, 16, device=DEV)
    p = m.problem(4, 128, 3, 16, 1)
    idx = torch.tensor([[0, 1, 2], [3, 3, 4], [99, 5, 6], [-2, 7, 8]], device=DEV)
    clean = torch.tensor([[0, 1, 2], [3, -1, 4], [-1, 5, 6], [-1, 7, 8]], device=DEV)
    g = torch.randn(4, 3, device=DEV)
    for r in (m.router("sigmoid"), m.router("softmax", renormalize=False)):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        got, want = torch.empty_like(x), torch.empty_like(x)
        m.ep_route_backward(p, r, x, idx, g, got, st)
        assert int(st.item()) == m.EP_STATUS_BAD_EXPERT | m.EP_STATUS_DUP_EXPERT
        m.ep_route_backward(p, r, x, clean, g, want)
        assert torch.equal(got, want)


def test_route_feeds_the_layout(m):
    """Ids and weights of ep_route go through layout, dispatch and combine unchanged."""
    T, E, k, R, H = 64, 32, 4, 4, 256
    p = m.problem(T, H, k, E, R)
    x = torch.randn(T, E, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    idx, w = run_route(m, p, m.router("softmax"), x, None, st)
    lb = m.LayoutBuffers(p, DEV).run(p, idx, dev_status=st)
    assert int(lb.tokens_per_expert.sum()) == T * k and int(st.item()) == 0
    assert torch.equal(lb.tokens_per_expert.sum(0).long(), torch.bincount(idx.view(-1), minlength=E))


# --------------------------------------------------------------------------------------------------------------
# combine, backward
# --------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["rank_major", "expert_major"])
@pytest.mark.parametrize("R,Tr,H,E,k,drop", [
    (1, 1, 8, 1, 1, 0.0), (4, 8, 7168, 32, 8, 0.1), (3, 7, 264, 12, 5, 0.3), (2, 33, 1000, 64, 32, 0.2),
    (8, 5, 2056, 8, 8, 0.0), (64, 1, 128, 64, 20, 0.5), (2, 40, 512, 8, 3, 1.0)])
def test_combine_backward(m, layout, R, Tr, H, E, k, drop):
    T = R * Tr
    rng = np.random.default_rng(T + H + E)
    idx_h, _ = inputs.make_routing(T, E, k, seed=T)
    idx_h[rng.random((T, k)) < drop] = -1
    w_h = inputs.make_uniform_weights(T, k, seed=T)
    p = m.problem(T, H, k, E, R)
    idx, w = torch.from_numpy(idx_h).to(DEV), torch.from_numpy(w_h).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    lb = m.LayoutBuffers(p, DEV).run(p, idx, dev_status=st)
    rows = m.ep_recv_rows(p, layout)
    gen = torch.Generator(DEV).manual_seed(T)
    y = torch.randn(rows, H, generator=gen, device=DEV).bfloat16()
    go = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    out = {}
    for which in ("both", "y", "w"):
        gy = torch.full((rows, H), -5.0, dtype=torch.bfloat16, device=DEV) if which != "w" else None
        gw = torch.full((T, k), -5.0, device=DEV) if which != "y" else None
        m.ep_combine_backward(p, layout, go, y if which != "y" else None, idx, w, lb.rank_slot, lb.expert_slot, gy,
                              gw, st)
        out[which] = gy, gw
    assert int(st.item()) == 0
    assert torch.equal(out["both"][0], out["y"][0]) and torch.equal(out["both"][1], out["w"][1])
    gy, gw = out["both"]
    gw = gw.double().cpu()
    # by the definition, entry by entry
    want_gw, bound = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    share = {}
    rs, es = lb.rank_slot.cpu().numpy(), lb.expert_slot.cpu().numpy()
    for t in range(T):
        for j in range(k):
            e = int(idx_h[t, j])
            if e < 0:
                continue
            src = t // Tr
            row = ((e // (E // R)) * R + src) * Tr + rs[t, e // (E // R)] if layout == "rank_major" else \
                (e * R + src) * Tr + es[t, j]
            t0, s0 = share.get(row, (t, np.float32(0)))
            assert t0 == t
            share[row] = (t, np.float32(s0 + w_h[t, j]))
            want_gw[t, j] = row
    live = torch.from_numpy(idx_h >= 0)
    at = want_gw.long()[live]
    tt = torch.arange(T)[:, None].expand(T, k)[live]
    prod = go.cpu().double()[tt] * y.cpu().double()[at]
    want_gw = torch.zeros(T, k, dtype=torch.float64)
    want_gw[live] = prod.sum(1)
    bound[live] = prod.abs().sum(1)
    # a lane's chain of H / 256 products, five halvings, eight warps
    assert bool(((gw - want_gw).abs() <= (H / 256 + 16) * U * bound).all())
    want = torch.full((rows, H), -5.0, dtype=torch.bfloat16)
    if share:
        r = torch.tensor(sorted(share))
        tok = torch.tensor([share[int(i)][0] for i in r])
        sw = torch.tensor([float(share[int(i)][1]) for i in r], dtype=torch.float32)
        want[r] = (sw[:, None] * go.cpu().float()[tok]).bfloat16()
    assert torch.equal(gy.cpu(), want)


def test_combine_backward_matches_differences(m):
    """The forward combine is linear in weights and rows: <grad_out, out> moves by exactly the gradients."""
    R, Tr, H, E, k = 2, 6, 256, 8, 3
    T = R * Tr
    p = m.problem(T, H, k, E, R)
    idx_h, w_h = inputs.make_routing(T, E, k, seed=1)
    idx, w = torch.from_numpy(idx_h).to(DEV), torch.from_numpy(w_h).to(DEV)
    lb = m.LayoutBuffers(p, DEV).run(p, idx)
    rows = m.ep_recv_rows(p, "expert_major")
    y = torch.randn(rows, H, device=DEV).bfloat16()
    go = torch.randn(T, H, device=DEV).bfloat16()
    gw = torch.zeros(T, k, device=DEV)
    m.ep_combine_backward(p, "expert_major", go, y, idx, w, lb.rank_slot, lb.expert_slot, None, gw)

    def loss(weights):
        out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        m.ep_combine(p, "expert_major", y, idx, weights, lb.rank_slot, lb.expert_slot, out)
        return out.double() * go.double()
    # one entry's weight moved by 64: the outputs (bf16, rounded once) of that token move by 64 y
    for t, j in ((0, 0), (5, 2), (11, 1)):
        hi, lo = w.clone(), w.clone()
        hi[t, j] += 64
        lo[t, j] -= 64
        a, b = loss(hi), loss(lo)
        fd = (a - b)[t].sum() / 128
        tol = 2.0 ** -8 * (a.abs() + b.abs())[t].sum() / 128
        assert abs(float(fd - gw[t, j].double())) <= float(tol)


def test_combine_backward_flags_bad_handles(m):
    p = m.problem(4, 128, 2, 4, 2)
    idx = torch.tensor([[0, 0], [1, 9], [2, 3], [-1, 1]], device=DEV)
    w = torch.ones(4, 2, device=DEV)
    es = torch.tensor([[0, 0], [0, 0], [5, 0], [0, 0]], dtype=torch.int32, device=DEV)
    rs = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    y = torch.ones(16, 128, device=DEV).bfloat16()
    go = torch.ones(4, 128, device=DEV).bfloat16()
    gw = torch.full((4, 2), 9.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_combine_backward(p, "expert_major", go, y, idx, w, rs, es, None, gw, st)
    assert int(st.item()) == m.EP_STATUS_BAD_EXPERT | m.EP_STATUS_DUP_EXPERT | m.EP_STATUS_BAD_SLOT
    assert gw.tolist() == [[128, 0], [128, 0], [0, 128], [0, 128]]


# --------------------------------------------------------------------------------------------------------------
# expert products
# --------------------------------------------------------------------------------------------------------------

def cast_blocks(x, rows_per_scale):
    """e4m3 codes and scales of [.., N, K] in blocks of rows_per_scale x 128."""
    *lead, N, K = x.shape
    nb = -(-N // rows_per_scale)
    pad = torch.zeros(*lead, nb * rows_per_scale, K, device=x.device)
    pad[..., :N, :] = x
    b = pad.view(*lead, nb, rows_per_scale, K // 128, 128)
    amax = b.abs().amax((-3, -1))
    q = (b * (448.0 / amax.clamp_min(1e-30))[..., :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(*lead, nb * rows_per_scale, K)[..., :N, :].contiguous(), amax / 448.0


def expert_case(m, R, Tr, E, k, N, K, seed, drop=0.0, counts=None, value=None):
    """Layout and operands: every live receive row is random, the others are NaN codes with NaN scales."""
    T = R * Tr
    rng = np.random.default_rng(seed)
    p = m.problem(T, K, k, E, R)
    if counts is None:
        idx_h, _ = inputs.make_routing(T, E, k, seed=seed)
        idx_h[rng.random((T, k)) < drop] = -1
        counts = m.LayoutBuffers(p, DEV).run(p, torch.from_numpy(idx_h).to(DEV)).tokens_per_expert
    else:
        counts = torch.tensor(counts, dtype=torch.int32, device=DEV)
    gen = torch.Generator(DEV).manual_seed(seed)
    rows = E * T
    c = counts.clamp(0, Tr).t().contiguous()
    live = (torch.arange(Tr, device=DEV) < c[..., None]).reshape(-1)
    a = torch.full((rows, K), 0x7F, dtype=torch.uint8, device=DEV)
    s = torch.full((rows, K // 128), math.nan, device=DEV)
    x = torch.randn(int(live.sum()), K, generator=gen, device=DEV)
    if value is not None:
        x = value(x)
    a[live], s[live] = cast_blocks(x, 1)
    w, ws = cast_blocks(torch.randn(E, N, K, generator=gen, device=DEV) * K ** -0.5, 128)
    return p, counts, live, a, s, w, ws


def product64(live, a, s, w, ws, E):
    """(c, sum of |terms|) for every live row, in 64 bits."""
    rows = torch.nonzero(live)[:, 0]
    N = w.shape[1]
    c = torch.zeros(rows.numel(), N, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(c)
    per = live.numel() // E
    for e in range(E):
        mine = (rows // per) == e
        if not bool(mine.any()):
            continue
        at = rows[mine]
        av = a[at].view(torch.float8_e4m3fn).double() * s[at].double().repeat_interleave(128, 1)
        wv = w[e].view(torch.float8_e4m3fn).double()
        wv = wv * ws[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)[:N]
        c[mine] = av @ wv.t()
        mag[mine] = av.abs() @ wv.abs().t()
    return rows, c, mag


EXPERT = [
    # R, Tr, E, k, K, drop
    (1, 1, 1, 1, 128, 0.0), (1, 1, 8, 2, 256, 0.0), (4, 8, 16, 4, 1024, 0.0), (3, 5, 12, 3, 384, 0.5),
    (2, 61, 4, 2, 640, 0.1), (8, 33, 8, 4, 512, 0.0), (2, 150, 2, 1, 256, 0.0), (64, 3, 64, 8, 128, 0.2),
    (1, 700, 3, 2, 384, 0.0), (5, 7, 5, 2, 256, 1.0),
    (64, 3, 64, 32, 256, 0.1), (16, 20, 16, 4, 384, 0.0),     # many rows in many short segments
]


@pytest.mark.parametrize("N", [8, 128, 200, 384, 520])
@pytest.mark.parametrize("R,Tr,E,k,K,drop", EXPERT)
def test_expert_gemm(m, R, Tr, E, k, K, drop, N):
    p, counts, live, a, s, w, ws = expert_case(m, R, Tr, E, k, N, K, 7 * Tr + N, drop)
    y = torch.full((E * R * Tr, N), -5.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_expert_gemm(p, a, s, w, ws, counts, y, st)
    assert int(st.item()) == 0
    rows, c, mag = product64(live, a, s, w, ws, E)
    # exact products; 128 additions in a block, one product and addition for each block: twice u covers truncation
    assert rounds_to(y[rows], c, (128 + K / 128 + 8) * 2 * U * mag + 1e-30)
    assert bool((y[~live] == -5).all())
    again = torch.full_like(y, -5.0)
    m.ep_expert_gemm(p, a, s, w, ws, counts, again, st)
    assert torch.equal(y, again)


@pytest.mark.parametrize("I", [128, 384])
@pytest.mark.parametrize("R,Tr,E,k,K,drop", EXPERT)
def test_expert_swiglu(m, R, Tr, E, k, K, drop, I):
    p, counts, live, a, s, w, ws = expert_case(m, R, Tr, E, k, 2 * I, K, 5 * Tr + I, drop)
    check_swiglu(m, p, counts, live, a, s, w, ws, E, I, K)


def check_swiglu(m, p, counts, live, a, s, w, ws, E, I, K):
    n = live.numel()
    q = torch.full((n, I), 0x55, dtype=torch.uint8, device=DEV)
    qs = torch.full((n, I // 128), -5.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_expert_swiglu(p, a, s, w, ws, counts, q, qs, st)
    assert int(st.item()) == 0
    assert bool((q[~live] == 0x55).all()) and bool((qs[~live] == -5).all())
    rows, c, mag = product64(live, a, s, w, ws, E)
    if rows.numel() == 0:
        return
    err = (128 + K / 128 + 8) * 2 * U * mag
    g, up, eg, eu = c[:, :I], c[:, I:], err[:, :I], err[:, I:]
    sil = g / (1 + torch.exp(-g))
    h = sil * up
    # |silu'| <= 1.1; exp, quotient and products: a dozen roundings and that of the exponent's argument
    eh = 1.1 * eg * (up.abs() + eu) + sil.abs() * eu + (16 + 2 * g.abs()) * U * h.abs()
    top = h.view(-1, I // 128, 128).abs().amax(2)
    etop = eh.view(-1, I // 128, 128).amax(2)
    scale = qs[rows].double()
    assert bool(((scale - top / 448).abs() <= etop / 448 + 4 * U * top / 448 + 1e-45).all())
    dec = q[rows].view(torch.float8_e4m3fn).double() * scale.repeat_interleave(128, 1)
    step = torch.maximum(2.0 ** -4 * h.abs(), 2.0 ** -10 * scale.repeat_interleave(128, 1))
    tol = step * (1 + 2.0 ** -10) + 1.1 * eh
    assert bool(((dec - h).abs() <= tol).all()), float(((dec - h).abs() / tol).max())


@pytest.mark.parametrize("R,Tr,E,k", [(2, 16, 8, 2), (2, 150, 2, 1)])
def test_expert_outputs_at_sixteen_bytes(m, R, Tr, E, k):
    """Outputs that start 16 bytes off a 32-byte boundary give the same values (few and many rows an expert)."""
    K, N, I, rows = 256, 256, 128, E * R * Tr
    p, counts, live, a, s, w, ws = expert_case(m, R, Tr, E, k, N, K, 4)
    y = torch.zeros(rows * N, dtype=torch.bfloat16, device=DEV)
    y16 = torch.zeros(rows * N + 8, dtype=torch.bfloat16, device=DEV)[8:]
    q, qs = torch.zeros(rows * I, dtype=torch.uint8, device=DEV), torch.zeros(rows, device=DEV)
    q16 = torch.zeros(rows * I + 16, dtype=torch.uint8, device=DEV)[16:]
    assert y16.data_ptr() % 32 == 16 and q16.data_ptr() % 32 == 16
    m.ep_expert_gemm(p, a, s, w, ws, counts, y)
    m.ep_expert_gemm(p, a, s, w, ws, counts, y16)
    m.ep_expert_swiglu(p, a, s, w, ws, counts, q, qs)
    m.ep_expert_swiglu(p, a, s, w, ws, counts, q16, qs)
    assert torch.equal(y, y16) and torch.equal(q, q16)
    assert bool((y != 0).any()) and bool((q != 0).any())


def test_expert_swiglu_large_and_zero_values(m):
    """Gates far from zero (silu is 0 or the gate itself), zero rows (scale 0, codes 0), wide scales."""
    def value(x):
        x[0] = 0
        x[1] *= 1e4
        x[2] *= 1e-12
        return x
    R, Tr, E, K, I = 1, 40, 2, 256, 128
    p, counts, live, a, s, w, ws = expert_case(m, R, Tr, E, 1, 2 * I, K, 3, value=value)
    check_swiglu(m, p, counts, live, a, s, w, ws, E, I, K)
    q, qs = torch.zeros(E * Tr, I, dtype=torch.uint8, device=DEV), torch.ones(E * Tr, 1, device=DEV)
    m.ep_expert_swiglu(p, a, s, w, ws, counts, q, qs)
    zero = torch.nonzero(live)[0, 0]
    assert float(qs[zero, 0]) == 0 and bool((q[zero] & 0x7F == 0).all())


def test_expert_products_clamp_bad_counts(m):
    R, Tr, E, K, N = 2, 4, 4, 128, 64
    bad = [[9, -1, 2, 0], [0, 4, 1, 3]]
    p, counts, live, a, s, w, ws = expert_case(m, R, Tr, E, 1, N, K, 1, counts=bad)
    y = torch.full((E * R * Tr, N), -5.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_expert_gemm(p, a, s, w, ws, counts, y, st)
    assert int(st.item()) == m.EP_STATUS_BAD_SLOT
    good = torch.full_like(y, -5.0)
    m.ep_expert_gemm(p, a, s, w, ws, counts.clamp(0, Tr), good)
    assert torch.equal(y, good) and bool((y[~live] == -5).all())


def test_expert_gemm_one_expert_takes_every_token(m):
    """All rows on one expert of many (tiles of one expert only), and the busiest expert last."""
    R, Tr, E, K, N = 2, 200, 10, 256, 136
    for who in (0, 9):
        counts = np.zeros((R, E), np.int32)
        counts[:, who] = Tr
        p, cnt, live, a, s, w, ws = expert_case(m, R, Tr, E, 1, N, K, who, counts=counts.tolist())
        y = torch.full((E * R * Tr, N), -5.0, dtype=torch.bfloat16, device=DEV)
        m.ep_expert_gemm(p, a, s, w, ws, cnt, y)
        rows, c, mag = product64(live, a, s, w, ws, E)
        assert rounds_to(y[rows], c, (128 + K / 128 + 8) * 2 * U * mag + 1e-30)
        assert bool((y[~live] == -5).all())


def test_operators_on_a_side_stream_and_in_a_graph(m):
    """All of them on a stream that is not the tensors' own, then replayed from a graph with new inputs."""
    R, Tr, E, k, K, I = 2, 16, 8, 2, 256, 128
    T = R * Tr
    p, counts, live, a, s, w, ws = expert_case(m, R, Tr, E, k, 2 * I, K, 2)
    r = m.router("sigmoid", 4, 2, 2)
    x = torch.randn(T, E, device=DEV)
    bufs = dict(idx=torch.zeros(T, k, dtype=torch.int64, device=DEV), w=torch.zeros(T, k, device=DEV),
                gx=torch.zeros(T, E, device=DEV), q=torch.zeros(E * T, I, dtype=torch.uint8, device=DEV),
                qs=torch.zeros(E * T, 1, device=DEV))
    gw = torch.randn(T, k, device=DEV)

    def step():
        m.ep_route(p, r, x, None, bufs["idx"], bufs["w"])
        m.ep_route_backward(p, r, x, bufs["idx"], gw, bufs["gx"])
        m.ep_expert_swiglu(p, a, s, w, ws, counts, bufs["q"], bufs["qs"])
    step()
    want = {n: b.clone() for n, b in bufs.items()}
    side = torch.cuda.Stream()
    for b in bufs.values():
        b.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(bufs[n], want[n]) for n in bufs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.copy_(torch.randn(T, E, device=DEV))
    g.replay()
    got = {n: b.clone() for n, b in bufs.items()}
    step()
    assert all(torch.equal(bufs[n], got[n]) for n in bufs)


def test_empty_problem(m):
    p = m.problem(0, 128, 2, 4, 2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=DEV)
    i64, bf, u8 = torch.int64, torch.bfloat16, torch.uint8
    m.ep_route(p, m.router(), e(0, 4), None, e(0, 2, dt=i64), e(0, 2), st)
    m.ep_route_backward(p, m.router(), e(0, 4), e(0, 2, dt=i64), e(0, 2), e(0, 4), st)
    m.ep_combine_backward(p, "expert_major", e(0, 128, dt=bf), e(0, 128, dt=bf), e(0, 2, dt=i64), e(0, 2), None,
                          e(0, 2, dt=torch.int32), e(0, 128, dt=bf), e(0, 2), st)
    cnt = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    m.ep_expert_gemm(p, e(0, 128, dt=u8), e(0, 1), e(4, 8, 128, dt=u8), e(4, 1, 1), cnt, e(0, 8, dt=bf), st)
    m.ep_expert_swiglu(p, e(0, 128, dt=u8), e(0, 1), e(4, 256, 128, dt=u8), e(4, 2, 1), cnt, e(0, 128, dt=u8),
                       e(0, 1), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0

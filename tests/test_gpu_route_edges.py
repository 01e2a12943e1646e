"""Routing and its gradient where signs and rounding decide."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -24      # unit roundoff of fp32


@pytest.fixture(scope="module")
def m():
    return load_ep()


def choose(m, x, bias, k, router):
    T, E = x.shape
    idx = torch.full((T, k), -7, dtype=torch.int64, device=DEV)
    m.ep_route(m.problem(T, 128, k, E, 1), router, x, bias, idx, torch.empty(T, k, device=DEV))
    return idx.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_zeros_of_either_sign_tie(m, dtype, scoring):
    """-0 and +0 are equal keys, of experts and of groups: the lowest index first."""
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -0.0, 0.0, 0.0, 0.0], [0.0, -0.0] * 4], dtype=dtype, device=DEV)
    for bias in (None, torch.full((8,), -0.0, device=DEV), torch.tensor([-0.0, 0.0] * 4, device=DEV)):
        assert choose(m, x, bias, 5, m.router(scoring)) == [[0, 1, 2, 3, 4]] * 2
        # (32 lanes hold two groups as lanes of their own, or four of them one after the other)
        for groups, best in ((2, 1), (4, 1), (4, 2)):
            per = 8 // groups
            assert choose(m, x, bias, per, m.router(scoring, groups, 1, best)) == [list(range(per))] * 2


def sigmoid_grad64(x, g, renorm, scale):
    """Gradient for rows whose entries are all of x [T, k], and the size of its terms."""
    s, t = 1.0 / (1.0 + np.exp(-x)), 1.0 / (1.0 + np.exp(x))
    if not renorm:
        return scale * g * s * t, np.abs(scale * g) * s * t
    p = s / s.sum(1, keepdims=True)
    return (scale * (g - (g * p).sum(1, keepdims=True)) * p * t,
            scale * (np.abs(g) + (np.abs(g) * p).sum(1, keepdims=True)) * p * t)


@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_at_both_ends(m, renorm):
    rows = [[12.0, 13.0], [16.0, 17.0], [17.5, 12.25], [24.0, 30.0], [30.0, 30.5], [80.0, 88.0], [0.0, 25.0],
            [-84.0, -84.5], [-86.0, -86.5], [-87.0, -88.0], [-88.0, -88.5], [-30.0, -88.0], [-88.0, 20.0]]
    x = np.array(rows, dtype=np.float32)
    T, k, E, scale = len(rows), 2, 6, 2.5
    for g0 in ((20.0, -20.0), (-0.75, 3.0), (1e-3, 1e-3)):
        g = np.tile(np.array(g0, dtype=np.float32), (T, 1))
        logits = torch.full((T, E), -1.0, device=DEV)
        idx = torch.tensor([[4, 1]] * T, device=DEV)
        logits.scatter_(1, idx, torch.from_numpy(x).to(DEV))
        grad = torch.full((T, E), 7.0, device=DEV)
        m.ep_route_backward(m.problem(T, 128, k, E, 1), m.router("sigmoid", renormalize=renorm, scale=scale), logits, idx,
                            torch.from_numpy(g).to(DEV), grad)
        got = grad.gather(1, idx).cpu().double().numpy()
        want, mag = sigmoid_grad64(x.astype(np.float64), g.astype(np.float64), renorm, scale)
        # a score: exp 2 ulp, sum, reciprocal, and its own spacing below 2^-126 (2 u at -88.5); their sum, the quotient,
        # the mean and the products: below 64 u of the terms, and fp32's spacing of a result below 2^-126
        tol = 64 * U * mag + 2.0 ** -149 * max(1.0, np.abs(g).max() * scale)
        assert np.isfinite(got).all()
        assert np.all(np.abs(got - want) <= tol), (g0, rows[int(np.argmax(np.abs(got - want) / tol) // k)])
        rest = torch.ones(T, E, dtype=torch.bool, device=DEV).scatter_(1, idx, False)
        assert bool((grad[rest] == 0).all())
        # and against central differences of the weights (64 bits; step 1e-4: error 1e-8 of the third derivative)
        def loss(z):
            w = 1.0 / (1.0 + np.exp(-z))
            return scale * ((w / w.sum(1, keepdims=True) if renorm else w) * g).sum(1)
        for j in range(k):
            d = np.zeros((1, k))
            d[0, j] = 1e-4
            fd = (loss(x + d) - loss(x.astype(np.float64) - d)) / 2e-4
            assert np.all(np.abs(got[:, j] - fd) <= tol[:, j] + 1e-8 * mag[:, j] + 2e-11 * np.abs(g0).max() * scale)


# --------------------------------------------------------------------------------------------------------------
# softmax with the score as the key
# --------------------------------------------------------------------------------------------------------------

def softmax64(x):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x.astype(np.float64), np.finfo(np.float32).max))
    top = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def score_keys64(x, bias):
    key = softmax64(x) + (0 if bias is None else bias.astype(np.float64))
    return np.where((x > -np.inf) & (key > -np.inf), key, -np.inf)


def select64(key, k, groups, keep, best):
    """One row's choice: best first, lowest id among equals, -1 for none."""
    E = key.size
    per = E // groups
    if groups > 1:
        score = []
        for g in range(groups):
            v = [z for z in sorted(key[g * per:(g + 1) * per], reverse=True)[:best] if z > -np.inf]
            score.append(sum(v) if v else -np.inf)
        kept = sorted((g for g in range(groups) if score[g] > -np.inf), key=lambda g: (-score[g], g))[:keep]
        key = np.array([key[e] if e // per in kept else -np.inf for e in range(E)])
    ids = sorted((e for e in range(E) if key[e] > -np.inf), key=lambda e: (-key[e], e))[:k]
    return ids + [-1] * (k - len(ids))


def near(v, rel, off):
    """Rows in which two different numbers of v are nearer than rel of the larger, and off."""
    v = np.sort(v, 1)
    with np.errstate(invalid="ignore"):
        d = np.diff(v, axis=1)
        return ((d > 0) & (d < rel * np.maximum(np.abs(v[:, 1:]), np.abs(v[:, :-1])) + off)).any(1)


@pytest.mark.parametrize("T,E,k,dtype,with_bias,groups,keep,best,renorm,spread,masked", [
    (1, 8, 2, "bf16", True, 1, 1, 1, True, 1.0, 0.0), (64, 256, 8, "fp32", True, 1, 1, 1, True, 1.0, 0.0),
    (33, 256, 8, "bf16", True, 8, 4, 2, True, 1.0, 0.1), (50, 160, 6, "fp32", False, 8, 3, 2, False, 2.0, 0.0),
    (40, 60, 4, "bf16", True, 5, 2, 2, False, 1.0, 0.6), (20, 1024, 32, "fp32", True, 64, 40, 2, True, 1.0, 0.3),
    (25, 999, 9, "fp32", False, 3, 2, 2, True, 1.0, 0.0), (37, 1, 1, "fp32", True, 1, 1, 1, False, 1.0, 0.3),
    (16, 512, 8, "bf16", True, 16, 4, 1, True, 0.5, 0.98)])
def test_softmax_score_keys(m, T, E, k, dtype, with_bias, groups, keep, best, renorm, spread, masked):
    rng = np.random.default_rng(7 * T + E)
    # a balance bias: a quarter of the mean score, in steps of 1 / 1024 of it
    bias = (np.round(rng.standard_normal(E) * 256) / (1024 * E)).astype(np.float32) if with_bias else None
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    draw = lambda n: torch.from_numpy((rng.standard_normal((n, E)) * spread).astype(np.float32)).to(dt)
    x = draw(T)
    off = torch.from_numpy(rng.random((T, E)) < masked)
    x[off] = -math.inf
    for _ in range(60):
        key = score_keys64(x.float().numpy(), bias)
        # a score's error: exp 2 ulp, the rounding of x - max, sums and quotient: below (32 + range) u of it; a key's
        # score is at most the key and the bias
        fin = np.where(np.isfinite(x.float().numpy()), x.float().numpy(), 0)
        rel = 2 * (32 + np.ptp(fin)) * U
        off_b = 0.0 if bias is None else rel * float(np.abs(bias).max())
        bad = near(key, rel, off_b)
        if groups > 1:
            v = -np.sort(-key.reshape(T, groups, -1), 2)[:, :, :best]
            bad |= near(np.where(v > -np.inf, v, 0).sum(2), rel, 2 * off_b)
        if not bad.any():
            break
        x[torch.from_numpy(bad)] = draw(int(bad.sum())).masked_fill_(off[torch.from_numpy(bad)], -math.inf)
    assert not bad.any()
    r = m.router("softmax", groups, keep, best, renorm, 1.5, softmax_key="score")
    p = m.problem(T, 128, k, E, 1)
    idx, w = torch.full((T, k), -7, dtype=torch.int64, device=DEV), torch.full((T, k), -7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_route(p, r, x.to(DEV), None if bias is None else torch.from_numpy(bias).to(DEV), idx, w, st)
    assert int(st.item()) == 0
    want = np.array([select64(key[t], k, groups, keep, best) for t in range(T)])
    assert np.array_equal(idx.cpu().numpy(), want)
    s = np.where(want >= 0, np.take_along_axis(softmax64(x.float().numpy()), np.maximum(want, 0), 1), 0.0)
    if renorm:
        s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
    assert np.all(np.abs(w.cpu().numpy() - 1.5 * s) <= (32 + 2 * np.ptp(fin)) * U * 1.5 * s)


def test_softmax_keys_choose_differently(m):
    """Where the two keys differ: groups scored by two keys, one of them with one eligible expert, and a small bias."""
    inf = math.inf
    x = torch.tensor([[-1.0, -inf, -0.9, -0.8], [-3.0, -inf, -1.0, -1.1]], device=DEV)
    for key, first in (("score", [[3, 2], [2, 3]]), ("logit", [[0, -1], [2, 3]])):
        r = m.router("softmax", 2, 1, 2, softmax_key=key)
        if key == "logit":
            assert choose(m, x[:1], None, 2, r) == first[:1]        # -1 against -1.7
        else:
            assert choose(m, x, None, 2, r) == first
    E = 256
    x = torch.zeros(1, E, device=DEV)
    x[0, 0] = 0.1                              # scores 1.1 / 256 and 1 / 256: a bias of 0.001 is a quarter of one
    bias = torch.zeros(E, device=DEV)
    bias[200] = 0.001
    assert choose(m, x, bias, 2, m.router("softmax", softmax_key="score")) == [[200, 0]]
    assert choose(m, x, bias, 2, m.router("softmax", softmax_key="logit")) == [[0, 200]]


def test_softmax_score_keys_extremes(m):
    inf, nan, big = math.inf, math.nan, float(np.finfo(np.float32).max)
    x = torch.tensor([[-inf] * 4, [nan] * 4, [nan, 1.0, -inf, 0.0], [inf, 0.0, inf, 1.0], [-big, -big, -big, big],
                      [-200.0, 0.0, -300.0, -400.0]], device=DEV)
    T, E, k = 6, 4, 3
    for renorm in (True, False):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        idx, w = torch.zeros(T, k, dtype=torch.int64, device=DEV), torch.zeros(T, k, device=DEV)
        m.ep_route(m.problem(T, 128, k, E, 1), m.router("softmax", renormalize=renorm, softmax_key="score"), x, None, idx,
                   w, st)
        assert int(st.item()) == m.EP_STATUS_BAD_LOGIT
        # scores that round to 0 tie: the lowest index
        assert idx.tolist() == [[-1] * 3, [-1] * 3, [1, 3, -1], [0, 2, 1], [3, 0, 1], [1, 0, 2]]
        assert bool(torch.isfinite(w).all()) and w[3].tolist() == [0.5, 0.5, 0] and w[4].tolist() == [1, 0, 0]
    bias = torch.tensor([-inf, 0.0, 0.0, 2.0], device=DEV)
    r = m.router("softmax", softmax_key="score")
    assert choose(m, torch.tensor([[3.0, 2.0, 1.0, 0.0]], device=DEV), bias, 4, r) == [[3, 1, 2, -1]]

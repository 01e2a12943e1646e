"""Routing and its gradient where signs and rounding decide."""
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

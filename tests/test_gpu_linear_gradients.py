"""Gradients of the dense products against the products of what the kernels multiply: the gradient of the
pre-activations rounded to bf16 (either neighbour, where the slope's fp32 steps leave the rounding open), so that the
tolerance is that of an fp32 sum and a single row or column that is left out shows.  Both products' kernels, rows of the
outputs that start anywhere, and fp32 results in several turns and column tiles.
"""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep
from test_gpu_linear import ACTS, U, act64, act_tol, grad64, make, within

pytestmark = pytest.mark.gpu

KERNELS = ["EP_LINEAR_FEW_ROWS", "EP_LINEAR_MANY_ROWS"]


@pytest.fixture(scope="module")
def m():
    return load_ep()


def strided(M, K, before, behind, dtype=torch.bfloat16):
    """(the whole, a view [M, K] of it whose rows have `before` numbers in front and `behind` after them)"""
    whole = torch.full((M, before + K + behind), 7.0, dtype=dtype, device=DEV)
    return whole, whole[:, before:before + K]


def check(m, kernel, M, K, N, act, grad32, w32, before=0, behind=0, seed=0):
    x, w, _, rand, wide = make(M, K, N, act, seed)
    g = rand(M, N).to(torch.float32 if grad32 else torch.bfloat16)
    pre = None if act == "none" else (rand(M, wide) * 2).bfloat16()
    whole, gx = strided(M, K, before, behind)
    gw = torch.full((wide, K), 7.0, dtype=torch.float32 if w32 else torch.bfloat16, device=DEV)
    ws = torch.full((m.ep_linear_backward_workspace_bytes(M, K, N, act),), 255, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_selftest_linear_backward(getattr(m, kernel), 1 << 32, g, x, w, gx, gw, None, pre, act, ws, st)
    assert m.ep_get_status(st) == 0
    assert bool((whole[:, :before] == 7).all()) and bool((whole[:, before + K:] == 7).all())
    G = grad64(g.double(), None if pre is None else pre.double(), act, N)
    a = g.double().abs()
    if act in ("none", "relu"):
        e32 = torch.zeros_like(G)
    elif act == "swiglu":
        gate, up = pre.double()[:, :N].abs(), pre.double()[:, N:].abs()
        e32 = 256 * U * torch.cat([a * (1 + up) * (1 + gate), a * (1 + gate)], 1)
    else:
        e32 = 256 * U * a * (1 + pre.double().abs())
    lo, hi = ((G + s * e32).float().bfloat16().double() for s in (-1, 1))
    mid, rad = (lo + hi) / 2, (hi - lo) / 2
    xd, wd = x.double(), w.double()
    size = mid.abs() + rad
    assert within(gx, mid @ wd, rad @ wd.abs() + 2 * (wide + 16) * U * (size @ wd.abs()))
    want = mid.t() @ xd
    assert within(gw, want, rad.t() @ xd.abs() + 2 * (M + 64) * U * (size.t() @ xd.abs()) + U * want.abs())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(3, 64, 9), (130, 136, 304), (515, 200, 129), (700, 1032, 520)])
def test_products_of_the_rounded_gradient(m, kernel, act, M, K, N):
    check(m, kernel, M, K, N, act, False, False)
    check(m, kernel, M, K, N, act, True, True, seed=1)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("before,behind", [(0, 1), (1, 0), (2, 2), (8, 0), (3, 13), (16, 16)])
@pytest.mark.parametrize("M,K,N", [(1, 64, 5), (70, 72, 40), (300, 520, 64), (2100, 264, 33)])
def test_rows_of_grad_x_start_anywhere(m, kernel, M, K, N, before, behind):
    check(m, kernel, M, K, N, "none", False, False, before, behind)
    check(m, kernel, M, K, N, "silu", True, False, before, behind, seed=1)


@pytest.mark.parametrize("M,K,N,act,extra", [(20000, 136, 600, "none", 0), (9000, 72, 1111, "gelu", 0),
                                             (10240, 520, 1024, "silu", 8), (20000, 64, 300, "swiglu", 1)])
def test_fp32_results_in_turns_and_column_tiles(m, M, K, N, act, extra):
    """More tiles than pairs of SMs, and several of them beside each other."""
    x, w, b, rand, wide = make(M, K, N, act, 9)
    res = rand(M, N).bfloat16()
    whole, out = strided(M, N, 0, extra, torch.float32)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_selftest_linear(m.EP_LINEAR_MANY_ROWS, 1 << 32, x, w, out, bias=b, residual=res, activation=act, dev_status=st)
    assert m.ep_get_status(st) == 0 and bool((whole[:, N:] == 7).all())
    z = x.double() @ w.double().t() + b.double()
    ez = 2 * (K + 16) * U * (x.double().abs() @ w.double().abs().t()) + 2 * U * z.abs()
    y, tol = act64(z, act, N) + res.double(), act_tol(z, ez, act, N)
    assert within(out, y, tol + 2 * U * (y.abs() + tol))

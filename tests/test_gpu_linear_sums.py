"""Sums of the dense products over long contractions.

The tensor core cuts its sums off, so that an accumulator of numbers of one sign lags behind: by up to two units in the
last place (2^-23 of it each) for every 16 products, over a whole contraction of K by K / 16 times 2^-23, because it grows
evenly.  Operands here have one sign, and the same distribution all along.
"""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return load_ep()


def outer(rows, K, gen, scale):
    """bf16 [rows, K] = a[row] * u[k], exact: both have 4 significant bits, between 1 and 2 (u: times `scale`)."""
    draw = lambda n: 1 + torch.randint(0, 8, (n,), generator=gen, device=DEV).double() / 8
    a, u = draw(rows), draw(K) * scale
    return a, u, a.bfloat16()[:, None] * u.bfloat16()[None, :]


def lag(K, most=512):
    """Relative error of a sum of K products of one sign in accumulators of at most `most` of them, added in fp32."""
    return (min(K, most) / 16 + 1) * 2.0 ** -23 + (K / most + 32) * 2.0 ** -24


def rounds(got, want, rel):
    """got is the rounding to its type of a number within `rel` of want (which is positive)."""
    lo, hi = (want * (1 - rel)).float().to(got.dtype), (want * (1 + rel)).float().to(got.dtype)
    return bool(((lo <= got) & (got <= hi)).all())


@pytest.mark.parametrize("form", ["forward", "swiglu", "grad_x", "grad_w"])
def test_bf16_results_of_long_contractions(m, form):
    """So many tiles that no contraction is split: 2^19 products of one sign, of which one accumulator would lose 3e-3, nearly
    the distance of two bf16 numbers."""
    L, R, C = 1 << 19, 1024, 4864
    gen = torch.Generator(DEV).manual_seed(1)
    # (sums of about 9 for the activation, where silu's slope is 1 to 1e-3 beside its own argument)
    a, u, A = outer(R, L, gen, 2.0 ** -9)
    b, v, B = outer(C, L, gen, 2.0 ** -9)
    z = a[:, None] * b[None, :] * (u * v).sum()
    rel = lag(L)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    if form == "forward":
        got = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
        m.ep_linear(A, B, got, dev_status=st)
    elif form == "swiglu":
        got = torch.empty(R, C // 2, dtype=torch.bfloat16, device=DEV)
        m.ep_linear(A, B, got, activation="swiglu", dev_status=st)
        g, up = z[:, :C // 2], z[:, C // 2:]
        z = g * torch.sigmoid(g) * up
        rel = 2.2 * rel + 64 * 2.0 ** -24
    elif form == "grad_x":                                  # sum over n of G[m, n] w[n, i]
        got = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
        w = B.t().contiguous()
        ws = torch.empty(m.ep_linear_backward_workspace_bytes(R, C, L), dtype=torch.uint8, device=DEV)
        m.ep_linear_backward(A, torch.empty_like(got), w, grad_x=got, workspace=ws, dev_status=st)
    else:                                                   # sum over m of G[m, n] x[m, i]
        got = torch.empty(R, C, dtype=torch.bfloat16, device=DEV)
        G, x = A.t().contiguous(), B.t().contiguous()
        ws = torch.empty(m.ep_linear_backward_workspace_bytes(L, C, R), dtype=torch.uint8, device=DEV)
        m.ep_linear_backward(G, x, got, grad_w=got, workspace=ws, dev_status=st)
    assert m.ep_get_status(st) == 0
    assert rounds(got, z, rel)


@pytest.mark.parametrize("K,most", [(1024, 1024), (8192, 8192), (8200, 512), (32768, 512)])
def test_bf16_results_do_not_lag(m, K, most):
    """The mean error of many outputs, whose roundings cancel: one accumulator of 32768 would be 1.5e-4 behind."""
    M = N = 2048
    gen = torch.Generator(DEV).manual_seed(2)
    rand = lambda rows: ((torch.rand(rows, K, generator=gen, device=DEV) / 2 + 0.5) *
                         (torch.rand(rows, 1, generator=gen, device=DEV) + 1)).bfloat16()
    x, w = rand(M), rand(N)
    out = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    m.ep_linear(x, w, out)
    want = x.double() @ w.double().t()
    # (roundings are independent, at most 2^-8 each: of their mean over 2^22, 5 standard deviations of 2^-8 / 3^0.5 / 2^11)
    assert abs(float(((out.double() - want) / want).mean())) <= lag(K, most) + 5 * 2.0 ** -8 / 3 ** 0.5 / 2 ** 11


@pytest.mark.parametrize("kernel", ["EP_LINEAR_FEW_ROWS", "EP_LINEAR_MANY_ROWS"])
@pytest.mark.parametrize("M,N,K", [(16, 256, 7168), (16, 256, 65536), (48, 200, 4096)])
def test_fp32_results_do_not_lag(m, kernel, M, N, K):
    """Every output, not the mean: a whole contraction of 7168 in one accumulator would be 2.6e-5 behind."""
    gen = torch.Generator(DEV).manual_seed(3)
    x, w = ((torch.rand(r, K, generator=gen, device=DEV) / 2 + 0.5).bfloat16() for r in (M, N))
    out = torch.empty(M, N, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_selftest_linear(getattr(m, kernel), 1 << 32, x, w, out, dev_status=st)
    assert m.ep_get_status(st) == 0
    want = x.double() @ w.double().t()
    assert bool(((out.double() - want).abs() <= lag(K) * want).all())


@pytest.mark.parametrize("M,N,K", [(2433, 256, 7168), (2432, 256, 7168), (700, 2048, 7168), (1, 256, 1 << 18)])
def test_fp32_results_do_not_lag_by_choice(m, M, N, K):
    """The same by whichever kernel the call takes."""
    gen = torch.Generator(DEV).manual_seed(4)
    x, w = ((torch.rand(r, K, generator=gen, device=DEV) / 2 + 0.5).bfloat16() for r in (M, N))
    out = torch.empty(M, N, device=DEV)
    m.ep_linear(x, w, out)
    want = x.double() @ w.double().t()
    assert bool(((out.double() - want).abs() <= lag(K) * want).all())


@pytest.mark.parametrize("M,N,K", [(65536, 64, 512), (65536, 1024, 1024), (9000, 8, 64)])
def test_fp32_matrix_gradients_do_not_lag(m, M, N, K):
    gen = torch.Generator(DEV).manual_seed(5)
    g, x = ((torch.rand(M, c, generator=gen, device=DEV) / 2 + 0.5).bfloat16() for c in (N, K))
    gw, gb = torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(M, K, N), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(g, x, torch.empty(N, K, dtype=torch.bfloat16, device=DEV), grad_w=gw, grad_bias=gb, workspace=ws)
    want = g.double().t() @ x.double()
    assert bool(((gw.double() - want).abs() <= lag(M) * want).all())
    # (fp32 sums of at most M / 8 rows of a block and a lane, rounded to nearest)
    assert bool(((gb.double() - g.double().sum(0)).abs() <= (M / 8 + 32) * 2.0 ** -25 * g.double().sum(0)).all())

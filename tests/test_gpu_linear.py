"""The dense products with an epilogue and their gradients against their definitions in 64 bits.

Tolerances follow from the arithmetic: u = 2^-24 is fp32's unit roundoff.  A sum of n products, in any order, each
step rounded or cut off to 24 bits, is within 2 (n + 16) u of the sum of the products' magnitudes.  A bf16 output has to
be the rounding of a value within that: it lies between the roundings of the tolerance's two ends.
"""
import math

import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GA, GB = math.sqrt(2 / math.pi), 0.044715
ACTS = ["none", "relu", "silu", "gelu", "swiglu"]


@pytest.fixture(scope="module")
def m():
    return load_ep()


def within(got, want, tol):
    """got rounds a value of want +- tol (infinities and NaN of want have to be the same)."""
    fine = torch.isfinite(want)
    if not torch.equal(fine, torch.isfinite(got)) or not torch.equal(torch.isnan(want), torch.isnan(got)):
        return False
    if not torch.equal(torch.where(torch.isinf(want), want, 0.0).to(got.dtype), torch.where(torch.isinf(got), got, 0.0)):
        return False
    want, tol = torch.where(fine, want, 0.0), torch.where(fine, tol, 0.0)
    got = torch.where(fine, got, 0.0)
    lo, hi = (want - tol).float().to(got.dtype), (want + tol).float().to(got.dtype)
    return bool(((lo <= got) & (got <= hi)).all())


def act64(z, act, N):
    if act == "swiglu":
        return z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * (1 + torch.tanh(GA * (z + GB * z ** 3)))}[act]()


def act_tol(z, ez, act, N):
    """How far act may be off where z is off by ez, with its own roundings (a dozen, each of relative size u, beside
    sigmoid's argument whose error grows with it: |u'| <= 2 |z| (1 + z^2))."""
    if act == "none" or act == "relu":
        return ez
    if act == "swiglu":
        g, p = z[:, :N], z[:, N:]
        y = (g * torch.sigmoid(g) * p).abs()
        return 1.1 * ez[:, :N] * (p.abs() + ez[:, N:]) + (g * torch.sigmoid(g)).abs() * ez[:, N:] + y * U * (16 + 2 * g.abs())
    y = act64(z, act, N).abs()
    grow = 2 * z.abs() if act == "silu" else 8 * z.abs() * (1 + z * z)
    return 1.2 * ez + z.abs() * U * (16 + grow) * torch.sigmoid(-z.abs() / 2 if act == "silu" else -z.abs()).clamp_min(0) + y * 16 * U


def make(M, K, N, act, seed=0, xs=0, scale=1.0):
    g = torch.Generator(DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    wide = 2 * N if act == "swiglu" else N
    x = (rand(M, K + xs) * scale).bfloat16()[:, :K]
    return x, (rand(wide, K) * K ** -0.5).bfloat16(), rand(wide), rand, wide


def check_forward(m, M, K, N, act, bias, residual, out32, pre, xs=0, extra=0, seed=0):
    x, w, b, rand, wide = make(M, K, N, act, seed, xs)
    b = b if bias else None
    res = rand(M, N + extra).bfloat16()[:, :N] if residual else None
    store = torch.full((M, N + extra), 7.0, dtype=torch.float32 if out32 else torch.bfloat16, device=DEV)
    out = store[:, :N]
    pr = torch.empty(M, wide, dtype=torch.bfloat16, device=DEV) if pre else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_linear(x, w, out, bias=b, residual=res, pre=pr, activation=act, dev_status=st)
    assert m.ep_get_status(st) == 0
    z = x.double() @ w.double().t() + (b.double() if bias else 0)
    mag = x.double().abs() @ w.double().abs().t()
    ez = 2 * (K + 16) * U * mag + (2 * U * z.abs() if bias else 0)
    y, tol = act64(z, act, N), act_tol(z, ez, act, N)
    if residual:
        y = y + res.double()
        tol = tol + U * (y.abs() + tol)
    assert within(out, y, tol + U * y.abs())
    if pre:
        assert within(pr, z, ez)
    if extra:
        assert bool((store[:, N:] == 7).all())
    again = torch.empty_like(store)[:, :N]
    m.ep_linear(x, w, again, bias=b, residual=res, activation=act)
    assert torch.equal(out, again)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (3, 8, 1), (40, 200, 77), (130, 136, 300), (257, 512, 129), (600, 72, 515),
                                   (1500, 64, 1030), (1300, 136, 1807), (1400, 200, 1284)])
def test_linear(m, act, M, K, N):
    check_forward(m, M, K, N, act, True, True, False, True)
    check_forward(m, M, K, N, act, False, False, True, False, seed=1)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 47, 63, 64, 65, 100, 127, 128, 129, 255, 256])
@pytest.mark.parametrize("act,K,N", [("none", 1024, 256), ("swiglu", 576, 384)])
def test_linear_row_counts(m, act, K, N, M):
    check_forward(m, M, K, N, act, False, True, act == "none", False)


@pytest.mark.parametrize("M,K,N,xs,extra", [(33, 128, 64, 8, 3), (300, 264, 96, 24, 8), (5, 64, 31, 64, 1), (70, 64, 128, 0, 16)])
@pytest.mark.parametrize("out32", [False, True])
def test_linear_row_strides(m, M, K, N, xs, extra, out32):
    check_forward(m, M, K, N, "silu", True, True, out32, True, xs, extra)


@pytest.mark.parametrize("M,K,N", [(5, 7168, 256), (300, 7168, 320), (2048, 1024, 1024)])
def test_linear_long(m, M, K, N):
    check_forward(m, M, K, N, "none", False, False, True, False)


def test_linear_into_its_residual(m):
    for M, N in ((9, 200), (300, 333)):
        x, w, b, rand, _ = make(M, 128, N, "gelu")
        res = rand(M, N).bfloat16()
        want = torch.empty_like(res)
        m.ep_linear(x, w, want, bias=b, residual=res, activation="gelu")
        m.ep_linear(x, w, res, bias=b, residual=res, activation="gelu")
        assert torch.equal(res, want)


@pytest.mark.parametrize("M", [4, 300])
def test_linear_infinities_and_nan(m, M):
    """A row of x with NaN or infinity spoils its own outputs only; large pre-activations saturate, not overflow."""
    K, N = 128, 160
    x, w, b, _, _ = make(M, K, N, "silu")
    clean = torch.empty(M, N, device=DEV)
    m.ep_linear(x, w, clean, activation="silu")
    x[1, 5] = math.nan
    x[2, 9] = math.inf
    out = torch.empty(M, N, device=DEV)
    m.ep_linear(x, w, out, activation="silu")
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(out[keep], clean[keep]) and bool(torch.isnan(out[1]).all())
    z = x[2].double() @ w.double().t()
    assert bool((out[2][z == math.inf] == math.inf).all())
    for act in ("silu", "gelu"):
        x.fill_(1e4)
        m.ep_linear(x, w, out, activation=act)
        z = x.double() @ w.double().t()
        far = z.abs() > 1e3
        assert bool(((out.double() - z.clamp_min(0)).abs() <= 2 * (K + 32) * U * (x.double().abs() @ w.double().abs().t()))[far].all())


def test_linear_no_rows(m):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(8, 64, dtype=torch.bfloat16, device=DEV)
    m.ep_linear(x, w, torch.empty(0, 8, device=DEV))
    gw, gb = torch.ones(8, 64, device=DEV), torch.ones(8, device=DEV)
    m.ep_linear_backward(torch.empty(0, 8, device=DEV), x, w, grad_w=gw, grad_bias=gb)
    assert bool((gw == 0).all()) and bool((gb == 0).all())


# --------------------------------------------------------------------------------------------------------------
# gradients
# --------------------------------------------------------------------------------------------------------------

def grad64(g, z, act, N):
    if act == "none":
        return g
    if act == "relu":
        return torch.where(z > 0, g, 0.0)
    zz = z.clone().requires_grad_()
    act64(zz, act, N).backward(g)
    return zz.grad


def check_backward(m, M, K, N, act, grad32, w32, bias=True, gs=0, xs=0, which="xwb", seed=0):
    x, w, _, rand, wide = make(M, K, N, act, seed, xs)
    g = rand(M, N + gs).to(torch.float32 if grad32 else torch.bfloat16)[:, :N]
    pre = None if act == "none" else (rand(M, wide) * 2).bfloat16()
    gx = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV) if "x" in which else None
    gw = torch.full((wide, K), 7.0, dtype=torch.float32 if w32 else torch.bfloat16, device=DEV) if "w" in which else None
    gb = torch.full((wide,), 7.0, device=DEV) if "b" in which else None
    ws = torch.full((m.ep_linear_backward_workspace_bytes(M, K, N, act) + 16,), 255, dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_linear_backward(g, x, w, gx, gw, gb, pre, act, ws[:-16], st)
    assert m.ep_get_status(st) == 0
    assert bool((ws[-16:] == 255).all())
    G = grad64(g.double(), None if pre is None else pre.double(), act, N)
    # fp32 steps of the slope: a dozen of size u, the sigmoid's argument growing to some 50 for |z| <= 10
    a = g.double().abs()
    if act in ("none", "relu"):
        e32 = torch.zeros_like(G)
    elif act == "swiglu":
        gate, up = pre.double()[:, :N].abs(), pre.double()[:, N:].abs()
        e32 = 256 * U * torch.cat([a * (1 + up) * (1 + gate), a * (1 + gate)], 1)
    else:
        e32 = 256 * U * a * (1 + pre.double().abs())
    exact = act in ("none", "relu") and not grad32
    eg = e32 + (0 if exact else 2.0 ** -8 * (G.abs() + e32))
    xd, wd = x.double(), w.double()
    if gx is not None:
        tol = eg @ wd.abs() + 2 * (wide + 16) * U * ((G.abs() + eg) @ wd.abs())
        assert within(gx, G @ wd, tol)
    if gw is not None:
        tol = eg.t() @ xd.abs() + 2 * (M + 64) * U * ((G.abs() + eg).t() @ xd.abs())
        assert within(gw, G.t() @ xd, tol + U * (G.t() @ xd).abs())
    if gb is not None:
        assert within(gb, G.sum(0), e32.sum(0) + 2 * (M + 16) * U * G.abs().sum(0))
    return g, x, w, pre, ws, gx, gw, gb


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (3, 8, 1), (40, 200, 77), (130, 136, 304), (515, 72, 129), (1000, 264, 64)])
def test_backward(m, act, M, K, N):
    check_backward(m, M, K, N, act, False, False)
    check_backward(m, M, K, N, act, True, True, seed=1)


@pytest.mark.parametrize("M,K,N", [(20, 128, 1000), (64, 256, 300), (200, 1000, 65), (96, 520, 129)])
@pytest.mark.parametrize("w32", [False, True])
def test_backward_tiles_of_rows(m, M, K, N, w32):
    """Rows of the matrix's gradient in several tiles, which start where copies may start."""
    check_backward(m, M, K, N, "none", False, w32)
    check_backward(m, M, K, N, "swiglu", True, w32)


@pytest.mark.parametrize("M,K,N", [(2500, 9000, 64), (2100, 8712, 200), (19500, 1040, 256), (2300, 9216, 33)])
def test_backward_short_contractions(m, M, K, N):
    """grad_x of a few outputs and many inputs: a part of the matrix stays in shared memory."""
    check_backward(m, M, K, N, "none", False, False, which="x")
    check_backward(m, M, K, N, "silu", True, False, which="x", gs=8)


@pytest.mark.parametrize("which", ["x", "w", "b", "xw", "wb"])
def test_backward_some_outputs(m, which):
    check_backward(m, 100, 128, 96, "none", False, True, which=which)
    check_backward(m, 100, 128, 96, "swiglu", True, False, which=which)


@pytest.mark.parametrize("gs,xs", [(3, 8), (8, 0), (16, 24)])
@pytest.mark.parametrize("grad32", [False, True])
def test_backward_row_strides(m, gs, xs, grad32):
    check_backward(m, 70, 136, 64, "none", grad32, False, gs=gs, xs=xs)
    check_backward(m, 70, 136, 56, "swiglu", grad32, False, gs=gs, xs=xs)


@pytest.mark.parametrize("M,K,N", [(9000, 512, 64), (64, 1024, 5000), (4096, 1024, 1024)])
def test_backward_split_contractions(m, M, K, N):
    g, x, w, pre, ws, gx, gw, gb = check_backward(m, M, K, N, "none", False, True)
    again = torch.empty_like(gx), torch.empty_like(gw), torch.empty_like(gb)
    m.ep_linear_backward(g, x, w, *again, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(again, (gx, gw, gb)))


@pytest.mark.parametrize("act", ACTS)
def test_backward_matches_differences(m, act):
    """The gradients against differences of the forward formula in 64 bits, at the bf16 pre-activations."""
    M, K, N = 6, 16, 5
    x, w, b, rand, wide = make(M, K, N, act, 3)
    pre, out = torch.empty(M, wide, dtype=torch.bfloat16, device=DEV), torch.empty(M, N, device=DEV)
    m.ep_linear(x, w, out, bias=b, pre=pre, activation=act)
    g = rand(M, N).bfloat16()
    gx, gw, gb = torch.empty_like(x), torch.empty(wide, K, device=DEV), torch.empty(wide, device=DEV)
    ws = torch.empty(max(16, m.ep_linear_backward_workspace_bytes(M, K, N, act)), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(g, x, w, gx, gw, gb, None if act == "none" else pre, act, ws)
    shift = pre.double() - (x.double() @ w.double().t() + b.double())      # the rounding of the pre-activations

    def loss(x_, w_, b_):
        return (act64(x_ @ w_.t() + b_ + shift, act, N) * g.double()).sum()
    xd, wd, bd, h = x.double(), w.double(), b.double(), 1e-4
    for got, at, n in ((gx, 0, 11), (gw, 1, 17), (gb, 2, 3)):
        args = [xd, wd, bd]
        i = tuple(int(v) for v in torch.unravel_index(torch.tensor(n % args[at].numel()), args[at].shape))
        d = torch.zeros_like(args[at])
        d[i] = h
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + d, args[at] - d
        fd = float(loss(*up) - loss(*dn)) / (2 * h)
        # G's rounding (2^-8 of each of up to 10 terms of size 4) and the differences' own error
        assert abs(fd - float(got[i])) <= 2.0 ** -8 * (abs(fd) + 40), (act, at)


def test_linear_on_another_stream_and_in_a_graph(m):
    M, K, N = 200, 128, 96
    x, w, b, rand, _ = make(M, K, N, "swiglu")
    g = rand(M, N).bfloat16()
    out, pre = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(M, 2 * N, dtype=torch.bfloat16, device=DEV)
    gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty(2 * N, device=DEV)
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(M, K, N, "swiglu"), dtype=torch.uint8, device=DEV)

    def both(stream=None):
        m.ep_linear(x, w, out, bias=b, pre=pre, activation="swiglu", stream=stream)
        m.ep_linear_backward(g, x, w, gx, gw, gb, pre, "swiglu", ws, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    s.synchronize()
    want = [t.clone() for t in (out, pre, gx, gw, gb)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(torch.cuda.current_stream())
    for t in (out, pre, gx, gw, gb):
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, t) for a, t in zip(want, (out, pre, gx, gw, gb)))
    x.copy_(torch.randn(M, K, device=DEV).bfloat16())
    graph.replay()
    got = [t.clone() for t in (out, pre, gx, gw, gb)]
    both()
    assert all(torch.equal(a, t) for a, t in zip(got, (out, pre, gx, gw, gb)))


@pytest.mark.parametrize("M,K,N,act", [(300, 264, 200, "swiglu"), (2100, 1040, 64, "none"), (64, 1024, 700, "gelu")])
def test_calls_behind_each_other_share_a_workspace(m, M, K, N, act):
    """Gradients' launches begin before the ones in front of them end: many calls in a row on one workspace, each with
    other inputs, give what each gives alone."""
    x, w, _, rand, wide = make(M, K, N, act, 5)
    gs = [rand(M, N).bfloat16() for _ in range(6)]
    pre = None if act == "none" else rand(M, wide).bfloat16()
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(M, K, N, act), dtype=torch.uint8, device=DEV)
    outs = lambda: (torch.empty_like(x), torch.empty(wide, K, device=DEV), torch.empty(wide, device=DEV))
    want, got = [outs() for _ in gs], [outs() for _ in gs]
    for g, o in zip(gs, want):
        ws.fill_(255)
        m.ep_linear_backward(g, x, w, *o, pre, act, ws)
        torch.cuda.synchronize()
    for _ in range(3):
        for g, o in zip(gs, got):
            m.ep_linear_backward(g, x, w, *o, pre, act, ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, q in zip(want, got) for a, b in zip(o, q))


@pytest.mark.parametrize("M,K,N,act", [(20000, 136, 200, "none"), (19457, 200, 128, "swiglu"), (38913, 72, 64, "gelu"),
                                       (39000, 64, 255, "silu")])
def test_linear_turns_of_equal_rows(m, M, K, N, act):
    """More rows than the SMs take at once, of one tile of columns: tiles that end within a box of results."""
    check_forward(m, M, K, N, act, True, True, False, True)
    check_forward(m, M, K, N, act, False, True, True, False, extra=8, seed=1)
    check_forward(m, M, K, N, act, True, False, False, False, extra=1, seed=2)
    check_backward(m, M, K, N, act, False, True, seed=3)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
def test_backward_far_from_zero(m, act):
    """Where an activation is its input or nothing, its gradient is the incoming one or nothing, however large the
    pre-activations are: no product in between overflows into NaN."""
    z = [s * v for v in (30.0, 32.0, 100.0, 1e4, 1e10, 2e19, 1e30, 3e38) for s in (1, -1)]
    N, K = len(z), 64
    z = torch.tensor(z, device=DEV).bfloat16()
    gate = z if act != "swiglu" else torch.cat([z, torch.full_like(z, 3.0)])
    pre = gate[None].contiguous()
    wide = pre.shape[1]
    g = torch.full((1, N), 1e20, device=DEV)
    x, w = torch.ones(1, K, device=DEV).bfloat16(), torch.ones(wide, K, device=DEV).bfloat16()
    gb = torch.empty(wide, device=DEV)
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(1, K, N, act), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(g, x, w, grad_bias=gb, pre=pre, activation=act, workspace=ws)
    zd, gd = z.double(), g[0].double()
    slope = (zd > 0).double()
    want = slope * gd * (3.0 if act == "swiglu" else 1.0)
    assert bool(((gb[:N].double() - want).abs() <= 1e-5 * 3.0 * gd).all())     # (from 30 on the slopes' rests are below 31 e^-30 = 3e-12)
    if act == "swiglu":
        up = gd * slope * zd
        fits = up < 3e38
        assert bool(((gb[N:].double() - up).abs() <= 1e-5 * up + 1e-5 * gd)[fits].all())
        assert not bool(torch.isnan(gb).any())


def test_swiglu_backward_product_order(m):
    """Beside a slope of zero, a gradient and an up row whose product is beyond fp32 leave zero."""
    g = torch.full((1, 8), 1e20, device=DEV)
    pre = torch.cat([torch.full((1, 8), -300.0, device=DEV), torch.full((1, 8), 1e30, device=DEV)], 1).bfloat16()
    x, w = torch.ones(1, 64, device=DEV).bfloat16(), torch.ones(16, 64, device=DEV).bfloat16()
    gb = torch.empty(16, device=DEV)
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(1, 64, 8, "swiglu"), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(g, x, w, grad_bias=gb, pre=pre, activation="swiglu", workspace=ws)
    assert bool((gb == 0).all())


@pytest.mark.parametrize("N", [8200, 8201])
def test_offsets_past_32_bits(m, N):
    """More than 2^31 outputs, pre-activations and gradients: the last rows are those of a call on them alone, which the
    tests above hold to the formula."""
    M, K, n = 262200, 64, 300
    x, w, b, rand, _ = make(M, K, N, "relu", 3)
    out, pre = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    m.ep_linear(x, w, out, bias=b, pre=pre, activation="relu")
    tail = x[-n:].contiguous()
    for rows in (slice(M - n, M), slice(0, n)):
        z = x[rows].double() @ w.double().t() + b.double()
        ez = 2 * (K + 16) * U * (x[rows].double().abs() @ w.double().abs().t()) + 2 * U * z.abs()
        assert within(pre[rows], z, ez)
        assert within(out[rows], z.clamp_min(0), ez)
    go, gx = out, torch.empty_like(x)               # (a gradient as large as the outputs)
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(M, K, N, "relu"), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(go, x, w, grad_x=gx, pre=pre, activation="relu", workspace=ws)
    gt = torch.empty_like(tail)
    ws2 = torch.empty(m.ep_linear_backward_workspace_bytes(n, K, N, "relu"), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(go[-n:].contiguous(), tail, w, grad_x=gt, pre=pre[-n:].contiguous(), activation="relu", workspace=ws2)
    g = torch.where(pre[-n:].double() > 0, go[-n:].double(), 0.0)
    tol = 2 * (N + 16) * U * (g.abs() @ w.double().abs())
    assert within(gx[-n:], g @ w.double(), tol) and within(gt, g @ w.double(), tol)

"""The layer for a few tokens against its definition in 64 bits, and its routing against ep_route's, bit by bit.

Tolerances follow from the arithmetic: u = 2^-24 is fp32's unit roundoff; a sum of n products is within 2 (n + 16) u of
the sum of their magnitudes.  An element of h whose cast that uncertainty leaves open counts with both codes; the others
have one.  A bf16 output has to be the rounding of a value within the tolerance.
"""
import math

import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    return load_ep()


def e4m3(v):
    """v >= 0 in 64 bits, rounded to e4m3 (nearest even, saturating)."""
    return v.clamp_max(448.0).to(torch.float8_e4m3fn).double()


class Layer:
    def __init__(self, m, T, E, k, H, I, seed=0, dtype=torch.float32, bias=False, residual=True, pad=0, **router):
        from combine_ep_layout_05_gb300.moe import quantize_blocks
        g = torch.Generator(DEV).manual_seed(seed)
        self.rand = rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
        self.m, self.T, self.E, self.k, self.H, self.I = m, T, E, k, H, I
        self.p, self.r = m.problem(T, H, k, E, 1), m.router(**router)
        self.gu, self.gus = quantize_blocks(rand(E, 2 * I, H) * H ** -0.5)
        self.dn, self.dns = quantize_blocks(rand(E, H, I) * I ** -0.5)
        self.x, self.logits = rand(T, H).bfloat16(), rand(T, E).to(dtype)
        if pad:
            self.logits[T - pad:] = -math.inf
        self.bias = rand(E) * 0.05 if bias else None
        self.residual = rand(T, H).bfloat16() if residual else None
        self.out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV)
        self.idx = torch.full((T, k), -7, dtype=torch.int64, device=DEV)
        self.w = torch.full((T, k), -7.0, device=DEV)
        n = m.ep_moe_few_workspace_bytes(self.p, I)
        self.guarded = torch.full((n + 256,), 255, dtype=torch.uint8, device=DEV)     # (NaN, whatever is read of it)
        self.ws = self.guarded[:n]
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, stream=None):
        self.m.ep_moe_few(self.p, self.r, self.x, self.logits, self.bias, self.gu, self.gus, self.dn, self.dns, self.out,
                          self.idx, self.w, self.ws, self.residual, self.status, stream)
        return self.out

    def check(self):
        m, T, k, H, I = self.m, self.T, self.k, self.H, self.I
        idx, w = torch.empty_like(self.idx), torch.empty_like(self.w)
        m.ep_route(self.p, self.r, self.logits, self.bias, idx, w)
        assert torch.equal(self.idx, idx) and torch.equal(self.w, w)
        assert bool((self.guarded[self.ws.numel():] == 255).all())
        # the dispatch's cast, whose factors and products are fp32 by definition
        b = self.x.float().view(T, -1, 128)
        amax = b.abs().amax(2, keepdim=True)
        full = torch.full_like(amax, 448.0)
        inv = torch.where(amax > 0, (full / amax).clamp_max(torch.finfo(torch.float32).max), 0.0)
        a = ((b * inv).clamp(-448, 448).to(torch.float8_e4m3fn).double() * (amax / full).double()).view(T, H)
        want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        tol = torch.zeros_like(want)
        for e in sorted(set(idx.reshape(-1).tolist()) - {-1}):
            t, j = (idx == e).nonzero(as_tuple=True)
            wide = lambda q, s: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            gu, dn = wide(self.gu[e], self.gus[e]), wide(self.dn[e], self.dns[e])
            z, ez = a[t] @ gu.t(), 2 * (H + 16) * U * (a[t].abs() @ gu.abs().t())
            g, up = z[:, :I], z[:, I:]
            h = g * torch.sigmoid(g) * up
            eh = (1.1 * ez[:, :I] * (up.abs() + ez[:, I:]) + (g * torch.sigmoid(g)).abs() * ez[:, I:] +
                  h.abs() * U * (16 + 2 * g.abs()))
            mag, block = h.abs(), lambda v: v.view(len(t), -1, 128)
            top_lo, top_hi = (block(v).amax(2, keepdim=True) for v in ((mag - eh).clamp_min(0), mag + eh))
            lo = e4m3(block((mag - eh).clamp_min(0)) * (1 - 4 * U) * 448 / top_hi.clamp_min(1e-300)) * top_lo / 448
            hi = e4m3(block(mag + eh) * (1 + 4 * U) * 448 / top_lo.clamp_min(1e-300)) * top_hi / 448
            mid, rad = ((lo + hi) / 2).view_as(h) * h.sign(), ((hi - lo) / 2).view_as(h)
            ws = w[t, j].double()[:, None]
            want.index_add_(0, t, ws * (mid @ dn.t()))
            tol.index_add_(0, t, ws * (rad @ dn.abs().t() + 2 * (I + 16 + k) * U * ((mid.abs() + rad) @ dn.abs().t())))
        if self.residual is not None:
            want += self.residual.double()
            tol += U * want.abs()
        lo, hi = (want - tol).float().bfloat16(), (want + tol).float().bfloat16()
        assert bool(((lo <= self.out) & (self.out <= hi)).all())


SIZES = [
    # T, E, k, H, I
    (1, 8, 2, 128, 128), (1, 256, 8, 512, 256), (2, 3, 3, 256, 640), (5, 16, 3, 256, 128), (16, 40, 6, 384, 256),
    (17, 64, 8, 1152, 128), (32, 256, 8, 512, 256), (33, 64, 6, 384, 256), (48, 2, 1, 256, 384), (49, 12, 5, 128, 1024),
    (64, 4, 4, 256, 384), (64, 1, 1, 256, 256), (64, 256, 8, 512, 128), (64, 1024, 32, 128, 128), (3, 1000, 30, 256, 128),
]


@pytest.mark.parametrize("T,E,k,H,I", SIZES)
def test_layer(m, T, E, k, H, I):
    for seed, kw in enumerate((dict(), dict(dtype=torch.bfloat16, bias=True, scoring="sigmoid", scale=2.5, residual=False),
                               dict(renormalize=False, pad=min(T, 2)))):
        layer = Layer(m, T, E, k, H, I, seed, **kw)
        layer.run()
        assert m.ep_get_status(layer.status) == 0
        layer.check()
        first = layer.out.clone()
        layer.ws.fill_(255)
        layer.run()
        assert torch.equal(first, layer.out)


@pytest.mark.parametrize("scoring,softmax_key", [("softmax", "logit"), ("softmax", "score"), ("sigmoid", "logit")])
@pytest.mark.parametrize("E,groups,keep,best", [(64, 8, 4, 2), (64, 8, 3, 1), (60, 5, 2, 2), (48, 48, 20, 2), (36, 3, 1, 2),
                                                (256, 64, 7, 2), (1024, 32, 5, 2)])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_is_ep_routes(m, scoring, softmax_key, E, groups, keep, best, renorm):
    layer = Layer(m, 29, E, min(6, E // groups * keep), 128, 128, 5, bias=True, pad=2, scoring=scoring,
                  softmax_key=softmax_key, num_groups=groups, topk_groups=keep, group_best=best, renormalize=renorm)
    layer.logits[3, ::2] = -math.inf          # some experts are out
    layer.logits[4] = 0.5                     # ties everywhere
    layer.logits[5, 1:] = -math.inf           # one expert left
    layer.logits[6, 2] = math.inf
    layer.logits[7] *= 60
    layer.run()
    assert m.ep_get_status(layer.status) == 0
    layer.check()


def test_every_token_to_the_same_experts(m):
    layer = Layer(m, 64, 32, 4, 256, 256, 1)
    layer.logits[:, 5:9] += 100
    layer.run()
    layer.check()


def test_no_token_has_an_expert(m):
    layer = Layer(m, 9, 8, 2, 384, 128, 2, pad=9)
    assert torch.equal(layer.run(), layer.residual) and bool((layer.idx == -1).all()) and bool((layer.w == 0).all())
    layer.residual = None
    assert bool((layer.run() == 0).all())
    assert m.ep_get_status(layer.status) == 0


def test_rows_of_logits_apart(m):
    layer = Layer(m, 20, 24, 3, 256, 128, 3)
    layer.logits = torch.cat([layer.logits, torch.full((20, 5), math.nan, device=DEV)], 1)[:, :24]
    layer.run()
    assert m.ep_get_status(layer.status) == 0
    layer.check()


def test_out_is_the_residual(m):
    layer = Layer(m, 20, 24, 3, 256, 128, 4)
    want = layer.run().clone()
    layer.out = layer.residual
    assert torch.equal(layer.run(), want)


def test_nan_logits_are_flagged(m):
    layer = Layer(m, 20, 24, 3, 256, 128, 5)
    layer.logits[7, 3] = math.nan
    layer.run()
    assert m.ep_get_status(layer.status) == m.EP_STATUS_BAD_LOGIT
    layer.check()


def test_nan_and_zero_tokens(m):
    """A token with a NaN spoils its own row only; one of zeros comes out as its residual."""
    layer = Layer(m, 24, 6, 2, 256, 256, 6)
    clean = layer.run().clone()
    layer.x[3, 17] = math.nan
    layer.x[9] = 0
    out = layer.run()
    keep = [t for t in range(24) if t not in (3, 9)]
    assert torch.equal(out[keep], clean[keep]) and bool(torch.isnan(out[3]).all())
    assert torch.equal(out[9], layer.residual[9])


def test_no_tokens(m):
    layer = Layer(m, 1, 6, 2, 256, 256, 7)
    layer.p = m.problem(0, 256, 2, 6, 1)
    layer.x, layer.logits, layer.out, layer.residual = layer.x[:0], layer.logits[:0], layer.out[:0], layer.residual[:0]
    layer.run()


def test_in_graphs_that_share_a_workspace(m):
    layer = Layer(m, 32, 64, 6, 512, 256, 8, scoring="sigmoid")
    layer.run()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.run(torch.cuda.current_stream())
        graphs.append(g)
    for seed in range(4):
        gen = torch.Generator(DEV).manual_seed(seed)
        layer.x.copy_(torch.randn(32, 512, generator=gen, device=DEV).bfloat16())
        layer.logits.copy_(torch.randn(32, 64, generator=gen, device=DEV))
        layer.out.fill_(7)
        graphs[seed & 1].replay()
        layer.check()
    assert m.ep_get_status(layer.status) == 0


def test_on_two_streams_at_once(m):
    layers = [Layer(m, 40, 32, 4, 512, 384, s) for s in (9, 10)]
    want = [x.run().clone() for x in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for x, s in zip(layers, streams):
            x.run(s)
    torch.cuda.synchronize()
    assert all(torch.equal(x.out, w) for x, w in zip(layers, want))


def test_calls_behind_each_other_share_a_workspace(m):
    """The launches of a call begin before the ones in front of them end: many calls in a row on one workspace, each with
    other inputs, give what each gives alone."""
    layers = [Layer(m, 24, 48, 5, 384, 256, 11 + s) for s in range(5)]
    want = []
    for x in layers:
        x.ws = layers[0].ws
        want.append(x.run().clone())
        torch.cuda.synchronize()
    for _ in range(4):
        for x in layers:
            x.out.fill_(7)
        for x in layers:
            x.run()
        torch.cuda.synchronize()
        assert all(torch.equal(x.out, w) for x, w in zip(layers, want))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 2048, 128), (40, 3, 2, 1536, 128), (7, 2, 1, 4096, 256), (16, 5, 2, 128, 2048)])
def test_split_units(m, T, E, k, H, I):
    """Few experts and long contractions: a unit of work is shared by several SMs."""
    for seed in range(2):
        layer = Layer(m, T, E, k, H, I, seed)
        first = layer.run().clone()
        assert m.ep_get_status(layer.status) == 0
        layer.check()
        for _ in range(5):
            assert torch.equal(first, layer.run())

"""MoeLayer, the operators together: forward against the definition in 64
bits with the layer's own FP8 roundings, the router's gradient against
differences of the forward formula, and a recorded graph."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return load_ep()


def make(T, H, I, E, k, R, seed=0, **router):
    m = load_ep()
    from combine_ep_layout_05_gb300.moe import MoeLayer, quantize_blocks
    g = torch.Generator(DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    gu, down = rand(E, 2 * I, H) * H ** -0.5, rand(E, H, I) * I ** -0.5
    layer = MoeLayer(T, H, I, E, k, R, *quantize_blocks(gu), *quantize_blocks(down), router=m.router(**router))
    return layer, rand(T, H).bfloat16(), rand(T, E)


def widen(codes, scales, rows):
    """e4m3 codes [.., N, K] times their scales, rows x 128 a scale, in 64 bits."""
    s = scales.double().repeat_interleave(128, -1)
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., :codes.shape[-2], :]
    return codes.view(torch.float8_e4m3fn).double() * s


@pytest.mark.parametrize("T,H,I,E,k,R", [(8, 256, 128, 8, 2, 4), (60, 384, 256, 10, 3, 5), (512, 256, 128, 4, 2, 2)])
def test_forward(m, T, H, I, E, k, R):
    layer, x, logits = make(T, H, I, E, k, R, scoring="sigmoid", scale=2.0)
    out = layer.forward(x, logits)
    assert m.ep_get_status(layer.status) == 0
    # the dispatch's cast of each token, taken from its first row; the experts' cast is checked by its own tests
    idx, w, slot = layer.idx.cpu(), layer.weights.double(), layer.pipe.buf.expert_slot.cpu()
    tok = torch.arange(T)[:, None].expand(T, k).reshape(-1)
    row = ((idx * R + (torch.arange(T) // (T // R))[:, None]) * (T // R) + slot).reshape(-1).to(DEV)
    e = idx.reshape(-1).to(DEV)
    a = widen(layer.pipe.recv[row], layer.pipe.recv_scales[row], 1)
    xs = x.double()[tok.to(DEV)]
    assert bool(((a - xs).abs() <= 2.0 ** -4 * xs.abs() + 2.0 ** -9 * layer.pipe.recv_scales[row].double()
                 .repeat_interleave(128, 1)).all())
    gu, down = widen(layer.gate_up, layer.gate_up_scales, 128), widen(layer.down, layer.down_scales, 128)
    c = torch.einsum("nk,nik->ni", a, gu[e])
    h = c[:, :I] * torch.sigmoid(c[:, :I]) * c[:, I:]
    act = widen(layer.act[row], layer.act_scales[row], 1)
    step = layer.act_scales[row].double().repeat_interleave(128, 1)
    assert bool(((act - h).abs() <= 2.0 ** -4 * h.abs() + 2.0 ** -9 * step + 1e-4 * h.abs().amax()).all())
    y = torch.einsum("ni,nhi->nh", act, down[e])
    mag = torch.einsum("ni,nhi->nh", act.abs(), down[e].abs())
    want = (y.view(T, k, H) * w[:, :, None]).sum(1)
    # y rounded to bf16 (2^-8 each), fp32 sums (2^-15 of the magnitudes covers both products' lengths), out rounded
    tol = ((2.0 ** -8 * y.abs() + 2.0 ** -15 * mag).view(T, k, H) * w[:, :, None]).sum(1) * 1.01 + 2.0 ** -8 * want.abs()
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_router_grad_matches_differences(m, scoring, renorm):
    T, H, I, E, k, R = 12, 256, 128, 8, 3, 2
    layer, x, logits = make(T, H, I, E, k, R, seed=3, scoring=scoring, renormalize=renorm, scale=1.5)
    layer.forward(x, logits)
    go = torch.randn(T, H, generator=torch.Generator(DEV).manual_seed(9), device=DEV).bfloat16()
    grad = torch.empty(T, E, device=DEV)
    layer.router_grad(go, logits, grad)
    assert m.ep_get_status(layer.status) == 0
    # the loss <go, out> as a function of the logits in 64 bits: experts' rows and their choice fixed
    idx = layer.idx
    src = torch.arange(T, device=DEV)[:, None] // (T // R)
    row = (idx * R + src) * (T // R) + layer.pipe.buf.expert_slot
    dots = (layer.pipe.y[row].double() * go.double()[:, None, :]).sum(2)

    def loss(z):
        s = torch.softmax(z, 1) if scoring == "softmax" else torch.sigmoid(z)
        sel = s.gather(1, idx)
        if renorm:
            sel = sel / sel.sum(1, keepdim=True)
        return (1.5 * sel * dots).sum()
    z = logits.double().requires_grad_()
    loss(z).backward()
    big = 1.5 * dots.abs().sum(1, keepdim=True)
    assert bool(((grad.double() - z.grad).abs() <= 1e-5 * big).all())
    for t, e in ((0, 0), (5, int(idx[5, 1])), (11, 7)):
        d = torch.zeros_like(logits, dtype=torch.float64)
        d[t, e] = 1e-5
        fd = (loss(logits.double() + d) - loss(logits.double() - d)) / 2e-5
        assert abs(float(fd - grad[t, e].double())) <= 2e-5 * float(big[t, 0])


def test_forward_in_a_graph_follows_new_inputs(m):
    T, H, I, E, k, R = 32, 256, 128, 16, 4, 4
    layer, x, logits = make(T, H, I, E, k, R, num_groups=4, topk_groups=2)
    for _ in range(2):
        layer.forward(x, logits)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(x, logits, torch.cuda.current_stream())
    x.copy_(torch.randn(T, H, device=DEV).bfloat16())
    logits.copy_(torch.randn(T, E, device=DEV))
    g.replay()
    got, idx = layer.pipe.out.clone(), layer.idx.clone()
    want = layer.forward(x, logits)
    assert torch.equal(got, want) and torch.equal(idx, layer.idx)
    assert m.ep_get_status(layer.status) == 0


def test_padding_tokens_come_out_zero(m):
    T, H, I, E, k, R = 16, 256, 128, 8, 2, 2
    layer, x, logits = make(T, H, I, E, k, R, scoring="sigmoid")
    logits[5] = -math.inf
    logits[12] = -math.inf
    out = layer.forward(x, logits)
    assert m.ep_get_status(layer.status) == 0
    assert bool((out[[5, 12]] == 0).all()) and bool((layer.idx[[5, 12]] == -1).all())
    assert bool((out[0] != 0).any())


def test_layer_refuses_other_shapes(m):
    from combine_ep_layout_05_gb300.moe import MoeLayer, quantize_blocks
    z = torch.zeros(1, device=DEV)
    with pytest.raises(ValueError):
        MoeLayer(8, 256, 128, 4, 2, 2, torch.zeros(4, 128, 256, dtype=torch.uint8, device=DEV), z,
                 torch.zeros(4, 256, 128, dtype=torch.uint8, device=DEV), z)
    with pytest.raises(ValueError):
        quantize_blocks(torch.zeros(2, 128, 100, device=DEV))
    q, s = quantize_blocks(torch.zeros(2, 130, 256, device=DEV))
    assert q.shape == (2, 130, 256) and s.shape == (2, 2, 2) and bool((q & 0x7F == 0).all()) and bool((s == 0).all())

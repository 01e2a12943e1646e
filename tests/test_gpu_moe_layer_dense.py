"""MoeLayer with a gate, a shared expert and its form for few tokens: the operators together against the same calls one
by one, the definition in 64 bits, and differences."""
import math

import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return load_ep()


def make(T, H, I, E, k, R, S, few=False, seed=0, **router):
    m = load_ep()
    from combine_ep_layout_05_gb300.moe import MoeLayer, quantize_blocks
    g = torch.Generator(DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    experts = (*quantize_blocks(rand(E, 2 * I, H) * H ** -0.5), *quantize_blocks(rand(E, H, I) * I ** -0.5))
    kw = dict(router=m.router(**router), gate=(rand(E, H) * H ** -0.5).bfloat16())
    if S:
        kw |= dict(shared_gate_up=(rand(2 * S, H) * H ** -0.5).bfloat16(), shared_down=(rand(H, S) * S ** -0.5).bfloat16())
    return MoeLayer(T, H, I, E, k, R, *experts, few=few, **kw), rand(T, H).bfloat16()


def shared64(layer, x):
    z = x.double() @ layer.shared_gate_up.double().t()
    S = layer.shared_down.shape[1]
    return z[:, :S] * torch.sigmoid(z[:, :S]) * z[:, S:] @ layer.shared_down.double().t()


@pytest.mark.parametrize("T,H,I,E,k,R,S", [(8, 256, 128, 8, 2, 4, 128), (60, 384, 256, 10, 3, 5, 200), (512, 256, 128, 4, 2, 2, 72)])
def test_forward_is_its_parts(m, T, H, I, E, k, R, S):
    layer, x = make(T, H, I, E, k, R, S)
    plain, _ = make(T, H, I, E, k, R, 0)
    got = layer.forward(x)
    assert m.ep_get_status(layer.status) == 0
    logits = x.double() @ layer.gate.double().t()
    assert bool(((layer.logits.double() - logits).abs() <= 2 * (H + 16) * 2.0 ** -24 *
                 (x.double().abs() @ layer.gate.double().abs().t())).all())
    routed = plain.forward(x, layer.logits)          # a layer as it was: logits in, no shared expert
    assert torch.equal(plain.idx, layer.idx) and torch.equal(plain.weights, layer.weights)
    want = routed.double() + shared64(layer, x)
    # the shared expert's activations and its sum with the rest are rounded to bf16
    size = (x.double().abs() @ layer.shared_gate_up.double().abs().t()).amax()
    tol = 2.0 ** -8 * (layer.shared_act.double().abs() @ layer.shared_down.double().abs().t()) + 2.0 ** -8 * want.abs() + \
        1e-5 * size
    assert bool(((got.double() - want).abs() <= tol * 1.05).all())


@pytest.mark.parametrize("T,H,I,E,k,S", [(1, 256, 128, 8, 2, 128), (13, 384, 256, 10, 3, 200), (64, 256, 384, 32, 4, 0)])
def test_few_tokens_match_the_long_way(m, T, H, I, E, k, S):
    few, x = make(T, H, I, E, k, 1, S, few=True, scoring="sigmoid")
    long, _ = make(T, H, I, E, k, 1, S, scoring="sigmoid")
    a, b = few.forward(x), long.forward(x)
    assert m.ep_get_status(few.status) == 0
    assert torch.equal(few.idx, long.idx) and torch.equal(few.weights, long.weights)
    # The long way rounds each expert's rows to bf16, and its sum with the shared expert's twice.  Either way's fp32 sums
    # may leave a code of h on the other side of its border: 2^-4 of a value, of perhaps one in a thousand.
    w = long.weights.double().sum(1, keepdim=True)
    assert float((a.double() - b.double()).norm()) <= 2.0 ** -7 * float(b.double().norm())
    assert bool(((a.double() - b.double()).abs() <= 2.0 ** -6 * (b.double().abs() + w * b.double().abs().amax())).all())


@pytest.mark.parametrize("few", [False, True])
def test_layer_in_a_graph(m, few):
    layer, x = make(24, 256, 128, 16, 4, 1 if few else 4, 128, few=few)
    layer.forward(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.forward(x, stream=torch.cuda.current_stream())
    x.copy_(torch.randn(24, 256, device=DEV).bfloat16())
    g.replay()
    got, idx = out.clone(), layer.idx.clone()
    want = layer.forward(x)
    assert torch.equal(got, want) and torch.equal(idx, layer.idx)
    assert m.ep_get_status(layer.status) == 0


def test_gradients_of_gate_and_shared_expert(m):
    """Against autograd of the same formulas in 64 bits; the routed experts' rows and their choice are constants."""
    T, H, I, E, k, R, S = 40, 256, 128, 8, 3, 2, 96
    layer, x = make(T, H, I, E, k, R, S, seed=3)
    layer.forward(x)
    go = torch.randn(T, H, generator=torch.Generator(DEV).manual_seed(9), device=DEV).bfloat16()
    gl = torch.empty(T, E, device=DEV)
    gx, gg = torch.empty_like(x), torch.empty(E, H, device=DEV)
    sx, su, sd = torch.empty_like(x), torch.empty(2 * S, H, device=DEV), torch.empty(H, S, device=DEV)
    layer.router_grad(go, layer.logits, gl)
    layer.gate_grad(gl, x, gx, gg)
    layer.shared_grad(go, x, sx, su, sd)
    assert m.ep_get_status(layer.status) == 0
    xg, gate = x.double().requires_grad_(), layer.gate.double().requires_grad_()
    (xg @ gate.t()).backward(gl.double())
    up, down, xs = (t.double().requires_grad_() for t in (layer.shared_gate_up, layer.shared_down, x))
    z = xs @ up.t()
    (z[:, :S] * torch.sigmoid(z[:, :S]) * z[:, S:] @ down.t()).backward(go.double())
    # Each product has an operand rounded to bf16 (2^-8 of each term at most): the bound is of the sums of the terms'
    # sizes, which random signs leave some 10 times larger than the result.  The shared expert's gradient has three such
    # roundings behind each other (pre-activations, grad_act, G), and the activations' slope passes on the first.
    for got, want, steps in ((gx, xg.grad, 2), (gg, gate.grad, 1), (sx, xs.grad, 4), (su, up.grad, 4), (sd, down.grad, 2)):
        assert float((got.double() - want).norm()) <= steps * 2.0 ** -8 * float(want.norm())


def test_layer_refuses(m):
    from combine_ep_layout_05_gb300.moe import MoeLayer
    with pytest.raises(ValueError):
        make(65, 256, 128, 8, 2, 1, 0, few=True)
    layer, x = make(8, 256, 128, 8, 2, 1, 0, few=True)
    with pytest.raises(ValueError):
        layer.router_grad(x, layer.logits, layer.logits)
    layer.gate = None
    with pytest.raises(ValueError):
        layer.forward(x)
    z = torch.zeros(4, 256, 256, dtype=torch.uint8, device=DEV)
    s = torch.zeros(1, device=DEV)
    d = torch.zeros(4, 256, 128, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        MoeLayer(8, 256, 128, 4, 2, 2, z, s, d, s, gate=torch.zeros(5, 256, device=DEV))
    with pytest.raises(ValueError):
        MoeLayer(8, 256, 128, 4, 2, 2, z, s, d, s, shared_down=torch.zeros(256, 64, device=DEV))
    with pytest.raises(ValueError):
        MoeLayer(8, 256, 128, 4, 2, 2, z, s, d, s, shared_gate_up=torch.zeros(100, 256, device=DEV),
                 shared_down=torch.zeros(256, 64, device=DEV))


def test_gradients_refuse_what_the_layer_lacks(m):
    layer, x = make(8, 256, 128, 8, 2, 2, 0)
    with pytest.raises(ValueError):
        layer.shared_grad(x, x, torch.empty_like(x))
    layer.gate = None
    with pytest.raises(ValueError):
        layer.gate_grad(layer.logits, x, torch.empty_like(x))


def test_gradients_on_streams_and_in_a_graph(m):
    """The gate's and the shared expert's gradients at the same time, on streams of their own, while the current stream
    allocates and writes; then recorded, and replayed after other calls on the same layer."""
    T, H, S = 700, 512, 264
    layer, x = make(T, H, 128, 8, 2, 2, S, seed=4)
    layer.forward(x)
    gen = torch.Generator(DEV).manual_seed(11)
    go = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    gl = torch.randn(T, 8, generator=gen, device=DEV)
    outs = lambda: [torch.zeros_like(x), torch.zeros(8, H, device=DEV), torch.zeros_like(x),
                    torch.zeros(2 * S, H, device=DEV), torch.zeros(H, S, device=DEV)]

    def both(o, a, b):
        layer.gate_grad(gl, x, o[0], o[1], stream=a)
        layer.shared_grad(go, x, *o[2:], stream=b)
    got, want = outs(), outs()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    both(got, a, b)                                  # (the layer's first: its buffers are made here)
    for _ in range(8):
        torch.full((T, S), float("nan"), device=DEV, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    both(want, here, here)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(got, torch.cuda.current_stream(), torch.cuda.current_stream())
    other = outs()
    go2 = go.flip(0).contiguous()
    layer.shared_grad(go2, x, *other[2:])
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert m.ep_get_status(layer.status) == 0

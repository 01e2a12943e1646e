"""Buffers that MoeLayer's gradients make in their first call belong to the call's stream, however it is given."""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep
from test_gpu_moe_layer_dense import make

pytestmark = pytest.mark.gpu

KEPT = ("gate_workspace", "shared_grad_act", "shared_down_workspace", "shared_up_workspace")


def gradients(layer, x, go, gl, stream):
    T, H = x.shape
    S, E = layer.shared_down.shape[1], layer.gate.shape[0]
    o = [torch.zeros_like(x), torch.zeros(E, H, device=DEV), torch.zeros_like(x), torch.zeros(2 * S, H, device=DEV),
         torch.zeros(H, S, device=DEV)]
    if stream is not None:
        torch.cuda.synchronize()
    yield o
    layer.gate_grad(gl, x, o[0], o[1], stream=stream)
    layer.shared_grad(go, x, *o[2:], stream=stream)
    torch.cuda.synchronize()
    yield o


@pytest.mark.parametrize("kind", ["object", "handle", "default"])
def test_first_call_on_another_stream(kind):
    """Memory just freed on the current stream, where writes to it are still under way, is not what the gradients on
    another stream work in."""
    load_ep()
    T, H, S = 700, 512, 264
    make_one = lambda: make(T, H, 128, 8, 2, 2, S, seed=4)
    layer, x = make_one()
    gen = torch.Generator(DEV).manual_seed(11)
    go = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    gl = torch.randn(T, 8, generator=gen, device=DEV)
    layer.forward(x)
    first = gradients(layer, x, go, gl, None)
    next(first)
    want = [t.clone() for t in next(first)]
    sizes = [getattr(layer, n).numel() * getattr(layer, n).element_size() for n in KEPT]

    layer, x = make_one()
    layer.forward(x)
    other = torch.cuda.Stream()
    here = other if kind == "default" else torch.cuda.current_stream()      # the stream whose memory is freed
    stream = {"object": other, "handle": other.cuda_stream, "default": 0}[kind]
    second = gradients(layer, x, go, gl, stream)
    next(second)
    with torch.cuda.stream(here):
        freed = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in freed]
        torch.cuda.synchronize()
        for _ in range(300):
            for t in freed:
                t.fill_(255)                                               # (NaN, whatever is read of it)
        del t, freed
        got = next(second)
    for name in KEPT:
        lo = getattr(layer, name).data_ptr()
        hi = lo + getattr(layer, name).numel() * getattr(layer, name).element_size()
        assert all(hi <= a or b <= lo for a, b in spans), name
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_first_call_by_handle_in_a_graph():
    """Recorded by the capturing stream's handle, before the layer has any of these buffers; replayed beside eager calls."""
    load_ep()
    T, H, S = 200, 256, 136
    layer, x = make(T, H, 128, 8, 2, 2, S, seed=6)
    layer.forward(x)
    gen = torch.Generator(DEV).manual_seed(12)
    go = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    gl = torch.randn(T, 8, generator=gen, device=DEV)
    outs = lambda: [torch.zeros_like(x), torch.zeros(8, H, device=DEV), torch.zeros_like(x),
                    torch.zeros(2 * S, H, device=DEV), torch.zeros(H, S, device=DEV)]
    got, want = outs(), outs()

    def both(o, stream=None):
        layer.gate_grad(gl, x, o[0], o[1], stream=stream)
        layer.shared_grad(go, x, *o[2:], stream=stream)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both(got, torch.cuda.current_stream().cuda_stream)
    both(want)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))

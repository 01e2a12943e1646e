"""The smallest and the largest sizes of the dense products, and gradients of several calls at once."""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep
from test_gpu_linear import check_backward, check_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return load_ep()


@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 8, 1), (1, 1 << 24, 1), (2, 1 << 20, 9), (1, 8, (1 << 20) + 3), ((1 << 20) + 1, 8, 1),
                                   ((1 << 20) + 1, 16, 8), (200000, 64, 33)])
def test_forward(m, M, K, N, out32):
    check_forward(m, M, K, N, "none", False, False, out32, False)
    if K < 1 << 20:
        check_forward(m, M, K, N, "swiglu", True, True, out32, True, seed=1)


@pytest.mark.parametrize("M,K,N", [(1, 8, 1), (1, 1 << 20, 8), (2, 8, (1 << 20) + 3), ((1 << 20) + 1, 8, 1),
                                   ((1 << 20) + 1, 16, 8)])
def test_backward(m, M, K, N):
    check_backward(m, M, K, N, "none", False, False)
    check_backward(m, M, K, N, "gelu", True, True, seed=1)


def test_calls_at_once(m):
    """Forward and gradients on four streams, each with a workspace of its own, then all in one graph's branches."""
    M, K, N, act = 700, 520, 264, "swiglu"
    gen = torch.Generator(DEV).manual_seed(2)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    n = m.ep_linear_backward_workspace_bytes(M, K, N, act)
    calls = []
    for _ in range(4):
        x, w, g = rand(M, K).bfloat16(), (rand(2 * N, K) * K ** -0.5).bfloat16(), rand(M, N).bfloat16()
        outs = [torch.empty(M, N, device=DEV), torch.empty(M, 2 * N, device=DEV).bfloat16(), torch.empty_like(x),
                torch.empty_like(w), torch.empty(2 * N, device=DEV)]
        calls.append((x, w, g, torch.empty(n, dtype=torch.uint8, device=DEV), outs))

    def run(c, stream):
        x, w, g, ws, o = c
        m.ep_linear(x, w, o[0], pre=o[1], activation=act, stream=stream)
        m.ep_linear_backward(g, x, w, o[2], o[3], o[4], o[1], act, ws, stream=stream)
    want = []
    for c in calls:
        run(c, None)
        torch.cuda.synchronize()
        want.append([t.clone() for t in c[4]])

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w_, c in zip(want, calls) for a, b in zip(w_, c[4]))
        for c in calls:
            for t in c[4]:
                t.zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        torch.cuda.synchronize()
        for c, s in zip(calls, streams):
            run(c, s)
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        for c, s in zip(calls, streams):
            s.wait_stream(here)
            run(c, s)
        for s in streams:
            here.wait_stream(s)
    for _ in range(3):
        graph.replay()
        check()

"""NaN pre-activations: what the forward product lets through the gradients do not hide."""
import math

import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [8, 5, 300])
@pytest.mark.parametrize("grad32", [False, True])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
def test_gradients_keep_nan(act, grad32, N):
    """A NaN among the pre-activations makes NaN of its own column's sum, its row of grad_x and its row of grad_w."""
    m = load_ep()
    M, K, wide = 20, 64, 2 * N if act == "swiglu" else N
    gen = torch.Generator(DEV).manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    x, w, pre = rand(M, K).bfloat16(), rand(wide, K).bfloat16(), rand(M, wide).bfloat16()
    pre[7, 3] = math.nan
    g = rand(M, N).to(torch.float32 if grad32 else torch.bfloat16)
    gx, gw, gb = torch.empty_like(x), torch.empty(wide, K, device=DEV), torch.empty(wide, device=DEV)
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(M, K, N, act), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(g, x, w, gx, gw, gb, pre, act, ws)
    spoilt = {3, 3 + N} if act == "swiglu" else {3}          # (a NaN gate spoils the up row's gradient too)
    assert set(torch.isnan(gb).nonzero().flatten().tolist()) == spoilt
    assert set(torch.isnan(gw).all(1).nonzero().flatten().tolist()) == spoilt == set(
        torch.isnan(gw).any(1).nonzero().flatten().tolist())
    assert set(torch.isnan(gx).all(1).nonzero().flatten().tolist()) == {7} == set(
        torch.isnan(gx).any(1).nonzero().flatten().tolist())


def test_relu_beside_infinite_gradients():
    m = load_ep()
    pre = torch.tensor([[-1.0, 0.0, 2.0, -math.inf, math.inf, -0.0, 1.0, -3.0]], device=DEV).bfloat16()
    g = torch.full((1, 8), math.inf, device=DEV)
    gb = torch.empty(8, device=DEV)
    x, w = torch.ones(1, 64, device=DEV).bfloat16(), torch.ones(8, 64, device=DEV).bfloat16()
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(1, 64, 8, "relu"), dtype=torch.uint8, device=DEV)
    m.ep_linear_backward(g, x, w, grad_bias=gb, pre=pre, activation="relu", workspace=ws)
    i = math.inf
    assert gb.tolist() == [0, 0, i, 0, i, 0, i, 0]

"""Waits of the dense products and of the few-token layer that give up, and either products' kernel on the same shapes."""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep
from test_gpu_linear import U, act64, act_tol, make, within
from test_gpu_moe_few import Layer

pytestmark = pytest.mark.gpu

KERNELS = ["EP_LINEAR_FEW_ROWS", "EP_LINEAR_MANY_ROWS"]


@pytest.fixture(scope="module")
def m():
    return load_ep()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,K,N,act,out32", [(40, 2048, 200, "none", True), (40, 2048, 200, "none", False),
                                             (300, 1024, 520, "swiglu", False), (20, 72, 9, "gelu", True)])
def test_products_give_up(m, kernel, M, K, N, act, out32):
    """A limit of one cycle: the launch reports it and returns, and the next ordinary call is right."""
    x, w, b, rand, wide = make(M, K, N, act)
    dtype = torch.float32 if out32 else torch.bfloat16
    want, out = torch.empty(M, N, dtype=dtype, device=DEV), torch.empty(M, N, dtype=dtype, device=DEV)
    pre = torch.empty(M, wide, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.ep_selftest_linear(getattr(m, kernel), 1 << 32, x, w, want, bias=b, pre=pre, activation=act, dev_status=st)
    assert m.ep_get_status(st) == 0
    m.ep_selftest_linear(getattr(m, kernel), 1, x, w, out, bias=b, pre=pre, activation=act, dev_status=st)
    assert m.ep_get_status(st) == m.EP_STATUS_TIMEOUT
    st.zero_()
    m.ep_selftest_linear(getattr(m, kernel), 1 << 32, x, w, out, bias=b, pre=pre, activation=act, dev_status=st)
    assert m.ep_get_status(st) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,K,N,act", [(3000, 512, 64, "none"), (200, 264, 300, "swiglu")])
def test_gradients_give_up(m, kernel, M, K, N, act):
    x, w, _, rand, wide = make(M, K, N, act)
    g = rand(M, N)
    pre = None if act == "none" else rand(M, wide).bfloat16()
    outs = lambda: (torch.empty_like(x), torch.empty(wide, K, device=DEV), torch.empty(wide, device=DEV))
    ws = torch.empty(m.ep_linear_backward_workspace_bytes(M, K, N, act), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    want, out = outs(), outs()
    call = lambda clocks, o: m.ep_selftest_linear_backward(getattr(m, kernel), clocks, g, x, w, *o, pre, act, ws, st)
    call(1 << 32, want)
    assert m.ep_get_status(st) == 0
    call(1, out)
    assert m.ep_get_status(st) == m.EP_STATUS_TIMEOUT
    assert torch.equal(out[2], want[2])              # (the bias's gradient waits for nothing)
    st.zero_()
    ws.fill_(255)
    call(1 << 32, out)
    assert m.ep_get_status(st) == 0 and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("T,E,k,H,I", [(32, 64, 8, 512, 256), (1, 4, 2, 2048, 128), (7, 2, 1, 256, 2048)])
def test_layer_gives_up(m, T, E, k, H, I):
    """Whole and split units of work."""
    layer = Layer(m, T, E, k, H, I, 3)
    want = layer.run().clone()
    assert m.ep_get_status(layer.status) == 0
    m.ep_selftest_moe_few(1, layer.p, layer.r, layer.x, layer.logits, layer.bias, layer.gu, layer.gus, layer.dn, layer.dns,
                          layer.out, layer.idx, layer.w, layer.ws, layer.residual, layer.status)
    assert m.ep_get_status(layer.status) == m.EP_STATUS_TIMEOUT
    assert bool((layer.guarded[layer.ws.numel():] == 255).all())
    layer.status.zero_()
    assert torch.equal(layer.run(), want) and m.ep_get_status(layer.status) == 0
    layer.check()


@pytest.mark.parametrize("out32", [False, True])
@pytest.mark.parametrize("M,K,N,act", [(2432, 7168, 256, "none"), (2500, 7168, 256, "none"), (1024, 2048, 512, "swiglu"),
                                       (512, 2048, 7168, "none"), (130, 4096, 384, "silu"), (64, 1000, 1024, "gelu")])
def test_both_kernels_on_the_same_shapes(m, M, K, N, act, out32):
    """Either side of where the choice between them changes: each is within the definition's tolerance."""
    x, w, b, rand, wide = make(M, K, N, act, 7)
    res = rand(M, N).bfloat16()
    z = x.double() @ w.double().t() + b.double()
    ez = 2 * (K + 16) * U * (x.double().abs() @ w.double().abs().t()) + 2 * U * z.abs()
    y, tol = act64(z, act, N) + res.double(), act_tol(z, ez, act, N)
    tol = tol + U * (y.abs() + tol)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for kernel in KERNELS:
        out = torch.empty(M, N, dtype=torch.float32 if out32 else torch.bfloat16, device=DEV)
        pre = torch.empty(M, wide, dtype=torch.bfloat16, device=DEV)
        m.ep_selftest_linear(getattr(m, kernel), 1 << 32, x, w, out, bias=b, residual=res, pre=pre, activation=act,
                             dev_status=st)
        assert m.ep_get_status(st) == 0
        assert within(out, y, tol + U * y.abs()) and within(pre, z, ez)

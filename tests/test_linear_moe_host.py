"""Refusals and sizes of the dense products and of the layer for few tokens, on the host: bad arguments are rejected
before anything reaches the GPU (the addresses are fakes and never read)."""
import ctypes

import pytest
import torch

from combine_ep_layout_05_gb300 import build as epbuild

OK = 1 << 20


@pytest.fixture(scope="module")
def ep():
    epbuild.build()
    from combine_ep_layout_05_gb300 import ep as epmod
    return epmod


def linear(ep, rows=4, K=64, N=32, act=0, x=OK, xs=64, w=OK, bias=None, res=None, rs=0, dt=0, out=OK, os=32, pre=None, st=None):
    return ep.lib().ep_linear(rows, K, N, act, x, xs, w, bias, res, rs, dt, out, os, pre, st, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only argument checks; fake pointers stay off GPUs")
@pytest.mark.parametrize("kw,why", [
    (dict(act=5), "activation"), (dict(act=-1), "activation"), (dict(rows=-1), "rows"), (dict(rows=(1 << 30) + 1), "rows"),
    (dict(K=60), "in_features"), (dict(K=0), "in_features"), (dict(K=1 << 25, xs=1 << 25), "in_features"),
    (dict(N=0), "out_features"), (dict(N=1 << 25, os=1 << 25), "out_features"), (dict(xs=56), "x_stride"),
    (dict(xs=68), "x_stride"), (dict(os=31), "out_stride"), (dict(res=OK, rs=31), "residual_stride"), (dict(dt=1), "out must"),
    (dict(x=None), "x / w"), (dict(x=OK + 8), "x / w"), (dict(w=OK + 2), "x / w"), (dict(w=None), "x / w"),
    (dict(out=None), "out NULL"), (dict(out=OK + 2, dt=2), "out NULL"), (dict(out=OK + 1), "out NULL"),
    (dict(bias=OK + 2), "bias"), (dict(res=OK + 1, rs=32), "residual"), (dict(pre=OK + 1), "pre"), (dict(st=OK + 2), "dev_status"),
    (dict(rows=1 << 30, K=64, N=1 << 20, os=1 << 20), "too large"),
])
def test_linear_refuses(ep, kw, why):
    assert linear(ep, **kw) == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()


def test_linear_without_rows_is_done(ep):
    assert linear(ep, rows=0, x=None, w=None, out=None) == ep.EP_OK


def backward(ep, rows=4, K=64, N=32, act=0, gdt=0, g=OK, gs=32, x=OK, xs=64, w=OK, pre=None, gx=OK, gxs=64, wdt=0, gw=OK,
             gb=OK, ws=OK, n=1 << 30, st=None):
    return ep.lib().ep_linear_backward(rows, K, N, act, gdt, g, gs, x, xs, w, pre, gx, gxs, wdt, gw, gb, ws, n, st, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only argument checks; fake pointers stay off GPUs")
@pytest.mark.parametrize("kw,why", [
    (dict(act=9), "activation"), (dict(K=4), "in_features"), (dict(gdt=1), "grad_out must"), (dict(wdt=1), "grad_w must"),
    (dict(gs=31), "grad_stride"), (dict(gxs=63), "grad_x_stride"), (dict(xs=60), "x_stride"), (dict(g=None), "grad_out"),
    (dict(g=OK + 2, gdt=2), "grad_out"), (dict(act=1), "pre"), (dict(act=4, pre=OK + 1), "pre"), (dict(x=None), "x NULL"),
    (dict(x=OK + 8), "x NULL"), (dict(w=None), "w NULL"), (dict(gw=OK + 8), "grad_w"), (dict(gb=OK + 2), "grad_bias"),
    (dict(gx=OK + 1), "grad_x"), (dict(ws=None), "workspace"), (dict(ws=OK + 8), "workspace"), (dict(n=64), "workspace"),
    (dict(st=OK + 1), "dev_status"),
])
def test_backward_refuses(ep, kw, why):
    assert backward(ep, **kw) == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()


def test_backward_without_outputs_is_done(ep):
    assert backward(ep, gx=None, gw=None, gb=None, g=None, ws=None, n=0) == ep.EP_OK


def test_backward_workspace(ep):
    need = ep.ep_linear_backward_workspace_bytes
    # G rounded up to 8 columns, and 16 blocks' sums of 5 columns
    assert need(128, 64, 5) == 128 * 8 * 2 + 16 * 5 * 4
    assert need(0, 64, 5) == 0 + 5 * 4 + 12
    assert need(128, 60, 5) == 0 and need(-1, 64, 5) == 0
    # a long contraction is split: the parts of the matrix's gradient are in it
    assert need(32768, 7168, 256) >= 32768 * 256 * 2 + 2 * 256 * 7168 * 4
    assert need(1 << 30, 8, 8) >= (1 << 30) * 16


def test_binding_refuses_other_tensors(ep):
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)
    with pytest.raises(ValueError):
        ep.ep_linear(z(4, 64), z(32, 64), z(4, 32))                 # not on a GPU
    with pytest.raises(ValueError):
        ep.ep_linear(z(4, 64), z(32, 56), z(4, 32))
    with pytest.raises(ValueError):
        ep.ep_linear(z(4, 64), z(31, 64), z(4, 15), activation="swiglu")
    with pytest.raises(ValueError):
        ep.ep_linear(z(4, 64), z(32, 64), z(4, 32), activation="tanh")
    with pytest.raises(ValueError):
        ep.ep_linear(z(256), z(32, 64), z(4, 32))
    p, r = ep.problem(4, 128, 2, 8, 1), ep.router()
    with pytest.raises(ValueError):
        ep.ep_moe_few(p, r, z(4, 128), z(4, 8), None, z(8, 200, 128), None, None, None, None, None, None, None)


def few(ep, T=4, H=256, k=2, E=8, R=1, I=128, r=None, x=OK, dt=2, logits=OK, ls=8, bias=None, gu=OK, gus=OK, dn=OK, dns=OK,
        res=None, out=OK, idx=OK, w=OK, ws=OK, n=1 << 30, st=None):
    p, r = ep.problem(T, H, k, E, R), ep.router() if r is None else r
    return ep.lib().ep_moe_few(ctypes.byref(p), ctypes.byref(r), I, x, dt, logits, ls, bias, gu, gus, dn, dns, res, out, idx,
                               w, ws, n, st, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only argument checks; fake pointers stay off GPUs")
@pytest.mark.parametrize("kw,why", [
    (dict(T=65), "at most 64"), (dict(H=192), "hidden"), (dict(I=192), "intermediate"), (dict(I=0), "intermediate"),
    (dict(I=1 << 24), "intermediate"), (dict(k=33), "out of range"), (dict(dt=1), "EP_FP32"), (dict(ls=7), "stride"),
    (dict(H=1 << 24, I=1 << 16), "2^39"), (dict(x=None), "x / gate_up"), (dict(x=OK + 8), "x / gate_up"),
    (dict(gu=OK + 8), "x / gate_up"), (dict(dn=None), "x / gate_up"), (dict(gus=None), "scales"), (dict(dns=OK + 2), "scales"),
    (dict(out=None), "out"), (dict(out=OK + 4), "out"), (dict(res=OK + 4), "out"), (dict(idx=OK + 4), "topk_idx"),
    (dict(w=None), "topk_idx"), (dict(logits=None), "logits"), (dict(bias=OK + 2), "bias"), (dict(ws=None), "workspace"),
    (dict(ws=OK + 128), "workspace"), (dict(n=1024), "workspace"), (dict(st=OK + 2), "dev_status"),
])
def test_few_refuses(ep, kw, why):
    assert few(ep, **kw) == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()


def test_few_sizes(ep):
    assert few(ep, T=0, x=None, logits=None, ws=None) == ep.EP_OK
    need = lambda T, I=128, k=2: ep.ep_moe_few_workspace_bytes(ep.problem(T, 256, k, 8, 1), I)
    assert need(65) == 0 and need(4, 100) == 0
    # the expert rows alone: codes, scales and the products
    assert need(64, 2048, 8) >= 64 * 8 * (2048 + 16 * 4 + 256 * 4)

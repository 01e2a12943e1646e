"""Argument checks of the dense products' and the few-token layer's self-tests, on the host."""
import ctypes

import pytest

from combine_ep_layout_05_gb300 import build as epbuild

OK = 1 << 20     # an aligned address that is never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def ep():
    epbuild.build()
    from combine_ep_layout_05_gb300 import ep as epmod
    return epmod


def linear(ep, kernel=0, clocks=1, st=OK, N=32):
    return ep.lib().ep_selftest_linear(kernel, clocks, 4, 64, N, 0, OK, 64, OK, None, None, 0, 0, OK, 32, None, st, None)


def backward(ep, kernel=0, clocks=1, st=OK, N=32):
    return ep.lib().ep_selftest_linear_backward(kernel, clocks, 4, 64, N, 0, 0, OK, 32, OK, 64, OK, None, OK, 64, 0, OK, OK, OK,
                                                1 << 30, st, None)


@pytest.mark.parametrize("call", [linear, backward])
@pytest.mark.parametrize("kw,why", [
    (dict(kernel=2), "kernel"), (dict(kernel=-1), "kernel"), (dict(clocks=0), "clocks"), (dict(clocks=(1 << 32) + 1), "clocks"),
    (dict(st=None), "dev_status"), (dict(st=OK + 2), "dev_status"), (dict(N=0), "out_features")])
def test_products_refuse(ep, call, kw, why):
    assert call(ep, **kw) == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()


@pytest.mark.parametrize("clocks,st,I,why", [(0, OK, 128, "clocks"), ((1 << 32) + 1, OK, 128, "clocks"),
                                             (1, None, 128, "dev_status"), (1, OK + 2, 128, "dev_status"),
                                             (1, OK, 100, "intermediate")])
def test_layer_refuses(ep, clocks, st, I, why):
    p, r = ep.problem(4, 256, 2, 8, 1), ep.router()
    rc = ep.lib().ep_selftest_moe_few(clocks, ctypes.byref(p), ctypes.byref(r), I, OK, 2, OK, 8, None, OK, OK, OK, OK, None, OK,
                                      OK, OK, OK, 1 << 30, st, None)
    assert rc == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()

"""Argument checks of the expert products' self-test, on the host."""
import ctypes

import pytest

from combine_ep_layout_05_gb300 import build as epbuild

OK16 = 1 << 20     # an aligned address that is never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def ep():
    epbuild.build()
    from combine_ep_layout_05_gb300 import ep as epmod
    return epmod


@pytest.mark.parametrize("at,bad,why", [
    (1, 2, "kernel"), (1, -1, "kernel"), (2, 12, "out_features"), (3, 200, "128"), (4, OK16 + 8, "a / w"),
    (8, None, "tokens_per_expert"), (9, OK16 + 8, "y"), (12, 0, "clocks"), (12, (1 << 32) + 1, "clocks"),
    (13, None, "dev_status")])
def test_refuses(ep, at, bad, why):
    a = [ctypes.byref(ep.problem(32, 256, 8, 256, 4)), 0, 512, 256, OK16, OK16, OK16, OK16, OK16, OK16, None, None, 1, OK16,
         None]
    a[at] = bad
    assert ep.lib().ep_selftest_expert_timeout(*a) == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()


def test_swiglu_form_needs_its_outputs(ep):
    a = [ctypes.byref(ep.problem(32, 256, 8, 256, 4)), 1, 512, 256, OK16, OK16, OK16, OK16, OK16, None, OK16, OK16, 1, OK16,
         None]
    for at, bad in ((10, None), (10, OK16 + 8), (11, None), (11, OK16 + 2), (2, 384)):
        b = list(a)
        b[at] = bad
        assert ep.lib().ep_selftest_expert_timeout(*b) == ep.EP_ERR_INVALID_ARG

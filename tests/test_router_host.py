"""The router's fields on the host: nothing here reaches a GPU."""
import ctypes

import pytest

from combine_ep_layout_05_gb300 import build as epbuild

OK16 = 1 << 20     # an aligned address that is never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def ep():
    epbuild.build()
    from combine_ep_layout_05_gb300 import ep as epmod
    return epmod


def test_softmax_key(ep):
    assert ep.router().softmax_key == ep.EP_KEY_LOGIT
    assert ep.router(softmax_key="score").softmax_key == ep.EP_KEY_SCORE
    with pytest.raises(KeyError):
        ep.router(softmax_key="probability")
    r = ep.router()
    for bad in (2, -1):
        r.softmax_key = bad
        rc = ep.lib().ep_route(ctypes.byref(ep.problem(32, 128, 8, 256, 4)), ctypes.byref(r), 2, OK16, 256, None, OK16,
                               OK16, None, None)
        assert rc == ep.EP_ERR_INVALID_ARG and "softmax_key" in ep.ep_last_error_string()

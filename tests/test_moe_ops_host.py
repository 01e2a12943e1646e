"""Argument checks of the routing, combine-backward and expert-product entry
points, on the host: nothing here reaches a GPU."""
import ctypes
import math

import pytest
import torch

from combine_ep_layout_05_gb300 import build as epbuild

OK16 = 1 << 20     # an aligned address that is never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def ep():
    epbuild.build()
    from combine_ep_layout_05_gb300 import ep as epmod
    return epmod


def route(ep, p, r, dtype=2, logits=OK16, stride=256, bias=None, idx=OK16, w=OK16, status=None):
    return ep.lib().ep_route(ctypes.byref(p), None if r is None else ctypes.byref(r), dtype, logits, stride, bias, idx,
                             w, status, None)


@pytest.mark.parametrize("change,why", [
    (dict(scoring=2), "scoring"), (dict(num_groups=0), "num_groups"), (dict(num_groups=7), "num_groups"),
    (dict(num_groups=4, topk_groups=5), "topk_groups"), (dict(topk_groups=0), "topk_groups"),
    (dict(group_best=3), "group_best"), (dict(group_best=0), "group_best"), (dict(scale=math.nan), "scale"),
    (dict(scale=math.inf), "scale")])
def test_router_rejected(ep, change, why):
    p = ep.problem(32, 128, 8, 256, 4)
    r = ep.router()
    for k, v in change.items():
        setattr(r, k, v)
    assert route(ep, p, r) == ep.EP_ERR_INVALID_ARG
    assert why in ep.ep_last_error_string()
    rc = ep.lib().ep_route_backward(ctypes.byref(p), ctypes.byref(r), 2, OK16, 256, OK16, OK16, OK16, 256, None, None)
    assert rc == ep.EP_ERR_INVALID_ARG and why in ep.ep_last_error_string()


def test_route_arguments_rejected(ep):
    p, r = ep.problem(32, 128, 8, 256, 4), ep.router()
    for kw in (dict(dtype=1), dict(dtype=7), dict(logits=None), dict(logits=OK16 + 2), dict(stride=255),
               dict(bias=OK16 + 2), dict(idx=None), dict(idx=OK16 + 4), dict(w=None), dict(w=OK16 + 2),
               dict(status=OK16 + 2), dict(dtype=0, logits=OK16 + 1)):
        assert route(ep, p, r, **kw) == ep.EP_ERR_INVALID_ARG, kw
    assert route(ep, p, None) == ep.EP_ERR_INVALID_ARG
    assert route(ep, ep.problem(30, 128, 8, 256, 4), r) == ep.EP_ERR_INVALID_ARG
    lib = ep.lib()
    args = [ctypes.byref(p), ctypes.byref(r), 2, OK16, 256, OK16, OK16, OK16, 256, None, None]
    for at, bad in ((3, None), (4, 100), (5, None), (6, None), (7, None), (7, OK16 + 2), (8, 100), (9, OK16 + 1)):
        a = list(args)
        a[at] = bad
        assert lib.ep_route_backward(*a) == ep.EP_ERR_INVALID_ARG, (at, bad)


def test_combine_backward_arguments_rejected(ep):
    p, lib = ep.problem(32, 128, 8, 256, 4), ep.lib()
    args = [ctypes.byref(p), 1, OK16, OK16, OK16, OK16, OK16, OK16, OK16, OK16, None, None]
    for at, bad in ((1, 5), (2, None), (2, OK16 + 8), (3, None), (3, OK16 + 8), (4, None), (5, None), (7, None),
                    (8, OK16 + 8), (9, OK16 + 2), (10, OK16 + 2)):
        a = list(args)
        a[at] = bad
        assert lib.ep_combine_backward(*a) == ep.EP_ERR_INVALID_ARG, (at, bad)
    rank = list(args)
    rank[1], rank[6] = 0, None
    assert lib.ep_combine_backward(*rank) == ep.EP_ERR_INVALID_ARG
    none = list(args)
    none[8] = none[9] = None      # nothing asked for
    assert lib.ep_combine_backward(*none) == ep.EP_OK


def test_expert_arguments_rejected(ep):
    p, lib = ep.problem(32, 256, 8, 256, 4), ep.lib()
    g = [ctypes.byref(p), 512, 256, OK16, OK16, OK16, OK16, OK16, OK16, None, None]
    for at, bad, why in ((1, 0, "out_features"), (1, 12, "out_features"), (1, 1 << 25, "out_features"), (2, 0, "128"),
                         (2, 200, "128"), (3, None, "a / w"), (3, OK16 + 8, "a / w"), (4, None, "scales"),
                         (5, OK16 + 4, "a / w"), (6, OK16 + 2, "scales"), (7, None, "tokens_per_expert"),
                         (8, None, "y"), (8, OK16 + 8, "y"), (9, OK16 + 2, "dev_status")):
        a = list(g)
        a[at] = bad
        assert lib.ep_expert_gemm(*a) == ep.EP_ERR_INVALID_ARG, (at, bad)
        assert why in ep.ep_last_error_string()
    s = [ctypes.byref(p), 128, OK16, OK16, OK16, OK16, OK16, OK16, OK16, None, None]
    for at, bad in ((1, 0), (1, 192), (2, None), (3, None), (4, None), (5, None), (6, None), (7, None), (7, OK16 + 8),
                    (8, None), (8, OK16 + 2)):
        a = list(s)
        a[at] = bad
        assert lib.ep_expert_swiglu(*a) == ep.EP_ERR_INVALID_ARG, (at, bad)
    odd = ep.problem(32, 264, 8, 256, 4)                       # hidden % 128
    s[0] = ctypes.byref(odd)
    assert lib.ep_expert_swiglu(*s) == ep.EP_ERR_INVALID_ARG
    huge = ep.problem(1 << 24, 256, 8, 256, 4)                 # E * T above int32
    g[0] = ctypes.byref(huge)
    assert lib.ep_expert_gemm(*g) == ep.EP_ERR_INVALID_ARG
    assert "int32" in ep.ep_last_error_string()
    wide = ep.problem(1 << 22, 256, 8, 256, 4)                 # 2^24 tiles of rows, 2^17 of columns
    g[0], g[1] = ctypes.byref(wide), 1 << 24
    assert lib.ep_expert_gemm(*g) == ep.EP_ERR_INVALID_ARG
    assert "too large" in ep.ep_last_error_string()


def test_python_binding_refuses(ep):
    p = ep.problem(8, 128, 2, 8, 2)
    with pytest.raises(KeyError):
        ep.router("relu")
    with pytest.raises(ValueError):
        ep.ep_route(p, ep.router(), torch.zeros(8, 8), None, torch.zeros(8, 2, dtype=torch.int64), torch.zeros(8, 2))
    with pytest.raises(TypeError):
        ep.ep_route(p, ep.router(), [0.0], None, None, None)
    with pytest.raises(ValueError):
        ep.ep_expert_gemm(p, None, None, torch.zeros(4, 8, 128), None, None, None)
    with pytest.raises(ValueError):
        ep.ep_expert_swiglu(p, None, None, torch.zeros(8, 256, 256), None, None, None, None)

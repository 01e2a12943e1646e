"""Routing where signs and rounding decide."""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return load_ep()


def choose(m, x, bias, k, router):
    T, E = x.shape
    idx = torch.full((T, k), -7, dtype=torch.int64, device=DEV)
    m.ep_route(m.problem(T, 128, k, E, 1), router, x, bias, idx, torch.empty(T, k, device=DEV))
    return idx.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_zeros_of_either_sign_tie(m, dtype, scoring):
    """-0 and +0 are equal keys, of experts and of groups: the lowest index first."""
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -0.0, 0.0, 0.0, 0.0], [0.0, -0.0] * 4], dtype=dtype, device=DEV)
    for bias in (None, torch.full((8,), -0.0, device=DEV), torch.tensor([-0.0, 0.0] * 4, device=DEV)):
        assert choose(m, x, bias, 5, m.router(scoring)) == [[0, 1, 2, 3, 4]] * 2
        # (32 lanes hold two groups as lanes of their own, or four of them one after the other)
        for groups, best in ((2, 1), (4, 1), (4, 2)):
            per = 8 // groups
            assert choose(m, x, bias, per, m.router(scoring, groups, 1, best)) == [list(range(per))] * 2

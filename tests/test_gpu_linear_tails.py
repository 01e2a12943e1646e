"""Shares of a tile's outputs whose lanes leave at different turns, in front of the cluster's last barrier."""
import pytest
import torch

from gpu_helpers import DEV, ep as load_ep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [64, 512, 2048])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 127), (3, 5), (7, 70), (13, 131), (33, 258), (61, 29)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_ragged_shares(K, M, N, act):
    m = load_ep()
    gen = torch.Generator(DEV).manual_seed(M * N)
    wide = 2 * N if act == "swiglu" else N
    x, w = (torch.randint(-4, 5, s, generator=gen, device=DEV).bfloat16() / 8 for s in ((M, K), (wide, K)))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, again = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV)
    for _ in range(20):                                      # (one after the other: clusters of two calls meet on an SM)
        m.ep_linear(x, w, out, activation=act, dev_status=st)
    m.ep_linear(x, w, again, activation=act, dev_status=st)
    assert m.ep_get_status(st) == 0 and torch.equal(out, again)
    z = x.double() @ w.double().t()                          # (multiples of 1 / 64 below 2^11: the sums are exact)
    if act == "none":
        assert torch.equal(out.double(), z)
    else:
        want = z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]
        # (expf 2 units, 1 + x, the reciprocal 1, two products; the sigmoid's argument is exact)
        assert bool(((out.double() - want).abs() <= 16 * 2.0 ** -24 * want.abs()).all())

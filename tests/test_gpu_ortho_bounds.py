"""Orthogonalised updates: coefficients whose largest value on the way is hard to
see, and matrices of zeros with the smallest eps."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.adapt_util import ortho64, ortho_norm_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


@pytest.mark.parametrize("c", [1e-15, -1e-16, 1e-16, 1e-300, 0.0])
def test_a_small_fifth_power(c):
    """p(s) = 30 s - 29 s^3 (+ c s^5) is 1 at s = 1 and 11.8 on the way.  Three equal
    singular values of 1 / sqrt 3 each come to 11.7 in one element."""
    G = torch.zeros((100, 90))
    for i in range(3):
        G[i, i] = 1.0
    steps = [(30.0, -29.0, c), (0.05, 0.0, 0.0)]
    got = rs.orthogonalize(G.cuda(), coefficients=steps).cpu().double()
    ref = ortho64(G, steps)
    assert float((got - ref).norm()) <= ortho_norm_bound(G, steps) + 2.0 ** -24 * float(ref.norm())


@pytest.mark.parametrize("eps", [1e-160, 1e-200, 1e-308, 5e-324, 1e-60])
@pytest.mark.parametrize("shape", [(16, 40), (40, 30), (64, 200), (1, 1), (70, 80)], ids=lambda s: "x".join(map(str, s)))
def test_zeros_with_the_smallest_eps(shape, eps):
    G = torch.zeros((2, *shape), device="cuda")
    G[1, 0, 0] = 2.0
    O = rs.orthogonalize(G, eps=eps)
    assert not O[0].any()
    ref = ortho64(G[1].cpu(), [rs.MUON] * 5, eps)
    bound = ortho_norm_bound(G[1].cpu(), [rs.MUON] * 5, eps) + 2.0 ** -24 * float(ref.norm())
    assert float((O[1].cpu().double() - ref).norm()) <= bound

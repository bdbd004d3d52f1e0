"""Orthogonalised updates: coefficients whose largest value on the way is hard to
see."""
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

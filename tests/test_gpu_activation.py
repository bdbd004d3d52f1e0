"""Activations of the gated feed-forward block and their derivatives far from
zero, evaluated by the kernels on given values."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.ff_util import ACTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


def derivative(act, g):
    """act'(g) (and act(g)) of the elementwise part of the backward pass: dG
    and dU for dH = U = 1, left in G and U."""
    G, U = g[None].cuda().contiguous(), torch.ones((1, g.numel()), device="cuda")
    one = torch.ones((1, 1), device="cuda")
    W = torch.ones((1, g.numel()), device="cuda")
    rs.glu_backward(torch.ones_like(U), one, W, W, G, U, act=act, need_dx=False, need_dw=False,
                    inplace=True)
    return G[0].cpu(), U[0].cpu()


@pytest.mark.parametrize("act", ACTS)
def test_derivatives_of_far_values(act):
    """From |g| = 30 on every derivative is within 30 exp(-30) < 2^-38 of its
    limit (0 or 1, sigmoid 0 on both sides), up to the largest float."""
    far = torch.tensor([30.0, 100.0, 1e6, 1.2e13, 2e13, 4e19, 5e19, 1e20, 3.4e38])
    for g, limit in ((-far, 0.0), (far, 0.0 if act == "sigmoid" else 1.0)):
        da, _ = derivative(act, g)
        assert ((da - limit).abs() <= 2.0 ** -23).all(), (act, g, da)

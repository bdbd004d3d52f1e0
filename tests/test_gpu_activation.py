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


def tails64(act, g):
    """act(g), act'(g) in 64 bits, and bounds on their float errors that shrink
    with the values, so that each tail is held to its own size.

    Roundings are counted in units u = 2^-24.  exp is good to 3 units in the
    last place and erfc to 16 (the OpenCL figures), 6 u and 32 u of the value.
    An argument that is off by d moves exp by the factor 1 + d and erfc(x) by
    1 + (2 x^2 + 1) d / |x| at most.  Where a value is below the smallest normal
    float, steps of 2^-149 count in place of u; the last term holds them with
    what multiplies them."""
    u, step = 2.0 ** -24, 2.0 ** -149
    a = g.abs()
    if act == "relu":
        return g.clamp_min(0), (g > 0).double(), 0 * a, 0 * a
    if act == "gelu":
        # 0.5 g erfc(x), x = -g / sqrt 2 off by 2 u: 2 x^2 = g^2.
        c = 0.5 * torch.erfc(-g / 2 ** 0.5)
        p = torch.exp(-0.5 * g * g) / (2 * torch.pi) ** 0.5
        ec = c * (2 * g * g + 40) * u
        # The exponent g^2 / 2 is rounded once.
        ep = a * p * (0.5 * g * g + 12) * u
        return g * c, c + g * p, a * ec + 32 * (a + 1) * step, ec + ep + 32 * (a + 1) * step
    # The logistic function of v, which tanh-gelu forms with 6 roundings.
    v, dv, ev = g, torch.ones_like(g), 0.0
    if act == "gelu_tanh":
        c2 = 2 * (2 / torch.pi) ** 0.5
        v, dv, ev = c2 * (g + 0.044715 * g ** 3), c2 * (1 + 0.134145 * g * g), 6.1
    s, r = torch.sigmoid(v), torch.sigmoid(-v)
    # exp(-|v|), 1 + it, the quotient and a product; either of s and r.
    e = (ev * v.abs() + 10) * u
    if act == "sigmoid":
        return s, s * r, s * e + 8 * step, s * r * (2 * e + u) + 8 * step
    # s + g s r v': s r with both errors and up to six more roundings.  A small
    # s is multiplied by 1 + |g| v': silu up to 1 + 104, tanh-gelu up to 1 + 300
    # where s is not 0 yet (g = -10.7: v' = 26).
    t = a * s * r * dv
    return (g * s, s + g * s * r * dv, a * s * (e + u) + 8 * (a + 1) * step,
            s * (e + u) + t * (2 * e + 6 * u) + 8 * (1 + (a * dv).clamp_max(300)) * step)


def assert_tails(act, name, g, got, want, err):
    off = (got.double() - want).abs()
    worst = int((off / err.clamp_min(1e-300)).argmax())
    assert (off <= err).all(), (act, name, float(g[worst]), float(got[worst]), float(want[worst]))


def tail_points():
    return torch.cat([torch.linspace(-120, 120, 9601), torch.linspace(-20, 20, 4001),
                      torch.tensor([-89.0, -88.73, 88.73, 16.7, 17.4, -13.9])])


@pytest.mark.parametrize("act", ACTS)
def test_tails_of_the_backward_pass(act):
    """Derivatives and values of the backward pass over both tails down to the
    smallest floats, at bounds relative to them."""
    g = tail_points()
    val, der, eval_, eder = tails64(act, g.double())
    da, a = derivative(act, g)
    assert_tails(act, "derivative", g, da, der, eder)
    assert_tails(act, "value", g, a, val, eval_)


@pytest.mark.parametrize("act", ACTS)
def test_tails_of_the_forward_pass(act):
    g = tail_points()
    val, _, err, _ = tails64(act, g.double())
    one = torch.ones((1, 1), device="cuda")
    H = rs.glu(one, g[None].cuda(), torch.ones((1, g.numel()), device="cuda"), act=act)
    assert_tails(act, "forward", g, H[0].cpu(), val, err)


@pytest.mark.parametrize("act", ACTS)
def test_non_finite_and_extreme_values(act):
    """NaN stays NaN, infinities go to their limits (where the formula has one
    in floats: not 0 times infinity), and finite values up to the largest stay
    finite."""
    nan, inf, big = float("nan"), float("inf"), 3.4028234e38
    g = torch.tensor([nan, inf, big, -big, 1e-45, -1e-45, 0.0, -0.0])
    one = torch.ones((1, 1), device="cuda")
    forward = rs.glu(one, g[None].cuda(), torch.ones((1, g.numel()), device="cuda"), act=act)[0].cpu()
    da, back = derivative(act, g)
    for a in (forward, back):
        assert torch.isnan(a[0])
        assert a[1] == (1.0 if act == "sigmoid" else inf)
        assert a[2] == (1.0 if act == "sigmoid" else big) and a[3] == 0.0
        at0 = 0.5 if act == "sigmoid" else 0.0
        assert ((a[4:] - at0).abs() <= 2.0 ** -149).all()
    assert torch.isfinite(da[2:]).all()
    assert da[3] == 0.0 and da[2] == (0.0 if act == "sigmoid" else 1.0)
    if act == "relu":  # compares with 0, which NaN does not exceed
        assert da[0] == 0.0 and da[4:].tolist() == [1.0, 0.0, 0.0, 0.0]
    else:
        assert torch.isnan(da[0]) and (da[4:] == (0.25 if act == "sigmoid" else 0.5)).all()

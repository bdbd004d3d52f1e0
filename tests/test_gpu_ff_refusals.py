"""Arguments of the feed-forward functions that are refused before any launch,
with an error that names what is wrong."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


def test_what_is_not_a_2d_tensor():
    X = torch.zeros((2, 64), device="cuda")
    w = torch.zeros((8, 32), dtype=torch.uint8, device="cuda")
    s = torch.ones((8, 2), device="cuda")
    for bad, kind in ((None, TypeError), ([[1]], TypeError), (w[0], ValueError), (w[0, 0], ValueError)):
        with pytest.raises(kind, match="weights"):
            rs.q4_matmul(X, bad, s, group=32)
        with pytest.raises(kind, match="weights"):
            rs.q4_glu(X, bad, s, w, s, group=32)
        with pytest.raises(kind, match="weights"):
            rs.q4_glu(X, w, s, bad, s, group=32)
    with pytest.raises(TypeError, match="scales"):
        rs.q4_matmul(X, w, None, group=32)
    for bad, kind in ((None, TypeError), (X[0], ValueError)):
        with pytest.raises(kind, match="weights"):
            rs.glu(X, bad, X)


def test_half_a_pair():
    X, W = torch.zeros((2, 8), device="cuda"), torch.zeros((8, 4), device="cuda")
    G = torch.zeros((2, 4), device="cuda")
    for save in ((None, G), (G, None), (None, None), (G,), (G, G, G)):
        with pytest.raises((TypeError, ValueError), match="save"):
            rs.glu(X, W, W, save=save)
    X = torch.zeros((2, 64), device="cuda")
    w, z = torch.zeros((2, 8, 32), dtype=torch.uint8, device="cuda")[0], torch.zeros((8, 2), dtype=torch.uint8, device="cuda")
    s = torch.ones((8, 2), device="cuda")
    for zeros in ((z, None), (None, z)):
        with pytest.raises(ValueError, match="zeros"):
            rs.q4_glu(X, w, s, w, s, *zeros, group=32)
    H = torch.zeros((2, 4), device="cuda")
    X8 = torch.zeros((2, 8), device="cuda")
    for dW in ((None, W), (W, None), (W,)):
        with pytest.raises((TypeError, ValueError), match="dW"):
            rs.glu_backward(H, X8, W, W.clone(), G, G.clone(), dW=dW)

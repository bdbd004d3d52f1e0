"""Ranks and rows that take the adapter kernels' less usual forms: ranks above
128 in tiles of 64 rows, long and odd ranks in tiles of 16 rows of the forward
pass, H saved."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.adapt_util import lora64, lora_backward64, make
from tests.ff_util import TYPES, Guarded, assert_within, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


SHAPES = [(300, 136, 200, 256, 2, "mixed"), (200, 72, 96, 131, 1, "one"), (100, 264, 512, 64, 40, "mixed"),
          (100, 72, 600, 200, 40, "mixed"), (90, 70, 300, 67, 30, "mixed"), (90, 520, 72, 256, 30, "mixed"),
          (100, 72, 96, 24, 40, "mixed"), (80, 65, 33, 35, 30, "mixed"), (200, 130, 72, 200, 2, "runs"),
          (70, 72, 40, 192, 1, "one"), (130, 600, 40, 250, 3, "mixed")]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forms(shape, t):
    M, N, K, R, L, kind = shape
    i = SHAPES.index(shape) + list(TYPES).index(t)
    gen = torch.Generator().manual_seed(i)
    X, A, B, ids, scale, base = make(gen, M, N, K, R, L, TYPES[t], kind)
    Y, H = Guarded(M, N, TYPES[t], gap=i % 3), Guarded(M, R, gap=i % 2)
    rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=base.cuda(), out=Y.view, save=H.view)
    (ref, h), (err, eh) = lora64(X, A, B, ids, scale, base)
    assert_within(H.view, h, eh, "H")
    assert_within(Y.view, ref, rounded(ref, err, TYPES[t]), "Y")
    assert Y.intact() and H.intact()
    dY = torch.randn((M, N), generator=gen).to(TYPES[t])
    Hs = torch.randn((M, R), generator=gen)
    gx = torch.randn((M, K), generator=gen).to(TYPES[t])
    got = rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), Hs.cuda(), ids.cuda(), scale=scale.cuda(),
                           base=gx.cuda())
    refs, errs = lora_backward64(dY, X, A, B, Hs, ids, scale, gx)
    for name, g, r, e in zip(("dX", "dA", "dB"), got, refs, errs):
        assert_within(g, r, rounded(r, e, TYPES[t]), name)

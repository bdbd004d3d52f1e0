"""Refusals of the gated feed-forward and 4-bit entry points: every bad call
is turned down on the host, before any HIP call."""
import os

import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.ff_util import ACTS, act64, glu64, glu_backward64

OK, DIM, LD, NULLPTR, VARIANT, ALIAS, LAUNCH, UNSUPPORTED, ARG, SCRATCH = range(10)
# Fake, well separated device addresses; validation never reads them.
P = [(i + 1) << 41 for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rs.library_path()):
        pytest.skip("libsgemm.so not built")
    return rs.load()


def glu(lib, act=0, transw=0, M=4, F=8, K=6, X=P[0], ldx=None, Wg=P[1], Wu=P[2], ldw=None, H=P[3],
        ldh=None, G=None, U=None, ldgu=8):
    return lib.sgemm_glu_f32(act, transw, M, F, K, X, max(K, 1) if ldx is None else ldx, Wg, Wu,
                             max(K if transw else F, 1) if ldw is None else ldw, H,
                             max(F, 1) if ldh is None else ldh, G, U, ldgu, None)


def test_glu_refusals(lib):
    assert glu(lib, act=-1) == ARG and glu(lib, act=5) == ARG
    assert glu(lib, transw=2) == ARG
    assert glu(lib, M=-1) == DIM and glu(lib, F=-1) == DIM and glu(lib, K=-1) == DIM
    assert glu(lib, M=(1 << 40) + 1) == DIM
    assert glu(lib, ldx=5) == LD and glu(lib, ldw=7) == LD and glu(lib, ldh=7) == LD
    assert glu(lib, transw=1, ldw=5) == LD
    assert glu(lib, G=P[4]) == ARG and glu(lib, U=P[4]) == ARG
    assert glu(lib, G=P[4], U=P[5], ldgu=7) == LD
    for name in ("X", "Wg", "Wu", "H"):
        assert glu(lib, **{name: None}) == NULLPTR, name
    # Empty outputs: nothing is read or written, null or not.
    assert glu(lib, M=0, X=None, Wg=None, Wu=None, H=None) == OK
    assert glu(lib, F=0, X=None, Wg=None, Wu=None, H=None) == OK


def test_glu_alias(lib):
    assert glu(lib, H=P[0] + 4) == ALIAS
    assert glu(lib, H=P[2] + 8) == ALIAS
    assert glu(lib, H=P[0] - 4 * (3 * 8 + 8) + 4) == ALIAS      # last element of H on X's first
    assert glu(lib, G=P[4], U=P[4], ldgu=8) == ALIAS
    assert glu(lib, G=P[3], U=P[5]) == ALIAS                     # G over H
    # G and U as column ranges of one buffer that share a column.
    assert glu(lib, G=P[4], U=P[4] + 4 * 7, ldgu=16) == ALIAS
    assert glu(lib, G=P[4], U=P[4] + 4 * 8, ldgu=15) == ALIAS    # U's row end on G's next row


def backward(lib, act=0, transw=0, M=4, F=8, K=6, X=P[0], ldx=None, Wg=P[1], Wu=P[2], ldw=None,
             G=P[3], U=P[4], ldgu=8, dH=P[5], lddh=8, dG=P[6], dU=P[7], lddgu=8, dX=P[8], lddx=6,
             dWg=P[9], dWu=P[10], lddw=None, beta=0.0):
    w = max(K if transw else F, 1)
    return lib.sgemm_glu_backward_f32(act, transw, M, F, K, X, max(K, 1) if ldx is None else ldx, Wg,
                                      Wu, w if ldw is None else ldw, G, U, ldgu, dH, lddh, dG, dU,
                                      lddgu, dX, lddx, dWg, dWu, w if lddw is None else lddw, beta,
                                      None)


def test_backward_refusals(lib):
    assert backward(lib, act=5) == ARG and backward(lib, transw=-1) == ARG
    assert backward(lib, M=-1) == DIM
    assert backward(lib, dWu=None) == ARG and backward(lib, dWg=None) == ARG
    for name in ("ldx", "ldw", "ldgu", "lddh", "lddgu", "lddx", "lddw"):
        assert backward(lib, **{name: 5}) == LD, name
    for name in ("X", "Wg", "Wu", "G", "U", "dH", "dG", "dU"):
        assert backward(lib, **{name: None}) == NULLPTR, name
    assert backward(lib, M=0, K=0, dX=None, dWg=None, dWu=None) == OK


def test_backward_alias(lib):
    assert backward(lib, dX=P[0]) == ALIAS
    assert backward(lib, dWg=P[1]) == ALIAS
    assert backward(lib, dWg=P[9], dWu=P[9]) == ALIAS
    assert backward(lib, dG=P[6], dU=P[6]) == ALIAS
    assert backward(lib, dG=P[3] + 4) == ALIAS          # shifted over G: not in place
    assert backward(lib, dG=P[3], lddgu=9) == ALIAS     # in place needs the same leading dimension
    assert backward(lib, dG=P[0]) == ALIAS              # only G, U and dH may be overwritten
    assert backward(lib, dX=P[3], lddx=8) == ALIAS


def q4(lib, act=None, xt=0, st=0, M=4, N=8, K=70, X=P[0], ldx=None, W=P[1], W2=P[2], ldw=None,
       group=32, S=P[3], S2=P[4], lds=3, Z=None, Z2=None, ldz=3, Y=P[7], ldy=8):
    ldx = max(K, 1) if ldx is None else ldx
    ldw = max((K + 1) // 2, 1) if ldw is None else ldw
    if act is None:
        return lib.sgemm_q4(xt, st, M, N, K, X, ldx, W, ldw, group, S, lds, Z, ldz, Y, ldy, None)
    return lib.sgemm_q4_glu(act, xt, st, M, N, K, X, ldx, W, W2, ldw, group, S, S2, lds, Z, Z2, ldz,
                            Y, ldy, None)


@pytest.mark.parametrize("act", [None, 0], ids=["plain", "gated"])
def test_q4_refusals(lib, act):
    assert q4(lib, act, xt=3) == ARG and q4(lib, act, st=-1) == ARG
    for group in (0, 16, 33, 96, -32):
        assert q4(lib, act, group=group) == ARG, group
    assert q4(lib, act, M=-1) == DIM and q4(lib, act, K=(1 << 40) + 1) == DIM
    assert q4(lib, act, ldx=69) == LD and q4(lib, act, ldw=34) == LD
    assert q4(lib, act, K=71, ldx=71, ldw=35) == LD       # an odd K's last byte counts
    assert q4(lib, act, lds=2) == LD and q4(lib, act, ldy=7) == LD
    assert q4(lib, act, Z=P[5], Z2=P[6], ldz=2) == LD
    for name in ("X", "W", "S", "Y"):
        assert q4(lib, act, **{name: None}) == NULLPTR, name
    assert q4(lib, act, Y=P[0] + 4) == ALIAS
    assert q4(lib, act, Y=P[1] + 40) == ALIAS
    assert q4(lib, act, Y=P[3]) == ALIAS
    assert q4(lib, act, Z=P[5], Z2=P[6], Y=P[5]) == ALIAS
    assert q4(lib, act, M=0, X=None, W=None, S=None, Y=None) == OK
    assert q4(lib, act, N=0, X=None, W=None, S=None, Y=None) == OK


def test_q4_glu_refusals(lib):
    assert q4(lib, 5) == ARG and q4(lib, -1) == ARG
    assert q4(lib, 0, Z=P[5]) == ARG and q4(lib, 0, Z2=P[5]) == ARG
    assert q4(lib, 0, W2=None) == NULLPTR and q4(lib, 0, S2=None) == NULLPTR
    assert q4(lib, 0, Y=P[2]) == ALIAS


def test_python_refusals():
    t = torch.zeros((4, 4))
    with pytest.raises(ValueError, match="unknown activation"):
        rs.glu(t, t, t, act="swish2")
    with pytest.raises(ValueError, match="GPU tensor"):
        rs.glu(t, t, t)
    with pytest.raises(TypeError, match="float32"):
        rs.glu(t.double(), t, t)
    with pytest.raises(ValueError, match="power of two"):
        rs.q4_matmul(t, t, t, group=48)
    with pytest.raises(TypeError):
        rs.q4_matmul(t.double(), t, t)


@pytest.mark.parametrize("act", ACTS)
def test_reference_gradients_match_differences(act):
    """The formulas the GPU gradients are held to, against central
    differences of the forward formula in 64 bits."""
    gen = torch.Generator().manual_seed(7)
    M, K, F = 3, 5, 4
    X, Wg, Wu, dH = (torch.randn(s, generator=gen, dtype=torch.float64)
                     for s in ((M, K), (K, F), (K, F), (M, F)))
    (_, G, Up), _ = glu64(act, X, Wg, Wu)
    (_, _, dX, dWg, dWu), _ = glu_backward64(act, X, Wg, Wu, G, Up, dH)
    args = [X, Wg, Wu]
    for i, grad in enumerate((dX, dWg, dWu)):
        for j in range(args[i].numel()):
            ends = []
            for h in (1e-6, -1e-6):
                moved = [a.clone() for a in args]
                moved[i].view(-1)[j] += h
                ends.append(float((glu64(act, *moved)[0][0] * dH).sum()))
            # Central difference: third derivatives of order 10 times h^2,
            # and 64-bit rounding of sums of order 10 over 2 h.
            assert abs((ends[0] - ends[1]) / 2e-6 - float(grad.view(-1)[j])) < 1e-7

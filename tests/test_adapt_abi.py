"""Refusals of the adapter and orthogonalising entry points: every bad call is
turned down on the host, before any HIP call.  And the formulas that the GPU's
gradients are held to, against differences."""
import ctypes
import os

import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.adapt_util import lora64, lora_backward64, make

OK, DIM, LD, NULLPTR, VARIANT, ALIAS, LAUNCH, UNSUPPORTED, ARG, SCRATCH = range(10)
# Fake, well separated device addresses; validation never reads them.
P = [(i + 1) << 41 for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(rs.library_path()):
        pytest.skip("libsgemm.so not built")
    return rs.load()


def lora(lib, t=0, M=4, N=8, K=6, R=2, L=3, X=P[0], ldx=6, A=P[1], lda=6, sa=12, B=P[2], ldb=2, sb=16,
         ids=P[3], bits=32, s=P[4], base=P[5], ldbase=8, Y=P[6], ldy=8, H=P[7], ldh=2, ws=P[8], n=1 << 40):
    return lib.sgemm_lora(t, M, N, K, R, L, X, ldx, A, lda, sa, B, ldb, sb, ids, bits, s, 1.0, base,
                          ldbase, Y, ldy, H, ldh, ws, n, None)


def test_lora_refusals(lib):
    assert lora(lib, t=3) == ARG and lora(lib, t=-1) == ARG and lora(lib, bits=16) == ARG
    for name in ("M", "N", "K"):
        assert lora(lib, **{name: -1}) == DIM and lora(lib, **{name: 1 << 31}) == DIM, name
    assert lora(lib, R=0) == DIM and lora(lib, R=257) == DIM
    assert lora(lib, L=0) == DIM and lora(lib, L=4097) == DIM
    for name, least in (("ldx", 6), ("lda", 6), ("ldb", 2), ("ldbase", 8), ("ldy", 8), ("ldh", 2)):
        assert lora(lib, **{name: least - 1}) == LD, name
    assert lora(lib, sa=-1) == LD and lora(lib, sb=-1) == LD
    for name in ("X", "A", "B", "Y"):
        assert lora(lib, **{name: None}) == NULLPTR, name
    big = dict(M=400, N=8, K=6, base=None, Y=1 << 50, H=None)  # few rows take none
    assert lora(lib, n=0, **big) == SCRATCH and lora(lib, n=4, **big) == SCRATCH
    assert lora(lib, ws=None) == ARG and lora(lib, ws=P[8] + 4) == ARG
    assert lora(lib, M=0, X=None, Y=None) == OK
    assert lora(lib, N=0, B=None, Y=None, H=None) == OK


def test_lora_alias(lib):
    assert lora(lib, Y=P[0]) == ALIAS
    assert lora(lib, Y=P[5] + 4) == ALIAS                # shifted over base: not in place
    assert lora(lib, Y=P[5], ldy=9) == ALIAS             # in place needs base's row stride
    assert lora(lib, Y=P[1] + 4 * (2 * 12 + 8)) == ALIAS  # in the last adapter
    assert lora(lib, Y=P[2]) == ALIAS and lora(lib, Y=P[3]) == ALIAS and lora(lib, Y=P[4]) == ALIAS
    assert lora(lib, H=P[6]) == ALIAS and lora(lib, H=P[5]) == ALIAS and lora(lib, H=P[0]) == ALIAS
    assert lora(lib, Y=P[8] + 64) == ALIAS


def backward(lib, t=0, M=4, N=8, K=6, R=2, L=3, dY=P[0], lddy=8, X=P[1], ldx=6, A=P[2], lda=6, sa=12, B=P[3],
             ldb=2, sb=16, H=P[4], ldh=2, ids=P[5], bits=64, s=P[6], base=P[7], ldbase=6, dX=P[8], lddx=6,
             dA=P[9], ldda=6, sda=12, dB=P[10], lddb=2, sdb=16, ws=P[11], n=1 << 40):
    return lib.sgemm_lora_backward(t, M, N, K, R, L, dY, lddy, X, ldx, A, lda, sa, B, ldb, sb, H, ldh, ids,
                                   bits, s, 1.0, base, ldbase, dX, lddx, dA, ldda, sda, dB, lddb, sdb, ws,
                                   n, None)


def test_backward_refusals(lib):
    assert backward(lib, t=3) == ARG and backward(lib, bits=8) == ARG
    assert backward(lib, R=257) == DIM and backward(lib, M=-1) == DIM
    for name, least in (("lddy", 8), ("ldx", 6), ("lda", 6), ("ldb", 2), ("ldh", 2), ("ldbase", 6),
                        ("lddx", 6), ("ldda", 6), ("lddb", 2)):
        assert backward(lib, **{name: least - 1}) == LD, name
    # Gradients of two adapters may not share elements.
    assert backward(lib, sda=11) == LD and backward(lib, sdb=0) == LD
    for name in ("dY", "X", "A", "B", "H"):
        assert backward(lib, **{name: None}) == NULLPTR, name
    assert backward(lib, n=8) == SCRATCH and backward(lib, ws=None) == ARG
    assert backward(lib, dX=None, dA=None, dB=None) == OK


def test_backward_alias(lib):
    assert backward(lib, dX=P[1]) == ALIAS and backward(lib, dX=P[7], lddx=7) == ALIAS
    assert backward(lib, dA=P[2]) == ALIAS and backward(lib, dB=P[3]) == ALIAS
    assert backward(lib, dA=P[10]) == ALIAS and backward(lib, dB=P[0]) == ALIAS
    assert backward(lib, dA=P[7]) == ALIAS               # only dX may be base
    assert backward(lib, dB=P[11]) == ALIAS


def ortho(lib, t=0, batch=2, M=4, N=6, G=P[0], ldg=6, sg=24, O=P[1], ldo=6, so=24, steps=1, coef=(1.5, -0.5, 0.0),
          eps=1e-7, ws=P[2], n=1 << 40):
    c = (ctypes.c_double * len(coef))(*coef) if coef is not None else None
    return lib.sgemm_orthogonalize(t, batch, M, N, G, ldg, sg, O, ldo, so, steps, c, eps, ws, n, None)


def test_ortho_refusals(lib):
    inf, nan = float("inf"), float("nan")
    assert ortho(lib, t=3) == ARG and ortho(lib, steps=0) == ARG and ortho(lib, steps=65) == ARG
    assert ortho(lib, eps=-1.0) == ARG and ortho(lib, eps=nan) == ARG and ortho(lib, eps=inf) == ARG
    assert ortho(lib, coef=(1.0, nan, 0.0)) == ARG and ortho(lib, coef=(inf, 0.0, 0.0)) == ARG
    assert ortho(lib, coef=(65.0, 0.0, 0.0)) == ARG and ortho(lib, coef=(0.0, 0.0, 0.0)) == ARG
    assert ortho(lib, coef=(1e-300, 0.0, 0.0)) == ARG
    assert ortho(lib, coef=(8.0, 0.0, 0.0) * 3, steps=3) == ARG       # grows past 64 in the third step
    assert ortho(lib, coef=None) == NULLPTR
    for name in ("batch", "M", "N"):
        assert ortho(lib, **{name: -1}) == DIM, name
    assert ortho(lib, M=65537) == DIM and ortho(lib, batch=65536) == DIM
    assert ortho(lib, ldg=5) == LD and ortho(lib, ldo=5) == LD and ortho(lib, so=23) == LD
    assert ortho(lib, G=None) == NULLPTR and ortho(lib, O=None) == NULLPTR
    assert ortho(lib, n=100) == SCRATCH and ortho(lib, ws=None) == ARG and ortho(lib, ws=P[2] + 16) == ARG
    assert ortho(lib, O=P[0] + 4) == ALIAS and ortho(lib, O=P[0], ldo=7, so=28) == ALIAS
    assert ortho(lib, O=P[2]) == ALIAS and ortho(lib, ws=P[0]) == ALIAS
    for name in ("batch", "M", "N"):
        assert ortho(lib, **{name: 0}, G=None, O=None) == OK, name


def test_workspaces(lib):
    assert lib.sgemm_lora_workspace(0, 3, 1, 1, 1, 1, 1) == -ARG
    assert lib.sgemm_lora_workspace(1, 0, 1, 1, 1, 300, 1) == -DIM
    assert lib.sgemm_orthogonalize_workspace(1, -1, 1) == -DIM
    for sizes in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (0, 0, 0), (70, 0, 0), (5000, 0, 9)):
        for backward in (0, 1):
            assert lib.sgemm_lora_workspace(backward, 0, *sizes, 4, 3) >= 0, sizes
        assert lib.sgemm_orthogonalize_workspace(*sizes) >= 0, sizes
    # Sizes stay in range at the largest arguments.
    big = (1 << 31) - 1
    assert lib.sgemm_lora_workspace(0, 2, 1, 4096, 4096, 16, 8) == 0
    assert 0 < lib.sgemm_lora_workspace(0, 0, big, big, big, 256, 4096) < 1 << 60
    assert 0 < lib.sgemm_lora_workspace(1, 0, big, big, big, 256, 4096) < 1 << 60
    assert 0 < lib.sgemm_orthogonalize_workspace(65535, 65536, 65536) < 1 << 60


def test_python_refusals():
    X, A, B = torch.zeros((4, 6)), torch.zeros((2, 3, 6)), torch.zeros((2, 5, 3))
    with pytest.raises(ValueError, match="GPU tensor"):
        rs.lora(X, A, B)
    with pytest.raises(TypeError):
        rs.lora(X.double(), A, B)
    with pytest.raises(TypeError):
        rs.orthogonalize(X.double())
    with pytest.raises(ValueError, match="matrix"):
        rs.orthogonalize(X[0])
    with pytest.raises(ValueError, match="triple"):
        rs.orthogonalize(X, coefficients=(1.0, 2.0))
    with pytest.raises(ValueError, match="triple"):
        rs.orthogonalize(X, coefficients=[])
    with pytest.raises(ValueError, match="GPU tensor"):
        rs.orthogonalize(X)


def test_reference_gradients_match_differences():
    gen = torch.Generator().manual_seed(5)
    M, N, K, R, L = 5, 4, 3, 2, 3
    X, A, B, ids, scale, _ = make(gen, M, N, K, R, L, torch.float32)
    ids = torch.tensor([0, 2, -1, 2, 0])
    args = [v.double() for v in (X, A, B)]
    dY = torch.randn((M, N), generator=gen, dtype=torch.float64)
    H = lora64(*args, ids, scale, None)[0][1]
    grads, _ = lora_backward64(dY, *args, H, ids, scale, None)
    for i, grad in enumerate(grads):
        for j in range(args[i].numel()):
            ends = []
            for h in (1e-6, -1e-6):
                moved = [a.clone() for a in args]
                moved[i].view(-1)[j] += h
                ends.append(float((lora64(*moved, ids, scale, None)[0][0] * dY).sum()))
            # Central difference of a polynomial of degree 1 in each argument:
            # only the 64-bit rounding of sums of order 10 over 2 h remains.
            assert abs((ends[0] - ends[1]) / 2e-6 - float(grad.reshape(-1)[j])) < 1e-7
    assert not grads[1][1].any() and not grads[2][1].any()  # no row has adapter 1


def test_coefficients_are_read_at_every_call():
    from roofline_sgemm_f32_amd.binding import _triples
    t = torch.tensor([2.0, -1.5, 0.5])
    assert list(_triples(t, 2)) == [2.0, -1.5, 0.5] * 2
    t[0] = 3.0
    assert list(_triples(t, 1)) == [3.0, -1.5, 0.5]
    u = torch.tensor([[2.0, -1.5, 0.5], [3.0, 0.0, 1.0]], dtype=torch.float64)
    assert list(_triples(u, 7)) == [2.0, -1.5, 0.5, 3.0, 0.0, 1.0]
    rows = [[2, -1.5, 0.5], (3, 0, 1)]
    assert list(_triples(rows, 7)) == list(_triples(u.numpy(), 7)) == list(u.flatten())
    for bad in ((), (1.0, 2.0), [[1.0, 2.0]], [(1, 2, 3), 4], torch.zeros(2, 2)):
        with pytest.raises(ValueError):
            _triples(bad, 1)
    with pytest.raises(ValueError):
        _triples((1.0, 2.0, 3.0), 0)

"""64-bit forms of the low-rank adapters, their gradients and the
orthogonalised update, with error bounds counted from the roundings, and input
makers shared by their tests."""
from __future__ import annotations

import math

import torch

from tests.ff_util import HALF_STEP, TINY, U  # noqa: F401

MUON = (3.4445, -4.7750, 2.0315)
# A value carried in two parts of 8 bits (bfloat16) is off by at most 2^-17 of
# itself; results of 16-bit types may be formed from such values of H and dH.
TWO_PARTS = {torch.float64: 0.0, torch.float32: 0.0, torch.float16: 2.0 ** -16, torch.bfloat16: 2.0 ** -16}


def sum_err(n):
    """Relative to the sum of magnitudes: n additions in float, each cut off
    (2 U) rather than rounded where a matrix instruction adds inside, and 24
    more where a sum is shared out and joined."""
    return 2 * (n + 24) * U


def make(gen, M, N, K, R, L, dtype, ids="mixed"):
    X = torch.randn((M, K), generator=gen).to(dtype)
    A = (torch.randn((L, R, K), generator=gen) / math.sqrt(max(K, 1))).to(dtype)
    B = (torch.randn((L, N, R), generator=gen) / math.sqrt(R)).to(dtype)
    base = torch.randn((M, N), generator=gen).to(dtype)
    scale = 0.5 + torch.rand((L,), generator=gen)
    if ids == "mixed":
        of = torch.randint(-1, L, (M,), generator=gen, dtype=torch.int32)
    elif ids == "runs":
        of = torch.sort(torch.randint(0, L, (M,), generator=gen, dtype=torch.int32))[0]
    elif ids == "one":
        of = torch.full((M,), L - 1, dtype=torch.int32)
    else:
        of = torch.full((M,), -1, dtype=torch.int32)
    return X, A, B, of, scale, base


def lora64(X, A, B, ids, scale, base):
    """(Y, H) in float64 on the CPU, and bounds on their float errors before
    the rounding to the type."""
    t = X.dtype
    X, A, B, scale = (v.detach().cpu().double() for v in (X, A, B, scale))
    (M, K), (L, R, _), N = X.shape, A.shape, B.shape[1]
    Y = base.detach().cpu().double().clone() if base is not None else torch.zeros((M, N), dtype=torch.float64)
    H = torch.zeros((M, R), dtype=torch.float64)
    eY, eH = 2 * U * Y.abs(), torch.zeros_like(H)
    for m in range(M):
        l = int(ids[m])
        if not 0 <= l < L:
            eY[m] = 0
            continue
        H[m] = A[l] @ X[m]
        eH[m] = sum_err(K) * (A[l].abs() @ X[m].abs())
        d, s = B[l] @ H[m], float(scale[l])
        e = B[l].abs() @ eH[m] + (sum_err(R) + TWO_PARTS[t]) * (B[l].abs() @ (H[m].abs() + eH[m]))
        eY[m] += s * (e + 3 * U * d.abs()) + 2 * U * (s * d).abs()
        Y[m] += s * d
    return (Y, H), (eY, eH)


def lora_backward64(dY, X, A, B, H, ids, scale, base):
    """(dX, dA, dB) in float64 on the CPU and their bounds."""
    t = X.dtype
    dY, X, A, B, H, scale = (v.detach().cpu().double() for v in (dY, X, A, B, H, scale))
    (M, K), (L, R, _), N = X.shape, A.shape, B.shape[1]
    dX = base.detach().cpu().double().clone() if base is not None else torch.zeros((M, K), dtype=torch.float64)
    eX = 2 * U * dX.abs()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    eA, eB = torch.zeros_like(A), torch.zeros_like(B)
    ids = ids.cpu()
    two = TWO_PARTS[t]
    for l in range(L):
        rows = (ids == l).nonzero()[:, 0]
        n, s = len(rows), float(scale[l])
        if not n:
            continue
        dy, x, h = dY[rows], X[rows], H[rows]
        dH = s * (dy @ B[l])
        eH = abs(s) * (sum_err(N) + 4 * U) * (dy.abs() @ B[l].abs())
        mag = dH.abs() + eH
        dX[rows] += dH @ A[l]
        eX[rows] += eH @ A[l].abs() + (sum_err(R) + two + 4 * U) * (mag @ A[l].abs())
        dA[l] = dH.t() @ x
        eA[l] = eH.t() @ x.abs() + (sum_err(n) + two) * (mag.t() @ x.abs())
        dB[l] = s * (dy.t() @ h)
        eB[l] = abs(s) * (sum_err(n) + two + 4 * U) * (dy.abs().t() @ h.abs())
    eX[~((ids >= 0) & (ids < L))] = 0
    return (dX, dA, dB), (eX, eA, eB)


def ortho64(G, coefficients, eps=1e-7, device="cpu"):
    """The update of one matrix in float64."""
    X = G.detach().to(device).double()
    X = X / (X.norm() + eps)
    for a, b, c in coefficients:
        S = X @ X.t()
        X = a * X + (b * S + c * S @ S) @ X
    return X


# Stored values have two float16 parts, 22 bits: off by at most Q of
# themselves, or by half the smallest float16 step under the power of two that
# scales them (2^-25 / 2^8 at least: bounds up to 64, factors up to 2^7 here).
Q, FLOOR = 2.0 ** -22, 2.0 ** -33


def product_err(k):
    """A product of two stored values without its low parts' product, summed
    over k: relative to the sum of magnitudes."""
    return 3 * Q + sum_err(k)


def ortho_step64(G, abc, eps=1e-7, device="cpu"):
    """One step in float64 and an elementwise bound of its error."""
    a, b, c = abc
    X = G.detach().to(device).double()
    if X.shape[0] > X.shape[1]:
        O, e = ortho_step64(G.t(), abc, eps, device)
        return O.t(), e.t()
    X = X / (X.norm() + eps)
    m, n = X.shape
    ax = X.abs()
    ex = (3 * U + Q) * ax + FLOOR
    S = X @ X.t()
    eS = product_err(n) * (ax @ ax.t()) + ex @ ax.t() + ax @ ex.t() + Q * S.abs() + FLOOR
    aS = S.abs() + eS
    eye = torch.eye(m, dtype=torch.float64, device=device)
    P = a * eye + b * S + c * (S @ S)
    eP = abs(b) * eS + abs(c) * (eS @ aS + aS @ eS + product_err(m) * (aS @ aS)) + Q * P.abs() + FLOOR
    eP += 4 * U * (abs(a) * eye + abs(b) * aS + abs(c) * (aS @ aS))
    aP = P.abs() + eP
    return P @ X, eP @ ax + aP @ ex + product_err(m) * (aP @ ax) + FLOOR


def ortho_norm_bound(G, coefficients, eps=1e-7, device="cpu"):
    """A bound of the Frobenius norm of the error after all steps.  A step's own
    error: a sum of k products x_i y_i has partial sums of at most |x| |y|, so k
    / 16 roundings of 2 U (matrix instructions add 16 at a time) and the parts'
    3 Q are relative to |X| |Y|, Frobenius norms.  Earlier errors grow at most
    by the largest |p'| over the singular values reached (the divided
    differences of an odd p are at most that); the values themselves may be off
    by a little, which the factor 1.05 covers."""
    X = G.detach().to(device).double()
    if X.shape[0] > X.shape[1]:
        X = X.t()
    X = X / (X.norm() + eps)
    m, n = X.shape
    e = (3 * U + Q) * X.norm()

    def rel(k):
        return 3 * Q + 2 * (k / 16 + 24) * U

    for a, b, c in coefficients:
        S = X @ X.t()
        P = a * torch.eye(m, dtype=torch.float64, device=device) + b * S + c * S @ S
        top = float(torch.linalg.matrix_norm(X, 2))
        s = torch.linspace(0, 1.05 * top, 2001, dtype=torch.float64)
        lip = float((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max())
        xf = float(X.norm())
        eS = (rel(n) + Q) * xf * xf
        sn = float(S.norm())
        eP = abs(b) * eS + abs(c) * (2 * top ** 2 * eS + rel(m) * sn * sn) + (Q + 4 * U) * float(P.norm())
        own = eP * top + (rel(m) + Q) * float(P.norm()) * xf
        X = P @ X
        e = lip * e + own
    return float(e)

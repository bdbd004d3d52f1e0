"""64-bit forms of the gated feed-forward block and of the products with
4-bit weights, with error bounds counted from the roundings of float sums,
and input makers shared by their tests."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24  # unit roundoff of float32
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# A rounding to the result's type is off by at most half a step.
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
LIPSCHITZ = 1.13  # largest |act'| of any of the activations (gelu: 1.129)


def act64(name, g):
    """(act(g), act'(g)) in float64."""
    if name == "relu":
        return g.clamp_min(0), (g > 0).double()
    s = torch.sigmoid(g)
    if name == "sigmoid":
        return s, s * torch.sigmoid(-g)
    if name == "silu":
        return g * s, s * (1 + g * torch.sigmoid(-g))
    if name == "gelu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * g * g)


def act_err(g):
    """Bound of one float evaluation of an activation or its derivative:
    sixteen roundings relative to |g| + 1 (exp, erfc and a division are good
    to a few units; an argument v of exp that is off by 2 u |v| moves the
    result by at most 2 u |v| s (1 - s) <= u)."""
    return 16 * U * (g.abs() + 1)


def glu64(act, X, Wg, Wu):
    """H, G, U and bounds on their float errors; weights K x F, float64."""
    K = X.shape[1]
    G, Up = X @ Wg, X @ Wu
    eg, eu = (4 * K * U * (X.abs() @ W.abs()) for W in (Wg, Wu))
    a, _ = act64(act, G)
    H = a * Up
    ea = LIPSCHITZ * eg + act_err(G)
    eh = ea * (Up.abs() + eu) + a.abs() * eu + 2 * U * H.abs()
    return (H, G, Up), (eh, eg, eu)


def glu_backward64(act, X, Wg, Wu, G, Up, dH):
    """dG, dU, dX, dWg, dWu and bounds; weights K x F, all float64."""
    M, K = X.shape
    F = G.shape[1]
    a, da = act64(act, G)
    dG, dU = dH * Up * da, dH * a
    eG = dH.abs() * Up.abs() * act_err(G) + 3 * U * dG.abs()
    eU = dH.abs() * act_err(G) + 2 * U * dU.abs()
    dX = dG @ Wg.t() + dU @ Wu.t()
    eX = (eG + 4 * (2 * F + 2) * U * dG.abs()) @ Wg.t().abs() + \
         (eU + 4 * (2 * F + 2) * U * dU.abs()) @ Wu.t().abs()
    dWg, dWu = X.t() @ dG, X.t() @ dU
    eWg, eWu = (X.t().abs() @ (e + 4 * M * U * d.abs()) for e, d in ((eG, dG), (eU, dU)))
    return (dG, dU, dX, dWg, dWu), (eG, eU, eX, eWg, eWu)


def q4_make(gen, N, K, group, stype, zeros, device="cuda"):
    """Random packed weights (bytes, scales, zero points or None)."""
    groups = -(-K // group)
    w = torch.randint(0, 256, (N, (K + 1) // 2), generator=gen, dtype=torch.uint8)
    s = ((torch.rand((N, groups), generator=gen) + 0.5) / (4 * math.sqrt(max(K, 1)))).to(stype)
    z = torch.randint(0, 16, (N, groups), generator=gen, dtype=torch.uint8) if zeros else None
    return tuple(t.to(device) if t is not None else None for t in (w, s, z))


def q4_int(w, z, K, group):
    """q - z as float64, N x K."""
    b = w.cpu().to(torch.int64)
    q = torch.stack([b & 15, b >> 4], 2).flatten(1)[:, :K]
    zz = z.cpu().to(torch.int64).repeat_interleave(group, 1)[:, :K] if z is not None else 8
    return (q - zz).double()


def q4_64(X, w, s, z, group):
    """X W^T in float64 and a bound on its error in float sums: at most
    `group` additions within a group, one scaling and addition per group and
    up to 24 more where a row's groups are shared out and joined."""
    K = X.shape[1]
    X = X.cpu().double()
    W = q4_int(w, z, K, group) * s.cpu().double().repeat_interleave(group, 1)[:, :K]
    n = min(K, group) + s.shape[1] + 24
    return X @ W.t(), n * U * (X.abs() @ W.t().abs())


def rounded(ref, err, dtype):
    """The bound after the result is rounded once to dtype."""
    return err + HALF_STEP[dtype] * (ref.abs() + err) + TINY[dtype]


def assert_within(got, ref, err, what=""):
    """got within err of ref, elementwise, with what is worst on failure."""
    d = (got.detach().cpu().double() - ref).abs()
    bad = ~(d <= err)
    if bad.any():
        i = int(torch.where(bad.flatten(), d.flatten() / err.flatten().clamp_min(1e-300), 0).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; worst at "
                             f"{i}: got {float(got.flatten()[i])}, want {float(ref.flatten()[i])} "
                             f"+- {float(err.flatten()[i])}")


class Guarded:
    """A rows x cols output inside a larger buffer: NaN where it is to be
    written, a sentinel in the row gaps and after the end."""

    def __init__(self, rows, cols, dtype=torch.float32, gap=0, tail=67):
        self.ld = cols + gap
        self.buf = torch.full((rows * self.ld + tail,), 77.0, dtype=dtype, device="cuda")
        self.view = torch.as_strided(self.buf, (rows, cols), (max(self.ld, 1), 1))
        self.view.fill_(float("nan"))

    def intact(self):
        keep = self.buf.clone()
        torch.as_strided(keep, self.view.shape, self.view.stride()).fill_(77.0)
        return bool((keep == 77.0).all())

"""H and dH of low-rank adapters count in full on the 16-bit matrix instructions:
to float's own precision, and beside infinities as the formula has it."""
import math

import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.ff_util import TYPES, U, assert_within, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


# (M, N, K, R, L): one launch for few rows; single rows; tiles of 16 rows (many
# adapters) and of 64 (few), each with ranks of every form, aligned and odd.
FORMS = [(3, 70, 40, 8, 2), (40, 700, 96, 40, 5),
         (100, 130, 72, 8, 40), (100, 72, 200, 12, 40), (90, 200, 136, 32, 30), (100, 264, 72, 64, 40),
         (90, 70, 300, 67, 30), (100, 130, 72, 200, 40),
         (200, 130, 72, 8, 2), (200, 72, 200, 12, 2), (150, 200, 136, 32, 1), (200, 264, 72, 40, 2),
         (300, 72, 300, 67, 3), (200, 136, 72, 128, 1), (200, 130, 72, 200, 2), (140, 70, 40, 255, 1)]
NAMES = ["x".join(map(str, f)) for f in FORMS]


def rows_of(gen, M, L):
    """An adapter for each row; the first two rows have the first."""
    ids = torch.randint(0, L, (M,), generator=gen, dtype=torch.int32)
    ids[:2] = 0
    return ids


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("form", FORMS, ids=NAMES)
def test_a_base_that_nearly_cancels(form, t):
    """One rank is not zero, so that H is one product of 22 bits at most and the
    sums over ranks add zeros; base is minus the rounded correction, and what is
    left shows the last bits of H, and of dH."""
    M, N, K, R, L = form
    dt = TYPES[t]
    gen = torch.Generator().manual_seed(FORMS.index(form))
    ids = rows_of(gen, M, L)
    r0, k0, n0 = R // 2, K // 3, N // 3
    X, A, B = torch.zeros((M, K)), torch.zeros((L, R, K)), torch.zeros((L, N, R))
    X[:, k0] = torch.randn((M,), generator=gen)
    A[:, r0, k0] = torch.randn((L,), generator=gen)
    B[:, :, r0] = torch.randn((L, N), generator=gen)
    X, A, B = X.to(dt), A.to(dt), B.to(dt)
    scale = 0.5 + torch.rand((L,), generator=gen)
    of, s = ids.long(), scale.double()[ids.long()][:, None]
    # In float32 H is rounded; in the 16-bit types it is exact.
    h = X[:, k0].double()[:, None] * A[of, r0, k0].double()[:, None]
    d = s * h * B[of, :, r0].double()
    base = (-d).to(dt)
    ref = base.double() + d
    # One product of H with an element of B, its (up to four) parts added, the scale
    # and base: at most eight roundings of 2 U of |d|.  Of float16, H beside a power of
    # two for its row, here of one number: nothing more.
    err = 16 * U * d.abs()
    Y, H = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=base.cuda(), save=True)
    want = torch.zeros((M, R), dtype=torch.float64)
    want[:, r0] = h[:, 0]
    assert_within(H, want, 2 * U * want.abs(), "H")
    assert_within(Y, ref, rounded(ref, err, dt), "Y")
    # dH = s dY B of one column, dX = base + dH A.
    dY = torch.zeros((M, N))
    dY[:, n0] = torch.randn((M,), generator=gen)
    A2 = torch.zeros((L, R, K))
    A2[:, r0] = torch.randn((L, K), generator=gen)
    dY, A2 = dY.to(dt), A2.to(dt)
    dh = s * dY[:, n0].double()[:, None] * B[of, n0, r0].double()[:, None]
    d = dh * A2[of, r0].double()
    base = (-d).to(dt)
    ref = base.double() + d
    dX, _, _ = rs.lora_backward(dY.cuda(), X.cuda(), A2.cuda(), B.cuda(), H, ids.cuda(), scale=scale.cuda(),
                                base=base.cuda(), need_dw=False)
    assert_within(dX, ref, rounded(ref, 16 * U * d.abs(), dt), "dX")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("R", [1, 8, 13, 16, 32, 45, 64, 130, 256])
@pytest.mark.parametrize("M", [2, 70, 1200])
def test_rows_that_nearly_cancel(M, R, t):
    """Two rows whose products differ by 2^-14 of themselves; the others are zero."""
    dt = TYPES[t]
    gen = torch.Generator().manual_seed(M + R)
    N, K, r0 = 72, 136, R // 2
    i, j = (0, 1) if M == 2 else (3, M - 2)
    scale = torch.tensor([1.2345678, 0.5772157])
    ids = torch.ones((M,), dtype=torch.int32)
    x = torch.randn((K,), generator=gen).to(dt)
    X = torch.zeros((M, K), dtype=dt)
    X[i], X[j] = x, -x
    A = torch.zeros((2, R, K), dtype=dt)
    B = torch.zeros((2, N, R), dtype=dt)
    dY = torch.zeros((M, N), dtype=dt)
    B[1, 0, r0], B[1, 1, r0] = 1.0, 2.0 ** -7
    dY[i, 0] = dY[j, 0] = 1.0
    dY[j, 1] = 2.0 ** -7
    H = torch.zeros((M, R))
    H[i, r0] = scale[1]                       # any number of 24 bits
    H[j, r0] = -scale[1] * (1 + 2.0 ** -14)
    _, dA, dB = rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), H.cuda(), ids.cuda(), scale=scale.cuda(),
                                 need_dx=False)
    s = scale.double()[1]
    want = torch.zeros((2, R, K), dtype=torch.float64)
    want[1, r0] = s * -2.0 ** -14 * x.double()
    mag = s * x.double().abs()
    err = torch.zeros_like(want)
    # dH of the two rows: three roundings of 2 U; the parts of each added, and each
    # other: eight at most.
    err[1, r0] = 2 * 11 * U * mag
    assert_within(dA, want, rounded(want, err, dt), "dA")
    want = torch.zeros((2, N, R), dtype=torch.float64)
    err = torch.zeros_like(want)
    want[1, 0, r0] = s * (H[i, r0].double() + H[j, r0].double())
    want[1, 1, r0] = s * 2.0 ** -7 * H[j, r0].double()
    err[1, :2, r0] = 2 * 9 * U * torch.tensor([2.0, 2.0 ** -7], dtype=torch.float64) * s * H[j, r0].double().abs()
    assert_within(dB, want, rounded(want, err, dt), "dB")


def same_kind(got, ref, what):
    """NaN and infinities where the formula has them, of its sign."""
    got = got.detach().cpu().double()
    for name, f in (("NaN", torch.isnan), ("inf", lambda v: v == math.inf), ("-inf", lambda v: v == -math.inf)):
        bad = f(got) != f(ref)
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} wrong as {name}; first at " \
                              f"{bad.nonzero()[0].tolist()}: got {float(got[bad][0])}, want {float(ref[bad][0])}"


def product(a, b):
    """a @ b in float64, term by term."""
    return torch.stack([(r[:, None] * b).sum(0) for r in a]) if len(a) else a @ b


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("form", FORMS, ids=NAMES)
def test_infinities(form, t):
    """An infinite element of B, A, X or dY: h inf is an infinity of h's sign also
    where h is a small whole number, whose low bits are zero, and NaN only where the
    formula has 0 inf or inf - inf."""
    M, N, K, R, L = form
    dt, inf = TYPES[t], math.inf
    gen = torch.Generator().manual_seed(100 + FORMS.index(form))
    ids = rows_of(gen, M, L)
    of = ids.long()

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=gen).to(dt)

    X, A, B, base = whole(M, K), whole(L, R, K), whole(L, N, R), whole(M, N)
    for r in range(0, R, 2):  # half of the ranks' H are not whole
        A[:, r] = (A[:, r].float() * (1 + torch.rand((L, K), generator=gen))).to(dt)
    scale = torch.ones((L,))
    scale[-1] = -0.5
    # Every adapter: an infinity in a row of B of its own rank; in one row of X; in
    # base, of both signs against B's.
    for l in range(L):
        B[l, 3, l % R] = inf
        B[l, 5, (l + 1) % R] = -inf
    X[2, K // 2] = inf
    X[1] = 0                                   # H = 0: 0 inf
    base[:, 3] = inf
    base[::2, 9] = -inf
    h = torch.stack([(A[of[m]].double() * X[m].double()).sum(1) for m in range(M)])
    d = torch.stack([(B[of[m]].double() * h[m]).sum(1) for m in range(M)]) * scale.double()[of][:, None]
    Y, H = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=base.cuda(), save=True)
    same_kind(H, h, "H")
    same_kind(Y, base.double() + d, "Y")
    # Backward: finite H, infinities in dY, X and A (each once for a row or adapter).
    dY, Hs = whole(M, N), torch.randint(-3, 4, (M, R), generator=gen).float()
    B, X = whole(L, N, R), whole(M, K)
    Hs[:, ::2] *= 1 + torch.rand((M, (R + 1) // 2), generator=gen)
    dY[0, 2] = inf
    dY[1, 4] = -inf
    X[2, 5] = inf
    X[-1, 6] = -inf
    for l in range(L):
        A[l, l % R, 7] = inf
    s = scale.double()[of][:, None]
    dH = torch.stack([(B[of[m]].double() * dY[m].double()[:, None]).sum(0) for m in range(M)]) * s
    dXr = torch.stack([(A[of[m]].double() * dH[m][:, None]).sum(0) for m in range(M)])
    dX, dA, dB = rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), Hs.cuda(), ids.cuda(), scale=scale.cuda())
    same_kind(dX, dXr, "dX")
    for l in range(L):
        rows = (of == l).nonzero()[:, 0]
        if not len(rows):
            assert not dA[l].any() and not dB[l].any()
            continue
        same_kind(dA[l], product(dH[rows].t(), X[rows].double()), f"dA {l}")
        same_kind(dB[l], product((s[rows] * dY[rows].double()).t(), Hs[rows].double()), f"dB {l}")


@pytest.mark.parametrize("M, L", [(100, 40), (200, 1)])
def test_small_numbers_beside_infinities(M, L):
    """h inf is an infinity for numbers far below the row's (and the rank's) largest
    too, whose parts would be zero."""
    N, K, R = 70, 40, 16
    gen = torch.Generator().manual_seed(M)
    ids = rows_of(gen, M, L)
    X = torch.zeros((M, K), dtype=torch.float16)
    A = torch.zeros((L, R, K), dtype=torch.float16)
    B = torch.ones((L, N, R), dtype=torch.float16)
    X[:, 0], X[:, 1] = 2.0 ** 10, 2.0 ** -20
    A[:, 0, 0], A[:, 1:, 1] = 2.0 ** 10, 2.0 ** -14
    B[:, 4, 5] = -math.inf
    Y = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda()).cpu()
    assert bool((Y[:, 4] == -math.inf).all()) and bool((Y[:, 5] == math.inf).all())  # 2^20
    H = torch.full((M, R), 2.0 ** -30)
    H[0] = 2.0 ** 10
    dY = torch.ones((M, N), dtype=torch.float16)
    dY[1, 6] = math.inf
    _, _, dB = rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), H.cuda(), torch.zeros_like(ids).cuda(),
                                need_dx=False)
    assert bool((dB[0, 6] == math.inf).all()) and bool(torch.isfinite(dB[0, :6]).all())


@pytest.mark.parametrize("M, L", [(3, 1), (100, 40), (200, 1)])
def test_zero_adapters_with_the_largest_scale(M, L):
    """A correction of zero times any finite scale is zero: the factor that undoes
    float16's power of two must not be infinite."""
    N, K, R = 600, 64, 16
    gen = torch.Generator().manual_seed(M)
    ids = rows_of(gen, M, L)
    X = torch.full((M, K), 2.0 ** 10).half()
    A = torch.full((L, R, K), 2.0 ** 10).half()
    B = torch.zeros((L, N, R)).half()
    base = torch.randn((M, N), generator=gen).half()
    scale = torch.full((L,), 3e38)
    args = (X.cuda(), A.cuda(), B.cuda(), ids.cuda())
    assert torch.equal(rs.lora(*args, scale=scale.cuda(), base=base.cuda()).cpu(), base)
    B[:, 1] = 1
    Y = rs.lora(args[0], args[1], B.cuda(), args[3], scale=scale.cuda(), base=base.cuda()).cpu()
    assert bool((Y[:, 1] == math.inf).all()) and torch.equal(Y[:, 2:], base[:, 2:])
    # dB from H above 2^15 and dY of zeros.
    H = torch.full((M, R), 2.0 ** 30)
    dY = torch.zeros((M, N)).half()
    _, dA, dB = rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), H.cuda(), ids.cuda(), scale=scale.cuda(),
                                 need_dx=False)
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("M, L, R", [(3, 1, 16), (100, 40, 16), (100, 40, 40), (200, 1, 16), (200, 1, 40)])
@pytest.mark.parametrize("e", [-100, -120, -126])
def test_the_smallest_normal_numbers_beside_infinities(e, M, L, R, t):
    """H = 2^e: what its parts hold is below bfloat16's normal numbers."""
    N, K, dt = 70, 40, TYPES[t]
    gen = torch.Generator().manual_seed(M)
    ids = rows_of(gen, M, L)
    X, A, B = torch.zeros((M, K)), torch.zeros((L, R, K)), torch.ones((L, N, R))
    X[:, 0], A[:, :, 0] = 2.0 ** (e // 2), 2.0 ** (e - e // 2)
    B[:, 4, 5], B[:, 6, 1] = -math.inf, math.inf
    Y, H = rs.lora(X.to(dt).cuda(), A.to(dt).cuda(), B.to(dt).cuda(), ids.cuda(), save=True)
    assert bool((H == 2.0 ** e).all())
    Y = Y.cpu()
    assert bool((Y[:, 4] == -math.inf).all()) and bool((Y[:, 6] == math.inf).all())
    # The parts of 2^e in whole numbers of the type's smallest, 2^-133: three roundings.
    assert_within(Y[:, :4], torch.full((M, 4), R * 2.0 ** e, dtype=torch.float64),
                  rounded(torch.tensor(R * 2.0 ** e, dtype=torch.float64), R * (3 * 2.0 ** -133 + 2 * (R + 24) * U * 2.0 ** e),
                          dt).expand(M, 4))
    dY = torch.ones((M, N))
    dY[1, 6] = math.inf
    _, _, dB = rs.lora_backward(dY.to(dt).cuda(), X.to(dt).cuda(), A.to(dt).cuda(), B.to(dt).cuda(), H,
                                torch.zeros_like(ids).cuda(), need_dx=False)
    assert bool((dB[0, 6] == math.inf).all()) and bool(torch.isfinite(dB[0, :6]).all())

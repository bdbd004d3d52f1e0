"""Low-rank adapters and their gradients on the GPU, against the 64-bit sums
within counted bounds."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.adapt_util import lora64, lora_backward64, make
from tests.ff_util import TYPES, Guarded, assert_within, q4_64, q4_make, rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


# (M, N, K, R, L, ids): one token to many rows; odd everywhere; ranks below,
# at and past the matrix instructions' 16, 32 and 64; more adapters than rows;
# rows without adapter; one adapter for all.
SHAPES = [(1, 64, 128, 16, 1, "one"), (1, 1, 1, 1, 1, "one"), (1, 4096, 4096, 16, 8, "one"),
          (1, 33, 70, 16, 4, "none"), (2, 65, 129, 3, 5, "mixed"), (3, 256, 513, 64, 2, "mixed"),
          (5, 100, 96, 8, 40, "mixed"), (8, 72, 2048, 256, 3, "mixed"), (16, 512, 640, 32, 4, "mixed"),
          (17, 31, 1000, 17, 3, "runs"), (33, 130, 64, 16, 33, "mixed"), (64, 264, 1032, 16, 9, "mixed"),
          (65, 63, 65, 33, 2, "runs"), (100, 1024, 256, 12, 100, "mixed"), (129, 128, 512, 64, 3, "runs"),
          (200, 511, 200, 100, 4, "mixed"), (257, 320, 384, 16, 5, "mixed"), (300, 1000, 72, 128, 1, "one"),
          (513, 96, 96, 8, 700, "mixed"), (777, 40, 31, 5, 2, "runs"), (1000, 64, 48, 4, 3, "none"),
          (1030, 136, 264, 65, 3, "runs"), (2049, 24, 16, 2, 6, "mixed")]


def where(ids, i):
    return ids.cuda().to((torch.int32, torch.int64)[i % 2])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, t):
    M, N, K, R, L, kind = shape
    i = SHAPES.index(shape) + list(TYPES).index(t)
    gen = torch.Generator().manual_seed(i)
    X, A, B, ids, scale, base = make(gen, M, N, K, R, L, TYPES[t], kind)
    gap = (0, 1, 8)[i % 3]
    Y, H = Guarded(M, N, TYPES[t], gap=gap), Guarded(M, R, gap=i % 2)
    rs.lora(X.cuda(), A.cuda(), B.cuda(), where(ids, i), scale=scale.cuda(), base=base.cuda(), out=Y.view,
            save=H.view)
    (ref, h), (err, eh) = lora64(X, A, B, ids, scale, base)
    assert_within(H.view, h, eh, "H")
    assert_within(Y.view, ref, rounded(ref, err, TYPES[t]), "Y")
    assert Y.intact() and H.intact()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, t):
    M, N, K, R, L, kind = shape
    i = SHAPES.index(shape) + list(TYPES).index(t)
    gen = torch.Generator().manual_seed(100 + i)
    X, A, B, ids, scale, _ = make(gen, M, N, K, R, L, TYPES[t], kind)
    dY = torch.randn((M, N), generator=gen).to(TYPES[t])
    H = torch.randn((M, R), generator=gen)
    base = torch.randn((M, K), generator=gen).to(TYPES[t])
    gap = (1, 8, 0)[i % 3]
    dX = Guarded(M, K, TYPES[t], gap=gap)
    dA, dB = Guarded(L * R, K, TYPES[t], gap=gap), Guarded(L * N, R, TYPES[t], gap=gap)
    dW = [g.buf.as_strided((L, r, c), (r * g.ld, g.ld, 1)) for g, r, c in ((dA, R, K), (dB, N, R))]
    rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), H.cuda(), where(ids, i), scale=scale.cuda(),
                     base=base.cuda(), dX=dX.view, dW=dW)
    refs, errs = lora_backward64(dY, X, A, B, H, ids, scale, base)
    for name, got, ref, err, guard in zip(("dX", "dA", "dB"), (dX.view, *dW), refs, errs, (dX, dA, dB)):
        assert_within(got, ref, rounded(ref, err, TYPES[t]), name)
        assert guard.intact(), name


# More rows than the sort holds at a time, in many groups and few; the most adapters.
@pytest.mark.parametrize("M, L, kind", [(8192, 3, "mixed"), (9001, 7, "mixed"), (9000, 4096, "mixed"), (20000, 40, "runs"),
                                        (8200, 1, "one"), (150, 4096, "mixed"), (65, 2, "none")])
def test_many_rows(M, L, kind):
    gen = torch.Generator().manual_seed(M)
    N, K, R = 24, 16, 4
    dt = (torch.float16, torch.bfloat16, torch.float32)[M % 3]
    X, A, B, ids, scale, base = make(gen, M, N, K, R, L, dt, kind)
    dY = torch.randn((M, N), generator=gen).to(dt)
    of = ids.long().clamp_min(0)
    has = (ids >= 0)[:, None].double()
    x, a, b, sc = X.double(), A.double()[of], B.double()[of], (scale.double()[of] * has[:, 0])[:, None]
    h = (a * x[:, None, :]).sum(2) * has
    eh = 2 * (K + 24) * 2.0 ** -24 * (a.abs() * x.abs()[:, None, :]).sum(2)
    d = (b * h[:, None, :]).sum(2)
    ed = (b.abs() * (eh + (2 * (R + 24) * 2.0 ** -24 + 2.0 ** -16) * h.abs())[:, None, :]).sum(2)
    ref = base.double() + sc * d
    err = sc * (ed + 4 * 2.0 ** -24 * d.abs()) + 4 * 2.0 ** -24 * (ref.abs() + base.double().abs())
    Y, H = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=base.cuda(), save=True)
    assert_within(H, h, eh, "H")
    assert_within(Y, ref, rounded(ref, err, dt), "Y")
    Hh = torch.randn((M, R), generator=gen)
    refs, errs = lora_backward64(dY, X, A, B, Hh, ids, scale, None)
    got = rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), Hh.cuda(), ids.cuda(), scale=scale.cuda())
    for name, g, r, e in zip(("dX", "dA", "dB"), got, refs, errs):
        assert_within(g, r, rounded(r, e, dt), name)


def test_small_halves_are_not_flushed():
    """float16 adapters and activations below its normal numbers count in full."""
    gen = torch.Generator().manual_seed(8)
    for M in (2, 40, 200):
        X, A, B, ids, scale, _ = make(gen, M, 72, 96, 16, 3, torch.float16)
        X, A, B = (v * 2.0 ** -16 if v is not B else v for v in (X, A, B)) if M == 2 else (X * 2.0 ** -17, A, B * 2.0 ** -16)
        scale = scale * 2.0 ** 30
        (ref, h), (err, eh) = lora64(X, A, B, ids, scale, None)
        Y, H = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), save=True)
        assert_within(H, h, eh, "H")
        assert_within(Y, ref, rounded(ref, err, torch.float16), "Y")


def test_offsets_past_32_bits():
    """Results and activations of more than 2^32 bytes: the first and last rows."""
    M, wide, N, K, R = 70000, 33000, 32768, 24, 4
    gen = torch.Generator().manual_seed(11)
    A, B = torch.randn((1, R, K), generator=gen).bfloat16(), torch.randn((1, N, R), generator=gen).bfloat16()
    buf = torch.zeros((M, wide), dtype=torch.bfloat16, device="cuda")
    X = buf[:, wide - K:]
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1])
    x = torch.randn((len(rows), K), generator=gen).bfloat16()
    X[rows.cuda()] = x.cuda()
    Y = rs.lora(X, A.cuda(), B.cuda())
    (ref, _), (err, _) = lora64(x, A, B, torch.zeros(len(rows), dtype=torch.int32), torch.ones(1), None)
    assert_within(Y[rows.cuda()], ref, rounded(ref, err, torch.bfloat16))
    assert not Y[2].any()
    # The same buffers as gradients: dY is Y, dX of its own.
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    H = torch.zeros((M, R), device="cuda")
    h = torch.randn((len(rows), R), generator=gen)
    H[rows.cuda()] = h.cuda()
    dy = Y[rows.cuda()].cpu()
    refs, errs = lora_backward64(dy, x, A, B, h, torch.zeros(len(rows), dtype=torch.int32), torch.ones(1), None)
    dX, dA, dB = rs.lora_backward(Y, X, A.cuda(), B.cuda(), H, ids)
    # Sums over 70000 rows, of which these few are not zero: adding zeros rounds nothing.
    for got, r, e in zip((dX[rows.cuda()], dA, dB), refs, errs):
        assert_within(got, r, rounded(r, 2 * e, torch.bfloat16))


def test_gradient_against_differences():
    """The kernels' own forward pass in float32 moved along one direction."""
    gen = torch.Generator().manual_seed(3)
    M, N, K, R, L = 70, 33, 40, 4, 3
    X, A, B, ids, scale, _ = (v.cuda() for v in make(gen, M, N, K, R, L, torch.float32))
    dY = torch.randn((M, N), generator=gen).cuda()
    _, H = rs.lora(X, A, B, ids, scale=scale, save=True)
    grads = rs.lora_backward(dY, X, A, B, H, ids, scale=scale)
    for i, grad in enumerate(grads):
        args = [X, A, B]
        d = torch.randn(args[i].shape, generator=gen).cuda()
        h = 0.125  # the map is linear in each argument: any step, no cut-off error
        ends = []
        for step in (h, -h):
            moved = list(args)
            moved[i] = args[i] + step * d
            ends.append((rs.lora(*moved, ids, scale=scale).double() * dY.double()).sum())
        got, want = float((ends[0] - ends[1]) / (2 * h)), float((grad.double() * d.double()).sum())
        # Each of the M N outputs is off by less than 2^-17 of |Y| <= 60, with
        # signs of their own: 8 sqrt(M N) 60 2^-17 / (2 h) at the very most.
        assert abs(got - want) < 8 * (M * N) ** 0.5 * 60 * 2 ** -17 / (2 * h), i


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M", [1, 7, 300])
def test_views_in_place_and_defaults(M, t):
    """Column views of wider buffers at odd offsets, adapters sliced from wider
    stacks or expanded from one, base overwritten, no ids, number as scale."""
    gen = torch.Generator().manual_seed(M)
    N, K, R, L, dt = 45, 77, 5, 3, TYPES[t]
    X, A, B, ids, scale, base = make(gen, M, N, K, R, L, dt)
    wide = lambda v: torch.cat([torch.full((*v.shape[:-1], 3), float("nan"), dtype=v.dtype), v,
                                torch.full((*v.shape[:-1], 2), float("nan"), dtype=v.dtype)], -1).cuda()[..., 3:-2]
    Yb = wide(base)
    (ref, _), (err, _) = lora64(X, A, B, ids, scale, base)
    out = rs.lora(wide(X), wide(A), wide(B), ids.cuda(), scale=scale.cuda(), base=Yb, out=Yb)
    assert out is Yb
    assert_within(Yb, ref, rounded(ref, err, dt))
    # One adapter, no ids, no base; then the same expanded to a stack (stride 0).
    (ref, _), (err, _) = lora64(X, A[:1], B[:1], torch.zeros(M, dtype=torch.int32), torch.tensor([0.75]), None)
    got = rs.lora(X.cuda(), A[:1].cuda(), B[:1].cuda(), scale=0.75)
    assert_within(got, ref, rounded(ref, err, dt))
    got2 = rs.lora(X.cuda(), A[:1].cuda().expand(L, R, K), B[:1].cuda().expand(L, N, R),
                   torch.full((M,), 2, device="cuda"), scale=0.75)
    assert_within(got2, ref, rounded(ref, err, dt))
    # The gradient of X in place of the one through the projection.
    dY = torch.randn((M, N), generator=gen).to(dt)
    H = torch.randn((M, R), generator=gen)
    xb = torch.randn((M, K), generator=gen).to(dt)
    dX = wide(xb)
    refs, errs = lora_backward64(dY, X, A, B, H, ids, scale, xb)
    got = rs.lora_backward(wide(dY), wide(X), wide(A), wide(B), H.cuda(), ids.cuda(), scale=scale.cuda(), base=dX, dX=dX)
    for g, r, e in zip(got, refs, errs):
        assert_within(g, r, rounded(r, e, dt))
    assert rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), H.cuda(), ids.cuda(), need_dx=False)[0] is None
    assert rs.lora_backward(dY.cuda(), X.cuda(), A.cuda(), B.cuda(), H.cuda(), ids.cuda(), need_dw=False)[1:] == (None, None)


@pytest.mark.parametrize("M", [3, 200])
def test_ids_outside_mean_no_adapter(M):
    gen = torch.Generator().manual_seed(M)
    X, A, B, _, scale, base = make(gen, M, 20, 24, 4, 3, torch.float32)
    ids = torch.randint(-3, 6, (M,), generator=gen, dtype=torch.int64)
    ids[0], ids[1], ids[2] = -2 ** 63, 2 ** 63 - 1, 1 << 32   # not adapter 0 of 32 bits
    (ref, h), (err, eh) = lora64(X, A, B, ids, scale, base)
    Y, H = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=base.cuda(), save=True)
    assert_within(Y, ref, rounded(ref, err, torch.float32))
    assert_within(H, h, eh)
    none = ~((ids >= 0) & (ids < 3))
    assert torch.equal(Y.cpu()[none], base[none]) and not H.cpu()[none].any()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M", [4, 150])
def test_other_rows_values_do_not_spread(M, t):
    """Infinities and NaN in one row, in an adapter that no row has, and in the
    rows without adapter stay where they are; padding of the rank adds none."""
    gen = torch.Generator().manual_seed(M)
    N, K, R, L, dt = 50, 40, 5, 4, TYPES[t]
    X, A, B, ids, scale, base = make(gen, M, N, K, R, L, dt)
    ids[ids == 2] = 1
    ids[0], ids[1], ids[2], ids[3] = 0, 0, 1, -1
    (ref, h), (err, eh) = lora64(X, A, B, ids, scale, base)
    bad = X.clone()
    bad[0, 3], bad[3, 0] = float("inf"), float("nan")
    A[2], B[2] = float("nan"), float("inf")
    scale[2] = float("nan")
    Y, H = rs.lora(bad.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=base.cuda(), save=True)
    assert_within(Y[1:], ref[1:], rounded(ref, err, dt)[1:])
    assert_within(H[1:], h[1:], eh[1:])
    assert not torch.isfinite(H[0]).any() and not torch.isfinite(Y[0]).any()
    # Backward: the NaN row has no adapter, so only its own dX could hold one.
    dY = torch.randn((M, N), generator=gen).to(dt)
    X2 = X.clone()
    X2[3] = float("nan")
    dY2 = dY.clone()
    dY2[3] = float("inf")
    Hn = torch.randn((M, R), generator=gen)
    Hb = Hn.clone()
    Hb[3] = float("nan")
    clean = [v.clone() for v in (A, B)]
    clean[0][2], clean[1][2] = 0, 0
    scale[2] = 1.0
    refs, errs = lora_backward64(dY, X, *clean, Hn, ids, scale, None)
    got = rs.lora_backward(dY2.cuda(), X2.cuda(), A.cuda(), B.cuda(), Hb.cuda(), ids.cuda(), scale=scale.cuda())
    for g, r, e in zip(got, refs, errs):
        assert_within(g, r, rounded(r, e, dt))


def test_empty_sizes():
    f = dict(device="cuda", dtype=torch.float32)
    z = lambda *s: torch.zeros(s, **f)
    ones = torch.ones((3, 5), **f)
    ids = torch.zeros(3, device="cuda", dtype=torch.int32)
    assert torch.equal(rs.lora(z(3, 0), z(1, 2, 0), z(1, 5, 2), ids, base=ones), ones)      # K = 0
    Y, H = rs.lora(torch.ones((3, 4), **f), torch.ones((1, 2, 4), **f), z(1, 0, 2), ids, save=True)  # N = 0
    assert Y.shape == (3, 0) and bool((H == 4).all())
    assert rs.lora(z(0, 4), z(1, 2, 4), z(1, 5, 2)).shape == (0, 5)
    dX, dA, dB = rs.lora_backward(z(0, 5), z(0, 4), torch.ones((2, 2, 4), **f), z(2, 5, 2), z(0, 2), ids[:0])
    assert dX.shape == (0, 4) and dA.shape == (2, 2, 4) and not dA.any() and not dB.any()
    dX, dA, dB = rs.lora_backward(z(3, 0), torch.ones((3, 4), **f), z(1, 2, 4), z(1, 0, 2), z(3, 2), ids,
                                  base=torch.ones((3, 4), **f))                               # N = 0
    assert bool((dX == 1).all()) and not dA.any() and dB.shape == (1, 0, 2)
    dX, dA, dB = rs.lora_backward(ones, z(3, 0), z(1, 2, 0), z(1, 5, 2), torch.ones((3, 2), **f), ids)  # K = 0
    assert dX.shape == (3, 0) and dA.shape == (1, 2, 0) and bool((dB == 3).all())


@pytest.mark.parametrize("M", [5, 400])
def test_same_bits_from_run_to_run_and_in_a_graph(M):
    """Replays of a captured forward and backward pass, with eager calls of
    other sizes between them, against the eager results, bit for bit."""
    gen = torch.Generator().manual_seed(M)
    N, K, R, L = 136, 264, 16, 5
    X, A, B, ids, scale, base = (v.cuda() for v in make(gen, M, N, K, R, L, torch.bfloat16))
    dY = torch.randn((M, N), generator=gen).bfloat16().cuda()

    def both():
        Y, H = rs.lora(X, A, B, ids, scale=scale, base=base, save=True)
        return (Y, H, *rs.lora_backward(dY, X, A, B, H, ids, scale=scale))

    want = [t.clone() for t in both()]
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        for t in got:
            t.fill_(float("nan"))
        rs.lora(X[: 2 + i], A, B, ids[: 2 + i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), i
    # Other ids and values in the same buffers: the graph follows them.
    ids.copy_(torch.randint(-1, L, (M,), generator=gen, dtype=torch.int32))
    X.copy_(torch.randn((M, K), generator=gen))
    want = [t.clone() for t in both()]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams():
    gen = torch.Generator().manual_seed(9)
    sets = [tuple(v.cuda() for v in make(gen, M, 256, 512, 16, 4, torch.float16)) for M in (300, 700)]
    want = [rs.lora(X, A, B, ids, scale=scale, base=base) for X, A, B, ids, scale, base in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            X, A, B, ids, scale, base = sets[i]
            with torch.cuda.stream(st):
                got[i].append(rs.lora(X, A, B, ids, scale=scale, base=base))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], g) for g in got[i])


def test_beside_a_4bit_projection_and_trained():
    """As they are used: a served projection with 4-bit weights and adapters
    beside it, the adapters' gradients, and their orthogonalised updates."""
    gen = torch.Generator().manual_seed(21)
    M, N, K, R, L, group, dt = 96, 192, 256, 16, 3, 64, torch.bfloat16
    X, A, B, ids, scale, _ = make(gen, M, N, K, R, L, dt)
    w, s, z = q4_make(gen, N, K, group, dt, True)
    Y0 = rs.q4_matmul(X.cuda(), w, s, z, group=group)
    Y, H = rs.lora(X.cuda(), A.cuda(), B.cuda(), ids.cuda(), scale=scale.cuda(), base=Y0, save=True)
    p, ep = q4_64(X, w, s, z, group)
    ep = rounded(p, ep, dt)  # the projection is stored in the type
    (d, _), (ed, _) = lora64(X, A, B, ids, scale, None)
    ref = p + d
    assert_within(Y, ref, rounded(ref, ep + ed + 2.0 ** -23 * ref.abs(), dt))
    dY = torch.randn((M, N), generator=gen).to(dt).cuda()
    _, dA, dB = rs.lora_backward(dY, X.cuda(), A.cuda(), B.cuda(), H, ids.cuda(), scale=scale.cuda(), need_dx=False)
    for g in (dA, dB):
        O = rs.orthogonalize(g.float())
        sv = torch.linalg.svdvals(O.cpu().double())
        # Five steps of the default coefficients send singular values from
        # 2e-3 of the norm up into 0.6 .. 1.25.
        keep = torch.linalg.svdvals(g.cpu().double()) / g.cpu().double().norm(dim=(1, 2), keepdim=True)[:, 0] > 4e-3
        assert bool((sv[keep] > 0.6).all()) and bool((sv[keep] < 1.25).all())


def test_refusals():
    f = dict(device="cuda")
    X, A, B = torch.zeros((4, 6), **f), torch.zeros((2, 3, 6), **f), torch.zeros((2, 5, 3), **f)
    ids = torch.zeros(4, dtype=torch.int32, **f)
    for bad in (X, A[0], torch.zeros((2, 3, 7), **f)):
        with pytest.raises(ValueError, match="A"):
            rs.lora(X, bad, B, ids)
    for bad in (B[0], torch.zeros((2, 5, 4), **f), torch.zeros((3, 5, 3), **f), B.cpu()):
        with pytest.raises(ValueError, match="B"):
            rs.lora(X, A, bad, ids)
    with pytest.raises(TypeError, match="A"):
        rs.lora(X, A.half(), B, ids)
    with pytest.raises(TypeError, match="B"):
        rs.lora(X, A, None, ids)
    with pytest.raises(ValueError, match="ids"):
        rs.lora(X, A, B)
    for bad in (ids[:3], ids.cpu(), ids[None], torch.zeros(8, dtype=torch.int32, **f)[::2]):
        with pytest.raises(ValueError, match="ids"):
            rs.lora(X, A, B, bad)
    for bad in (ids.float(), [0, 0, 0, 0]):
        with pytest.raises(TypeError, match="ids"):
            rs.lora(X, A, B, bad)
    with pytest.raises(ValueError, match="scale"):
        rs.lora(X, A, B, ids, scale=torch.ones(3, **f))
    with pytest.raises(TypeError, match="scale"):
        rs.lora(X, A, B, ids, scale=torch.ones(2, dtype=torch.float64, **f))
    with pytest.raises(ValueError, match="base"):
        rs.lora(X, A, B, ids, base=torch.zeros((4, 6), **f))
    with pytest.raises(ValueError, match="out"):
        rs.lora(X, A, B, ids, out=torch.zeros((3, 5), **f))
    with pytest.raises(ValueError, match="save"):
        rs.lora(X, A, B, ids, save=torch.zeros((4, 4), **f))
    with pytest.raises(rs.SgemmError, match="ALIAS"):
        rs.lora(torch.zeros((4, 5), **f), torch.zeros((2, 3, 5), **f), B, ids, out=X[:, :5], base=X[:, 1:6])
    with pytest.raises(rs.SgemmError, match="DIM"):
        rs.lora(X, torch.zeros((1, 300, 6), **f), torch.zeros((1, 5, 300), **f))
    dY, H = torch.zeros((4, 5), **f), torch.zeros((4, 3), **f)
    with pytest.raises(ValueError, match="H"):
        rs.lora_backward(dY, X, A, B, dY, ids)
    with pytest.raises(TypeError, match="H"):
        rs.lora_backward(dY, X, A, B, H.half(), ids)
    with pytest.raises(ValueError, match="dY"):
        rs.lora_backward(dY[:3], X, A, B, H, ids)
    for bad in ((A.clone(),), (A.clone(), None), A.clone()):
        with pytest.raises(ValueError, match="dW"):
            rs.lora_backward(dY, X, A, B, H, ids, dW=bad)
    with pytest.raises(rs.SgemmError, match="ALIAS"):
        rs.lora_backward(dY, X, A, B, H, ids, dW=(A, B.clone()))


@pytest.mark.parametrize("M", [1, 40])
def test_the_largest_floats_are_finite(M):
    # dH is 3.402e38, below the largest float (3.4028e38), in a rank whose A is zero:
    # its power of two must bring it into float16's range, or zero times inf is NaN.
    dY = torch.ones((M, 1), dtype=torch.float16, device="cuda")
    B = torch.tensor([[[1.0, 0.0, 0.0, 0.0]]], dtype=torch.float16, device="cuda")
    A = torch.zeros((1, 4, 70), dtype=torch.float16, device="cuda")
    A[:, 1:] = 1.0
    X = torch.ones((M, 70), dtype=torch.float16, device="cuda")
    base = torch.randn((M, 70), device="cuda").half()
    dX, dA, dB = rs.lora_backward(dY, X, A, B, torch.zeros((M, 4), device="cuda"), scale=3.402e38, base=base,
                                  need_dw=False)
    assert dA is None and dB is None and torch.equal(dX, base)

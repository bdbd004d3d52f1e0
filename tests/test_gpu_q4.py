"""Products with 4-bit weights on the GPU, against the 64-bit sum within
counted float bounds."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.ff_util import (ACTS, LIPSCHITZ, TYPES, U, Guarded, act64, act_err, assert_within, q4_64,
                           q4_int, q4_make, rounded)

pytestmark = pytest.mark.gpu
TINY_F32 = 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


def glu_bound(act, g, eg, u, eu, dtype):
    a, _ = act64(act, g)
    h = a * u
    eh = (LIPSCHITZ * eg + act_err(g)) * (u.abs() + eu) + a.abs() * eu + 2 * U * h.abs()
    return h, rounded(h, eh, dtype)


# (M, N, K, group): one row to many, odd everywhere, K below a group, a last
# group cut short, K not a whole byte, per-row scales.
SHAPES = [(1, 64, 128, 32), (1, 1, 1, 32), (1, 17, 31, 32), (1, 100, 4096, 128), (1, 33, 1000, 64),
          (2, 48, 255, 64), (3, 16, 96, 128), (4, 257, 512, 32), (5, 31, 2047, 64), (8, 64, 1024, 4096),
          (9, 40, 300, 128), (15, 129, 384, 64), (16, 16, 640, 32), (17, 130, 200, 32),
          (31, 65, 777, 128), (33, 64, 256, 64), (64, 320, 512, 128), (65, 33, 160, 32),
          (100, 100, 1025, 256), (128, 256, 448, 64), (130, 300, 320, 128), (257, 513, 96, 32),
          (300, 70, 2000, 128), (512, 512, 192, 64)]


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product(shape, x):
    M, N, K, group = shape
    i = SHAPES.index(shape) + list(TYPES).index(x)
    stype, zeros = list(TYPES.values())[i % 3], i % 2 == 0
    gen = torch.Generator().manual_seed(i)
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    w, s, z = q4_make(gen, N, K, group, stype, zeros)
    Y = Guarded(M, N, TYPES[x], gap=(0, 1, 8)[i % 3])
    rs.q4_matmul(X.cuda(), w, s, z, group=group, out=Y.view)
    ref, err = q4_64(X, w, s, z, group)
    assert_within(Y.view, ref, rounded(ref, err, TYPES[x]))
    assert Y.intact()


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("shape", SHAPES[1::2], ids=lambda s: "x".join(map(str, s)))
def test_gated(shape, x):
    M, N, K, group = shape
    i = SHAPES.index(shape) + list(TYPES).index(x)
    act, stype, zeros = ACTS[i % 5], list(TYPES.values())[i % 3], i % 2 == 0
    gen = torch.Generator().manual_seed(i)
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    gate, up = q4_make(gen, N, K, group, stype, zeros), q4_make(gen, N, K, group, stype, zeros)
    H = Guarded(M, N, TYPES[x], gap=(1, 0, 8)[i % 3])
    rs.q4_glu(X.cuda(), gate[0], gate[1], up[0], up[1], gate[2], up[2], group=group, act=act,
              out=H.view)
    g, eg = q4_64(X, *gate, group)
    u, eu = q4_64(X, *up, group)
    assert_within(H.view, *glu_bound(act, g, eg, u, eu, TYPES[x]))
    assert H.intact()


# Rows by 8190 columns that take each tile of the rule in turn (32 x 64, 32 x
# 128, 64 x 128, the largest), with K of whole and cut units.
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("M", [61, 125, 250, 1000])
def test_every_tile(M, x, group):
    gen = torch.Generator().manual_seed(M)
    N, K = 8190, {32: 384, 64: 290, 128: 135}[group]
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    stype = TYPES[x] if group != 64 else torch.float32
    w, s, z = q4_make(gen, N, K, group, stype, group != 32)
    Y = Guarded(M, N, TYPES[x], gap=2 if group == 64 else 0)
    rs.q4_matmul(X.cuda(), w, s, z, group=group, out=Y.view)
    ref, err = q4_64(X, w, s, z, group)
    assert_within(Y.view, ref, rounded(ref, err, TYPES[x]))
    assert Y.intact()


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("M", [61, 125, 250, 500])
def test_every_gated_tile(M, x):
    gen = torch.Generator().manual_seed(M)
    group = 32 << (M // 125 % 3)
    N, K, stype = 8190, 300, torch.float32 if M == 125 else torch.bfloat16
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    gate, up = (q4_make(gen, N, K, group, stype, M != 61) for _ in range(2))
    H = Guarded(M, N, TYPES[x], gap=1)
    rs.q4_glu(X.cuda(), gate[0], gate[1], up[0], up[1], gate[2], up[2], group=group, act="gelu_tanh",
              out=H.view)
    g, eg = q4_64(X, *gate, group)
    u, eu = q4_64(X, *up, group)
    assert_within(H.view, *glu_bound("gelu_tanh", g, eg, u, eu, TYPES[x]))
    assert H.intact()


@pytest.mark.parametrize("st", TYPES)
@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("M", [1, 6, 40, 200])
def test_every_pair_of_types(M, x, st):
    gen = torch.Generator().manual_seed(M)
    N, K, group = 96, 320, 64
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    w, s, z = q4_make(gen, N, K, group, TYPES[st], True)
    Y = rs.q4_matmul(X.cuda(), w, s, z, group=group)
    ref, err = q4_64(X, w, s, z, group)
    assert_within(Y, ref, rounded(ref, err, TYPES[x]))


@pytest.mark.parametrize("M", [1, 4, 16, 48, 160])
def test_every_float_bit_counts(M):
    """Rows with one 24-bit value each: the product is that value times q - z.
    The value is the sum of three parts of 8 bits; the first part's product
    (12 bits) is exact, adding each of the other two rounds once, and scaling
    by 1 and adding zeros is exact: two roundings, each at most half a unit,
    u = 2^-24 of the value then held, which is at most |v (q - z)| (1 + u).
    A part left out would be off by 2^-8 or 2^-16 of it."""
    gen = torch.Generator().manual_seed(M)
    N, K = 64, 192
    X = torch.zeros((M, K))
    v = torch.randint(1 << 23, 1 << 24, (M,), generator=gen).float() * 2.0 ** -20
    at = torch.randint(0, K, (M,), generator=gen)
    X[torch.arange(M), at] = v
    w, s, z = q4_make(gen, N, K, 32, torch.float32, True)
    s.fill_(1.0)
    Y = rs.q4_matmul(X.cuda(), w, s, z, group=32)
    ref = X.double() @ q4_int(w, z, K, 32).t()
    assert_within(Y, ref, 2 * U * (1 + U) * ref.abs())


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("M", [1, 3, 16, 33, 140])
def test_integers_are_exact(M, x):
    # Small integers and power-of-two scales: every sum is an integer below
    # 2^24 times a power of two; the result rounds once.
    gen = torch.Generator().manual_seed(M)
    N, K, group = 80, 544, 32
    X = torch.randint(-4, 5, (M, K), generator=gen).to(TYPES[x])
    w, s, z = q4_make(gen, N, K, group, torch.float32, True)
    s = (2.0 ** torch.randint(-3, 2, s.shape, generator=gen)).cuda()
    Y = rs.q4_matmul(X.cuda(), w, s.float(), z, group=group)
    ref, _ = q4_64(X, w, s, z, group)
    assert torch.equal(Y.cpu(), ref.to(TYPES[x]))


@pytest.mark.parametrize("M", [1, 20, 140])
def test_half_precision_subnormals(M):
    """float16 X below its normal range counts in full: integers times 2^-24,
    its smallest step, with scales that bring the sums back."""
    gen = torch.Generator().manual_seed(M)
    N, K, group = 64, 256, 64
    X = (torch.randint(-40, 41, (M, K), generator=gen).double() * 2.0 ** -24).to(torch.float16)
    w, s, z = q4_make(gen, N, K, group, torch.float32, True)
    s.fill_(2.0 ** 20)
    Y = rs.q4_matmul(X.cuda(), w, s, z, group=group)
    ref, _ = q4_64(X, w, s, z, group)
    assert torch.equal(Y.cpu(), ref.to(torch.float16))


@pytest.mark.parametrize("M", [1, 5, 40, 150])
def test_unaligned_views(M):
    """Odd row strides and start addresses of every operand."""
    gen = torch.Generator().manual_seed(M)
    N, K, group = 70, 333, 32
    groups = -(-K // group)
    for x in TYPES:
        X = torch.randn((M, K), generator=gen).to(TYPES[x])
        w, s, z = q4_make(gen, N, K, group, torch.float16, True)

        def shifted(t, gap, dtype):
            # NaN or 255 around the view: nothing outside it may count.
            fill = float("nan") if dtype.is_floating_point else 255
            b = torch.full((t.shape[0] * (t.shape[1] + gap) + 1,), fill, dtype=dtype, device="cuda")
            v = torch.as_strided(b, t.shape, (t.shape[1] + gap, 1), 1)
            v.copy_(t)
            return v

        Xd, wd = shifted(X, 3, TYPES[x]), shifted(w, 5, torch.uint8)
        sd, zd = shifted(s, 1, torch.float16), shifted(z, 2, torch.uint8)
        Y = rs.q4_matmul(Xd, wd, sd, zd, group=group)
        ref, err = q4_64(X, w, s, z, group)
        assert_within(Y, ref, rounded(ref, err, TYPES[x]), x)
        # The same values on whole rows give the same bits.
        assert torch.equal(Y, rs.q4_matmul(X.cuda(), w, s, z, group=group))


@pytest.mark.parametrize("M", [1, 7, 20, 130])
def test_non_finite_values(M):
    """A NaN or infinity in X reaches its own row only, an infinity with its
    sign (against a row without q == z), and a NaN scale its own column."""
    gen = torch.Generator().manual_seed(3)
    N, K, group = 48, 256, 64
    X = torch.randn((M, K), generator=gen)
    w, s, z = q4_make(gen, N, K, group, torch.float32, False)
    w |= 0x11  # q odd: never 8
    for x in TYPES:
        Xt = X.to(TYPES[x])
        base = rs.q4_matmul(Xt.cuda(), w, s, z, group=group)
        X2 = Xt.clone()
        X2[M // 2, 70] = float("inf")
        got = rs.q4_matmul(X2.cuda(), w, s, z, group=group)
        sign = torch.sign(q4_int(w, z, K, group)[:, 70])
        assert torch.equal(got[M // 2].cpu().double(), sign * float("inf")), x
        X2[M // 2, 70] = float("nan")
        got = rs.q4_matmul(X2.cuda(), w, s, z, group=group)
        assert torch.isnan(got[M // 2]).all()
        others = torch.arange(M) != M // 2
        assert torch.equal(got[others], base[others])
        s2 = s.clone()
        s2[9, 2] = float("nan")
        got = rs.q4_matmul(Xt.cuda(), w, s2, z, group=group)
        cols = torch.arange(N) != 9
        assert torch.isnan(got[:, 9]).all() and torch.equal(got[:, cols], base[:, cols])


@pytest.mark.parametrize("M", [1, 5, 40])
def test_infinite_last_scale(M):
    """An infinite scale gives infinities of its group's sign, not NaN, also
    where the row ends inside a step of the kernels (K = 96 + 32)."""
    for K in (96, 97, 160, 288):
        group = 32
        groups = -(-K // group)
        X = torch.ones((M, K))
        w = torch.full((16, (K + 1) // 2), 0x99, dtype=torch.uint8, device="cuda")  # q - z = 1
        s = torch.ones((16, groups), device="cuda")
        s[3, -1] = float("inf")
        for x in TYPES:
            Y = rs.q4_matmul(X.to(TYPES[x]).cuda(), w, s, group=group)
            assert torch.isinf(Y[:, 3]).all() and (Y[:, 3] > 0).all(), (K, x)
            assert (Y[:, 2].float() == K).all()


@pytest.mark.parametrize("M", [1, 9, 70])
@pytest.mark.parametrize("group", [1 << 31, 1 << 40, 1 << 62])
def test_one_group_of_any_length(M, group):
    gen = torch.Generator().manual_seed(M)
    N, K = 40, 700
    X = torch.randn((M, K), generator=gen)
    w, s, z = q4_make(gen, N, K, 1024, torch.float32, True)
    Y = rs.q4_matmul(X.cuda(), w, s, z, group=group)
    assert torch.equal(Y, rs.q4_matmul(X.cuda(), w, s, z, group=1024))
    ref, err = q4_64(X, w, s, z, 1024)
    assert_within(Y, ref, err + TINY_F32)


def test_nan_payload_of_low_bits():
    # A NaN whose set bits are all in the low half of the word stays a NaN.
    X = torch.zeros((2, 64))
    X[0, 5] = torch.tensor([0x7F800001], dtype=torch.int32).view(torch.float32)[0]
    gen = torch.Generator().manual_seed(1)
    w, s, z = q4_make(gen, 32, 64, 32, torch.float32, False)
    Y = rs.q4_matmul(X.cuda(), w | 0x11, s, z, group=32)
    assert torch.isnan(Y[0]).all() and not torch.isnan(Y[1]).any()


def test_empty_sizes():
    gen = torch.Generator().manual_seed(1)
    w, s, z = q4_make(gen, 8, 64, 32, torch.float16, False)
    X = torch.randn((3, 64), device="cuda")
    assert rs.q4_matmul(X[:0], w, s, group=32).shape == (0, 8)
    assert rs.q4_matmul(X, w[:0], s[:0], group=32).shape == (3, 0)
    Y = rs.q4_matmul(X[:, :0].contiguous(), w[:, :0].contiguous(), s[:, :0].contiguous(), group=32)
    assert Y.shape == (3, 8) and not Y.any()
    H = rs.q4_glu(X[:, :0].contiguous(), w[:, :0].contiguous(), s[:, :0].contiguous(),
                  w[:, :0].contiguous(), s[:, :0].contiguous(), group=32, act="sigmoid")
    assert H.shape == (3, 8) and not H.any()


@pytest.mark.parametrize("M", [1, 12, 96])
def test_capture_and_replay(M):
    gen = torch.Generator().manual_seed(M)
    N, K, group = 256, 512, 128
    X = torch.randn((M, K), device="cuda", dtype=torch.bfloat16)
    gate, up = (q4_make(gen, N, K, group, torch.bfloat16, False) for _ in range(2))
    down = q4_make(gen, 128, N, group, torch.bfloat16, False)
    H = torch.empty((M, N), device="cuda", dtype=torch.bfloat16)
    Y = torch.empty((M, 128), device="cuda", dtype=torch.bfloat16)

    def block():
        rs.q4_glu(X, gate[0], gate[1], up[0], up[1], group=group, out=H)
        rs.q4_matmul(H, down[0], down[1], group=group, out=Y)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for _ in range(3):
        X.copy_(torch.randn_like(X))
        Y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = (H.clone(), Y.clone())
        block()
        torch.cuda.synchronize()
        assert torch.equal(got[0], H) and torch.equal(got[1], Y)
        g, eg = q4_64(X, *gate, group)
        u, eu = q4_64(X, *up, group)
        assert_within(H, *glu_bound("silu", g, eg, u, eu, torch.bfloat16))
        ref, err = q4_64(H, *down, group)
        assert_within(Y, ref, rounded(ref, err, torch.bfloat16))


def test_two_streams_at_once():
    gen = torch.Generator().manual_seed(5)
    w, s, z = q4_make(gen, 512, 1024, 64, torch.float16, True)
    Xs = [torch.randn((m, 1024), device="cuda") for m in (1, 200)]
    want = [rs.q4_matmul(X, w, s, z, group=64) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    outs = []
    for st, X in zip(streams, Xs):
        with torch.cuda.stream(st):
            outs.append([rs.q4_matmul(X, w, s, z, group=64) for _ in range(4)])
    torch.cuda.synchronize()
    for o, r in zip(outs, want):
        assert all(torch.equal(t, r) for t in o)


def test_a_block_trained_then_served():
    """The four operators as they are used: a float step of the block with its
    gradients, then the same weights quantised and served."""
    gen = torch.Generator().manual_seed(9)
    M, K, F, group = 48, 128, 192, 64
    X = torch.randn((M, K), generator=gen).cuda()
    W = (torch.randn((2 * F, K), generator=gen) / K ** 0.5).cuda()
    H, G, Up = rs.glu(X, W[:F], W[F:], transw=True, save=True)
    dX, dWg, dWu = rs.glu_backward(torch.ones_like(H), X, W[:F], W[F:], G, Up, transw=True)
    W = W - 0.01 * torch.cat([dWg, dWu])
    g3 = W.view(2 * F, K // group, group)
    s = g3.abs().amax(2) / 7
    q = (torch.round(g3 / s[..., None]) + 8).clamp(0, 15).to(torch.uint8).view(2 * F, K)
    packed = q[:, 0::2] | (q[:, 1::2] << 4)
    Hq = rs.q4_glu(X, packed[:F], s[:F], packed[F:], s[F:], group=group)
    Wq = ((q.float() - 8).view(2 * F, K // group, group) * s[..., None]).view(2 * F, K)
    want = rs.glu(X, Wq[:F].contiguous(), Wq[F:].contiguous(), transw=True)
    # Two float routes to the same value: each within its own bound.
    g, eg = q4_64(X, packed[:F], s[:F], None, group)
    u, eu = q4_64(X, packed[F:], s[F:], None, group)
    h, eh = glu_bound("silu", g, eg, u, eu, torch.float32)
    assert_within(Hq, h, eh, "served")
    # The float weights are products rounded once more: K more roundings.
    assert_within(want, h, eh * 4 * K, "float")


def test_refusals():
    gen = torch.Generator().manual_seed(1)
    N, K, group = 24, 96, 32
    w, s, z = q4_make(gen, N, K, group, torch.float16, True)
    X = torch.randn((3, K), device="cuda")
    for bad in (48, 16, 0, -32):
        with pytest.raises(ValueError, match="power of two"):
            rs.q4_matmul(X, w, s, z, group=bad)
    with pytest.raises(ValueError, match="shape"):
        rs.q4_matmul(X, w, s, z, group=64)
    with pytest.raises(ValueError, match="shape"):
        rs.q4_matmul(X[:, :-2].contiguous(), w, s, z, group=group)
    with pytest.raises(TypeError):
        rs.q4_matmul(X, w.to(torch.int8), s, z, group=group)
    with pytest.raises(TypeError):
        rs.q4_matmul(X.double(), w, s, z, group=group)
    with pytest.raises(TypeError):
        rs.q4_matmul(X, w, s.double(), z, group=group)
    with pytest.raises(TypeError):
        rs.q4_matmul(X, w, s, z, group=group, out=torch.empty((3, N), device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        rs.q4_matmul(X, w.cpu(), s, z, group=group)
    with pytest.raises(TypeError, match="scales"):
        rs.q4_glu(X, w, s, w, s.float(), group=group)
    with pytest.raises(ValueError, match="activation"):
        rs.q4_glu(X, w, s, w, s, group=group, act="tanh")
    square = q4_make(gen, K, K, group, torch.float16, False)
    with pytest.raises(rs.SgemmError) as e:
        rs.q4_matmul(X, square[0], square[1], group=group, out=X)
    assert e.value.status == 5  # SGEMM_ERR_ALIAS


def test_one_weight_as_gate_and_up():
    gen = torch.Generator().manual_seed(2)
    N, K, group = 50, 130, 64
    w, s, z = q4_make(gen, N, K, group, torch.bfloat16, True)
    for M in (2, 30):
        X = torch.randn((M, K), generator=gen)
        H = rs.q4_glu(X.cuda(), w, s, w, s, z, z, group=group, act="relu")
        g, eg = q4_64(X, w, s, z, group)
        assert_within(H, *glu_bound("relu", g, eg, g, eg, torch.float32))


def test_offsets_past_32_bits():
    """More than 2^31 results, rows from both ends and the middle checked."""
    gen = torch.Generator().manual_seed(4)
    M, N, K, group = 66000, 33000, 40, 32
    X = torch.randn((M, K), generator=gen).to(torch.float16)
    w, s, z = q4_make(gen, N, K, group, torch.float16, False)
    Y = rs.q4_matmul(X.cuda(), w, s, group=group)
    rows = torch.tensor([0, 1, 32767, 40001, M - 2, M - 1])
    ref, err = q4_64(X[rows], w, s, z, group)
    assert_within(Y[rows.cuda()], ref, rounded(ref, err, torch.float16))

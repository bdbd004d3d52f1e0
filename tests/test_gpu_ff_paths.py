"""The gated feed-forward block and the 4-bit products on the paths that only
large strides, large outputs or long rows take."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.ff_util import (ACTS, LIPSCHITZ, TYPES, U, Guarded, act64, act_err, assert_within, glu64,
                           glu_backward64, q4_64, q4_int, q4_make, rounded)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


def strided(t, ld):
    """t with rows ld apart in a buffer of its own; what lies between is NaN
    (255 for bytes)."""
    fill = float("nan") if t.dtype.is_floating_point else 255
    buf = torch.full(((t.shape[0] - 1) * ld + t.shape[1],), fill, dtype=t.dtype, device="cuda")
    v = torch.as_strided(buf, t.shape, (ld, 1))
    v.copy_(t)
    return v


# Rows too long for 32-bit offsets within a tile: 4 Mi elements of X, 8 MiB of
# packed weights.
LONG_X, LONG_W = 1 << 22, 1 << 23


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("shape", [(1, 5, 70, 32), (3, 4, 257, 64), (2, 7, 1000, 128), (2, 3, 333, 512)],
                         ids=lambda s: "x".join(map(str, s)))
def test_4bit_rows_of_any_stride(shape, x):
    M, N, K, group = shape
    gen = torch.Generator().manual_seed(N)
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    w, s, z = q4_make(gen, N, K, group, TYPES[x], N % 2 == 0)
    ref, err = q4_64(X, w, s, z, group)
    wide_w = strided(w, LONG_W)
    Y = Guarded(M, N, TYPES[x], gap=2)
    rs.q4_matmul(X.cuda(), wide_w, s, z, group=group, out=Y.view)
    assert_within(Y.view, ref, rounded(ref, err, TYPES[x]), "long rows of weights")
    assert Y.intact()
    if M > 1:
        got = rs.q4_matmul(strided(X, LONG_X), w, s, z, group=group)
        assert_within(got, ref, rounded(ref, err, TYPES[x]), "long rows of X")
    up = q4_make(gen, N, K, group, TYPES[x], N % 2 == 0)
    u, eu = q4_64(X, *up, group)
    H = rs.q4_glu(X.cuda(), wide_w, s, strided(up[0], LONG_W), up[1], z, up[2], group=group, act="gelu")
    h = act64("gelu", ref)[0] * u
    eh = (LIPSCHITZ * err + act_err(ref)) * (u.abs() + eu) + act64("gelu", ref)[0].abs() * eu + 2 * U * h.abs()
    assert_within(H, h, rounded(h, eh, TYPES[x]), "gated")


@pytest.mark.parametrize("K", [96, 97, 288])
def test_4bit_infinite_scale_of_any_stride(K):
    """An infinite scale gives infinities of its group's sign, as on rows of
    ordinary strides, though the group is shared out over lanes."""
    group = 32
    X = torch.ones((2, K), device="cuda")
    X[1] = -1.0
    w = strided(torch.full((3, (K + 1) // 2), 0x99, dtype=torch.uint8, device="cuda"), LONG_W)  # q - z = 1
    s = torch.ones((3, -(-K // group)), device="cuda")
    s[1, 1] = float("inf")
    Y = rs.q4_matmul(X, w, s, group=group)
    assert Y[0, 1] == float("inf") and Y[1, 1] == -float("inf")
    assert (Y[0, [0, 2]] == K).all() and (Y[1, [0, 2]] == -K).all()


@pytest.mark.parametrize("save", [False, True])
def test_gated_rows_of_any_stride(save):
    """Rows of X of 4.2 Mi floats and rows of K x F weights of 17.4 Mi, past
    the matrix kernel's 32-bit offsets; and the products of the backward pass
    there."""
    gen = torch.Generator().manual_seed(1)
    M, K, F = 18, 21, 37
    X, W = torch.randn((M, K), generator=gen), torch.randn((2, K, F), generator=gen)
    ref, err = glu64("gelu_tanh", X.double(), W[0].double(), W[1].double())
    def check(X, Wg, Wu, transw):
        H, G, Up = Guarded(M, F, gap=1), Guarded(M, F), Guarded(M, F)
        rs.glu(X, Wg, Wu, act="gelu_tanh", transw=transw, out=H.view,
               save=(G.view, Up.view) if save else False)
        for o, r, e in zip((H, G, Up) if save else (H,), ref, err):
            assert_within(o.view, r, e)
            assert o.intact()
    T = W.transpose(1, 2).contiguous().cuda()
    check(strided(X, 4230000), T[0], T[1], True)
    wide = [strided(W[i, :6], 17400000) for i in range(2)]
    ref, err = glu64("gelu_tanh", X[:, :6].double(), W[0, :6].double(), W[1, :6].double())
    check(X[:, :6].contiguous().cuda(), wide[0], wide[1], False)
    G, Up, dH = (torch.randn((M, F), generator=gen) for _ in range(3))
    want, err = glu_backward64("silu", X[:, :6].double(), W[0, :6].double(), W[1, :6].double(), G.double(),
                               Up.double(), dH.double())
    dX, dWg, dWu = rs.glu_backward(dH.cuda(), X[:, :6].contiguous().cuda(), *wide, G.cuda(), Up.cuda())
    for o, r, e in zip((dX, dWg, dWu), want[2:], err[2:]):
        assert_within(o, r, e)


def test_packed_weights_past_the_offset_limit():
    """K x F weights whose rows just fit the matrix kernel's 32-bit offsets and
    whose packed copies, a few floats longer, do not.  Integers: every
    operation is exact."""
    M, K, F = 300, 32, 17318403
    gen = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randint(-2, 3, (M, K), generator=gen, device="cuda").float()
    Wg, Wu = (torch.randint(-2, 3, (K, F), generator=gen, device="cuda", dtype=torch.float32) for _ in range(2))
    H = rs.glu(X, Wg, Wu, act="relu")
    for c in (slice(0, 300), slice(F // 2, F // 2 + 300), slice(F - 300, F)):
        (h, _, _), _ = glu64("relu", *(t.cpu().double() for t in (X, Wg[:, c], Wu[:, c])))
        assert torch.equal(H[:, c].cpu().double(), h)


# Outputs of many tiles: 512 of 128 x 256 and 928 of them (the last round 13/16
# full), both with rows and columns past the edge or none, K of whole and cut
# slabs, and packed copies; then more than two rounds of 128 x 128 where the
# larger tile would leave a partial round.
TILE_SHAPES = [(2048, 64, 4096), (2040, 84, 4092), (3700, 20, 4096), (2040, 83, 4091),
               (4090, 52, 4220), (4096, 16, 4224), (4090, 51, 4219)]


def plan_tile(M, K, F, transw):
    """The tile of the product the gated form is planned as (aligned or packed)."""
    F, K = -(-F // 4) * 4, -(-K // 4) * 4
    return rs.plan_config(M, 2 * F, K, transb=transw)["tile"]


@pytest.mark.parametrize("transw", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("shape", TILE_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gated_large_tiles(shape, transw):
    M, K, F = shape
    assert plan_tile(M, K, F, transw) == ((128, 256) if M < 4090 else (128, 128))
    i = TILE_SHAPES.index(shape)
    act = ACTS[(i + transw) % len(ACTS)]
    gen = torch.Generator().manual_seed(i)
    X, W = torch.randn((M, K), generator=gen), torch.randn((2, K, F), generator=gen) / K ** 0.5
    D = (W.transpose(1, 2).contiguous() if transw else W).cuda()
    H, G, Up = Guarded(M, F, gap=(0, 3, 4)[i % 3]), Guarded(M, F), Guarded(M, F)
    rs.glu(X.cuda(), D[0], D[1], act=act, transw=transw, out=H.view, save=(G.view, Up.view))
    ref, err = glu64(act, X.double(), W[0].double(), W[1].double())
    for o, r, e, n in zip((H, G, Up), ref, err, "HGU"):
        assert_within(o.view, r, e, n)
        assert o.intact(), n
    assert torch.equal(rs.glu(X.cuda(), D[0], D[1], act=act, transw=transw), H.view)


# (M, N, K, x, group): X and scales staged in one, two or three chunks of K, in
# eight waves (small X) and sixteen (float X of several rows, or small groups of
# a gated pair), the last chunk whole, cut, or the unit that rows end in alone.
CHUNK_SHAPES = [(8, 33, 1700, "f32", 128), (8, 33, 2048, "f32", 128), (8, 40, 2050, "f32", 64),
                (8, 16, 4500, "f32", 32), (3, 33, 8200, "f32", 64), (5, 20, 6144, "f32", 256),
                (8, 33, 4097, "bf16", 128), (8, 17, 9000, "f16", 128), (1, 33, 8193, "f32", 128),
                (1, 20, 40001, "f16", 64), (2, 20, 20000, "bf16", 32), (7, 24, 4223, "f16", 32)]


@pytest.mark.parametrize("shape", CHUNK_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_4bit_long_rows_in_chunks(shape):
    M, N, K, x, group = shape
    i = CHUNK_SHAPES.index(shape)
    gen = torch.Generator().manual_seed(i)
    X = torch.randn((M, K), generator=gen).to(TYPES[x])
    stype, zeros = list(TYPES.values())[i % 3], i % 2 == 0
    gate, up = (q4_make(gen, N, K, group, stype, zeros) for _ in range(2))
    g, eg = q4_64(X, *gate, group)
    u, eu = q4_64(X, *up, group)
    Y = Guarded(M, N, TYPES[x], gap=1)
    rs.q4_matmul(X.cuda(), *gate, group=group, out=Y.view)
    assert_within(Y.view, g, rounded(g, eg, TYPES[x]))
    assert Y.intact()
    for _ in range(3):
        assert torch.equal(rs.q4_matmul(X.cuda(), *gate, group=group), Y.view)
    H = Guarded(M, N, TYPES[x], gap=1)
    rs.q4_glu(X.cuda(), gate[0], gate[1], up[0], up[1], gate[2], up[2], group=group, out=H.view)
    a, _ = act64("silu", g)
    eh = (LIPSCHITZ * eg + act_err(g)) * (u.abs() + eu) + a.abs() * eu + 2 * U * (a * u).abs()
    assert_within(H.view, a * u, rounded(a * u, eh, TYPES[x]), "gated")
    assert H.intact()


def test_workspace_calls_of_two_streams_at_once():
    """Gated calls that pack, split K, or both, and one whose copies pass the
    cached workspace, from two streams together: the smaller calls of one run
    while the other's grow the buffer."""
    def make(M, K, F, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        X = torch.randn((M, K), generator=gen, device="cuda")
        W = torch.randn((2, F, K), generator=gen, device="cuda") / K ** 0.5
        return X, W[0], W[1]
    # Split 32 x 32 tiles; split 64 x 64 tiles; packed (18 MB) and split; packed,
    # 39 MB, 145 MB, and 305 MB (more than the cached buffer holds).
    shapes = [(24, 2052, 130), (64, 4096, 4096), (300, 4097, 401), (700, 2047, 2053),
              (600, 4099, 4101), (2100, 4099, 8200)]
    plans = [rs.plan_config(M, 2 * F, K, transb=True) for M, K, F in shapes]
    assert [(p["packed"], p["splits"] > 1) for p in plans] == [
        (False, True), (False, True), (True, True), (True, False), (True, False), (True, False)]
    sets = [make(*s, i) for i, s in enumerate(shapes)]
    want = [rs.glu(*t, act="gelu", transw=True) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for i in range(len(sets)):
            # The streams go through the shapes in opposite orders.
            for st, j in zip(streams, (i, len(sets) - 1 - i)):
                with torch.cuda.stream(st):
                    outs.append((j, rs.glu(*sets[j], act="gelu", transw=True)))
    torch.cuda.synchronize()
    for j, o in outs:
        assert torch.equal(o, want[j]), shapes[j]
    for j in (0, 2):
        ref, err = glu64("gelu", *(t.cpu().double() for t in (sets[j][0], sets[j][1].t(), sets[j][2].t())))
        assert_within(want[j], ref[0], err[0], shapes[j])


@pytest.mark.parametrize("shape", [(64, 69, 16384), (64, 69, 16390), (192, 35, 6144), (512, 67, 2080),
                                   (448, 130, 2400), (128, 33, 8201), (576, 37, 2048), (256, 21, 16391)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gated_unaligned_full_tiles(shape):
    """Unaligned F x K weights under rows that fill 64-row tiles: as stored
    where the columns fill theirs, or are many, and otherwise as copies."""
    M, K, F = shape
    gen = torch.Generator().manual_seed(F)
    X, W = torch.randn((M, K), generator=gen), torch.randn((2, F, K), generator=gen) / K ** 0.5
    D = W.cuda()
    H, G, Up = Guarded(M, F, gap=1), Guarded(M, F), Guarded(M, F)
    rs.glu(X.cuda(), D[0], D[1], transw=True, out=H.view, save=(G.view, Up.view))
    ref, err = glu64("silu", X.double(), W[0].double().t(), W[1].double().t())
    for o, r, e, n in zip((H, G, Up), ref, err, "HGU"):
        assert_within(o.view, r, e, n)
        assert o.intact(), n


@pytest.mark.parametrize("M", [1, 20, 140])
def test_4bit_smallest_floats(M):
    """float X below 2^-110 counts in steps of 2^-133, cut towards zero, each
    times q - z and the scale; bfloat16 X in full."""
    gen = torch.Generator().manual_seed(M)
    N, K, group = 64, 256, 64
    w, s, z = q4_make(gen, N, K, group, torch.float32, True)
    s.fill_(2.0 ** 100)
    W = q4_int(w, z, K, group).abs().t() * 2.0 ** 100
    for e in (-111, -118, -126, -140):
        X = (torch.randint(1 << 23, 1 << 24, (M, K), generator=gen).double() * 2.0 ** (e - 23)).float()
        Y = rs.q4_matmul(X.cuda(), w, s, z, group=group)
        ref, err = q4_64(X, w, s, z, group)
        assert_within(Y, ref, err + torch.full((M, K), 2.0 ** -133, dtype=torch.float64) @ W, e)
    X = (torch.randint(-40, 41, (M, K), generator=gen).double() * 2.0 ** -133).to(torch.bfloat16)
    Y = rs.q4_matmul(X.cuda(), w, s, z, group=group)
    ref, _ = q4_64(X, w, s, z, group)
    assert torch.equal(Y.cpu(), ref.to(torch.bfloat16))

"""The gated feed-forward block and its gradients on the GPU, against their
64-bit forms within counted float bounds."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.ff_util import (ACTS, Guarded, assert_within, glu64, glu_backward64)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


def operands(M, K, F, transw, seed, kind="halves", integer=False):
    """X, Wg, Wu on the GPU as stored, and as float64 K x F on the host.
    kind: the weights are halves of one buffer, separate, or rows with gaps."""
    gen = torch.Generator().manual_seed(seed)
    def make(*shape):
        if integer:
            return torch.randint(-2, 3, shape, generator=gen).float()
        return torch.randn(shape, generator=gen)
    X = make(M, K)
    W = make(2 * F, K) if transw else make(K, 2 * F)
    if not integer:
        W /= max(K, 1) ** 0.5
    Wg, Wu = (W[:F], W[F:]) if transw else (W[:, :F], W[:, F:])
    host = [X.double()] + [(w.t() if transw else w).double() for w in (Wg, Wu)]
    if kind == "halves":
        D = W.cuda()
        dev = (D[:F], D[F:]) if transw else (D[:, :F], D[:, F:])
    elif kind == "separate":
        dev = (Wg.contiguous().cuda(), Wu.contiguous().cuda())
    else:
        dev = []
        for w in (Wg, Wu):
            g = torch.full((w.shape[0], w.shape[1] + 5), float("nan"), device="cuda")
            g[:, :w.shape[1]] = w.cuda()
            dev.append(g[:, :w.shape[1]])
    return X.cuda(), *dev, host


SHAPES = [(1, 64, 64), (1, 4096, 512), (2, 100, 37), (3, 1, 1), (5, 33, 257), (7, 515, 6151), (8, 2048, 300),
          (9, 16, 31), (9, 600, 7001), (13, 2050, 2052), (16, 512, 128), (16, 1024, 6200), (31, 65, 33), (33, 128, 96), (64, 256, 1024), (65, 127, 129),
          (129, 300, 260), (257, 64, 512), (512, 96, 640), (1000, 130, 700)]


@pytest.mark.parametrize("transw", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, transw):
    M, K, F = shape
    i = SHAPES.index(shape)
    act = ACTS[i % len(ACTS)]
    X, Wg, Wu, host = operands(M, K, F, transw, seed=i, kind=("halves", "separate", "gaps")[i % 3])
    H, G, U = (Guarded(M, F, gap=g) for g in (3, 0, 0))
    U.ld = G.ld
    rs.glu(X, Wg, Wu, act=act, transw=transw, out=H.view, save=(G.view, U.view))
    ref, err = glu64(act, *host)
    for o, r, e, n in zip((H, G, U), ref, err, "HGU"):
        assert_within(o.view, r, e, n)
        assert o.intact(), f"{n}: wrote outside its view"
    # Not keeping G and U changes nothing in H.
    assert torch.equal(rs.glu(X, Wg, Wu, act=act, transw=transw), H.view)


@pytest.mark.parametrize("transw", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("shape", [(1, 512, 512), (7, 129, 65), (128, 256, 384), (300, 100, 260),
                                   (1024, 64, 2048), (130, 1024, 1025)],
                         ids=lambda s: "x".join(map(str, s)))
def test_integer_operands_are_exact(shape, transw):
    # |partial sums| <= 4 K < 2^24 and relu: every operation is exact, and
    # the product of two sums of at most 4096 stays below 2^24.
    M, K, F = shape
    X, Wg, Wu, host = operands(M, K, F, transw, seed=1, integer=True)
    H, G, U = rs.glu(X, Wg, Wu, act="relu", transw=transw, save=True)
    (h, g, u), _ = glu64("relu", *host)
    assert torch.equal(G.cpu().double(), g) and torch.equal(U.cpu().double(), u)
    assert torch.equal(H.cpu().double(), h)


# Outputs of few tiles under a long K, which eager calls split across
# workgroups: 32 x 32 tiles (the last two F with 4-byte loads, as no row of
# the weights or of X is aligned), 64 x 64 tiles, chunks that end inside a
# slab, and packed copies that are split too (417 x 3001); and at most 32 rows
# of wide weights, split in two or not; and wide unaligned weights under few
# rows (packed or not) and many.
SPLIT_SHAPES = [(17, 4096, 256), (24, 2052, 130), (64, 1028, 60), (33, 16384, 4), (20, 2047, 255),
                (17, 1537, 1), (217, 2100, 1200), (65, 4100, 2052), (300, 2048, 516), (417, 3001, 1025),
                (32, 2080, 9216), (23, 2049, 9001), (17, 260, 8200), (32, 95, 16400),
                (20, 67, 16385), (64, 131, 16385), (128, 35, 8200), (100, 69, 8193), (310, 37, 4098)]


@pytest.mark.parametrize("transw", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("shape", SPLIT_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_long_sums_over_few_tiles(shape, transw):
    M, K, F = shape
    i = SPLIT_SHAPES.index(shape)
    act = ACTS[i % len(ACTS)]
    X, Wg, Wu, host = operands(M, K, F, transw, seed=100 + i, kind=("halves", "separate", "gaps")[i % 3])
    H, G, U = (Guarded(M, F, gap=g) for g in (3, 0, 0))
    U.ld = G.ld
    rs.glu(X, Wg, Wu, act=act, transw=transw, out=H.view, save=(G.view, U.view))
    ref, err = glu64(act, *host)
    for o, r, e, n in zip((H, G, U), ref, err, "HGU"):
        assert_within(o.view, r, e, n)
        assert o.intact(), f"{n}: wrote outside its view"
    for _ in range(3):
        assert torch.equal(rs.glu(X, Wg, Wu, act=act, transw=transw), H.view)
    # A captured call runs unsplit, within the same bounds on every replay.
    out = torch.empty((M, F), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.glu(X, Wg, Wu, act=act, transw=transw, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert_within(out, ref[0], err[0], "replay")
        assert torch.equal(rs.glu(X, Wg, Wu, act=act, transw=transw), H.view)


@pytest.mark.parametrize("act", ACTS)
def test_every_activation_over_its_range(act):
    # K = 1: G = x wg and U = x wu exactly representable, so only the
    # activation is tested, over both tails and the values around zero.
    g = torch.cat([torch.linspace(-30, 30, 1201), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0,
                                                              100.0, -100.0])])
    X = torch.ones((1, 1))
    H = rs.glu(X.cuda(), g[None].cuda(), torch.ones_like(g)[None].cuda(), act=act)
    (h, _, _), _ = glu64(act, X.double(), g[None].double(), torch.ones_like(g)[None].double())
    from tests.ff_util import act_err
    assert_within(H, h, act_err(g[None].double()), act)


def test_non_finite_values_stay_in_their_rows_and_columns():
    M, K, F = 70, 96, 140
    X, Wg, Wu, host = operands(M, K, F, False, seed=3)
    want = rs.glu(X, Wg, Wu, act="gelu")
    X2 = X.clone()
    X2[5, 7] = float("nan")
    X2[40, 0] = float("inf")
    Wu2 = Wu.clone()
    Wu2[3, 11] = float("nan")
    got = rs.glu(X2, Wg.contiguous(), Wu2, act="gelu")
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[[5, 40]] = False
    cols = torch.ones(F, dtype=torch.bool, device="cuda")
    cols[11] = False
    assert torch.isnan(got[5]).all() and not torch.isfinite(got[40]).any()
    assert torch.isnan(got[:, 11]).all()
    keep = rows[:, None] & cols[None]
    assert torch.allclose(got[keep], want[keep], rtol=0, atol=1e-5)


def test_empty_sizes():
    X, Wg, Wu, _ = operands(4, 6, 5, False, seed=1)
    assert rs.glu(X[:0], Wg, Wu).shape == (0, 5)
    assert rs.glu(X, Wg[:, :0], Wu[:, :0]).shape == (4, 0)
    H, G, U = rs.glu(X[:, :0].contiguous(), Wg[:0].contiguous(), Wu[:0].contiguous(), act="sigmoid",
                     save=True)
    assert all(bool((t == 0).all()) for t in (H, G, U))


GRAD_SHAPES = [(1, 64, 64), (2, 33, 17), (5, 1, 3), (8, 300, 64), (33, 65, 129), (64, 128, 256),
               (257, 100, 66), (300, 260, 170), (640, 96, 320)]


@pytest.mark.parametrize("transw", [False, True], ids=["KxF", "FxK"])
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, transw):
    M, K, F = shape
    i = GRAD_SHAPES.index(shape)
    act = ACTS[(i + transw) % len(ACTS)]
    X, Wg, Wu, host = operands(M, K, F, transw, seed=20 + i, kind=("halves", "separate", "gaps")[i % 3])
    gen = torch.Generator().manual_seed(100 + i)
    dH = torch.randn((M, F), generator=gen)
    _, G, U = rs.glu(X, Wg, Wu, act=act, transw=transw, save=True)
    ref, err = glu_backward64(act, *host, G.cpu().double(), U.cpu().double(), dH.double())
    wshape = (F, K) if transw else (K, F)
    dX, dWg, dWu = Guarded(M, K, gap=2), Guarded(*wshape, gap=1), Guarded(*wshape, gap=1)
    rs.glu_backward(dH.cuda(), X, Wg, Wu, G, U, act=act, transw=transw, dX=dX.view,
                    dW=(dWg.view, dWu.view))
    for o, r, e, n in zip((dX, dWg, dWu), ref[2:], err[2:], ("dX", "dWg", "dWu")):
        got = o.view.t() if transw and n != "dX" else o.view
        assert_within(got, r, e, n)
        assert o.intact(), n
    # The allocating form, with the weight gradients as halves of one buffer.
    dX2, dWg2, dWu2 = rs.glu_backward(dH.cuda(), X, Wg, Wu, G, U, act=act, transw=transw)
    for o, r, e in zip((dX2, dWg2.t() if transw else dWg2, dWu2.t() if transw else dWu2), ref[2:],
                       err[2:]):
        assert_within(o, r, e)


def test_backward_in_place_and_accumulating():
    M, K, F, act = 65, 96, 130, "silu"
    X, Wg, Wu, host = operands(M, K, F, True, seed=5)
    dH = torch.randn((M, F), generator=torch.Generator().manual_seed(6))
    _, G, U = rs.glu(X, Wg, Wu, act=act, transw=True, save=True)
    ref, err = glu_backward64(act, *host, G.cpu().double(), U.cpu().double(), dH.double())
    base = torch.randn((2 * F, K), device="cuda")
    dW = base.clone()
    dX, dWg, dWu = rs.glu_backward(dH.cuda(), X, Wg, Wu, G, U, act=act, transw=True, beta=2.0,
                                   dW=(dW[:F], dW[F:]), inplace=True)
    # In place: G and U now hold dG and dU.
    assert_within(G, ref[0], err[0], "dG")
    assert_within(U, ref[1], err[1], "dU")
    assert_within(dX, ref[2], err[2], "dX")
    for got, r, e, b in ((dWg, ref[3], err[3], base[:F]), (dWu, ref[4], err[4], base[F:])):
        b2 = 2 * b.cpu().double().t()
        assert_within(got.t(), r + b2, e + 3 * 2.0 ** -24 * (r.abs() + b2.abs() + e), "dW")


def test_backward_parts_and_empty_sizes():
    M, K, F = 12, 20, 16
    X, Wg, Wu, _ = operands(M, K, F, False, seed=8)
    dH = torch.randn((M, F), device="cuda")
    _, G, U = rs.glu(X, Wg, Wu, save=True)
    full = rs.glu_backward(dH, X, Wg, Wu, G, U)
    only_x = rs.glu_backward(dH, X, Wg, Wu, G, U, need_dw=False)
    only_w = rs.glu_backward(dH, X, Wg, Wu, G, U, need_dx=False)
    assert torch.equal(only_x[0], full[0]) and only_x[1] is None and only_x[2] is None
    assert only_w[0] is None and torch.equal(only_w[1], full[1]) and torch.equal(only_w[2], full[2])
    # No rows: the weight gradients are beta times what they held.
    e = rs.glu_backward(dH[:0], X[:0], Wg, Wu, G[:0], U[:0])
    assert e[0].shape == (0, K) and not e[1].any() and not e[2].any()
    # No columns: dX is zero.
    z = rs.glu_backward(dH[:, :0], X, Wg[:, :0], Wu[:, :0], G[:, :0], U[:, :0])
    assert not z[0].any() and z[1].shape == (K, 0)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(act):
    """The GPU gradients along a direction against 64-bit central differences
    of the forward formula."""
    M, K, F = 6, 40, 24
    X, Wg, Wu, host = operands(M, K, F, False, seed=9)
    gen = torch.Generator().manual_seed(10)
    dH = torch.randn((M, F), generator=gen)
    H, G, U = rs.glu(X, Wg, Wu, act=act, save=True)
    grads = rs.glu_backward(dH.cuda(), X, Wg, Wu, G, U, act=act)
    for i, g in enumerate(grads):
        V = torch.randn(host[i].shape, generator=gen, dtype=torch.float64)
        h, ends = 1e-5, []
        for step in (h, -h):
            moved = list(host)
            moved[i] = host[i] + step * V
            ends.append(float((glu64(act, *moved)[0][0] * dH.double()).sum()))
        slope = (ends[0] - ends[1]) / (2 * h)
        got = float((g.cpu().double() * V).sum())
        # float32 gradients: sums of up to 2 F + M terms; differences: h^2
        # times third derivatives of order 100 (relu: a kink within h of one
        # of M F values of G moves the slope by at most h |V|).
        scale = float((g.cpu().double().abs() * V.abs()).sum())
        assert abs(got - slope) <= 4 * (2 * F + M + K) * 2.0 ** -24 * scale + 1e-5 * max(1.0, scale) * 0.1


def test_capture_and_replay():
    """Forward and backward captured into one graph; replays on new inputs
    equal the eager calls, with eager work in between."""
    M, K, F, act = 200, 160, 240, "silu"
    X, Wg, Wu, _ = operands(M, K, F, True, seed=11)
    dH = torch.randn((M, F), device="cuda")
    H, G, U = (torch.empty((M, F), device="cuda") for _ in range(3))
    dX, dWg, dWu = torch.empty_like(X), torch.empty((F, K), device="cuda"), torch.empty((F, K), device="cuda")

    def step():
        rs.glu(X, Wg, Wu, act=act, transw=True, out=H, save=(G, U))
        rs.glu_backward(dH, X, Wg, Wu, G, U, act=act, transw=True, dX=dX, dW=(dWg, dWu), inplace=True)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(3):
        X.copy_(torch.randn_like(X))
        dH.copy_(torch.randn_like(dH))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (H, G, U, dX, dWg, dWu)]
        # The eager call may split K where a captured one does not: compare
        # both with the 64-bit form.
        host = [X.cpu().double(), Wg.t().cpu().double(), Wu.t().cpu().double()]
        (h, g, u), (eh, eg, eu) = glu64(act, *host)
        assert_within(got[0], h, eh, f"replay {r} H")
        ref, err = glu_backward64(act, *host, g, u, dH.cpu().double())
        # dG, dU come from the float G and U: their errors, through act'' <=
        # 1.2 and act' <= 1.13, join the bounds.
        d = dH.cpu().double().abs()
        err = list(err)
        err[0] += d * (1.2 * u.abs() * eg + 1.13 * eu + 1.2 * eg * eu)
        err[1] += d * 1.13 * eg
        err[2] = err[2] + err[0] @ host[1].t().abs() + err[1] @ host[2].t().abs()
        for o, (rr, ee) in zip(got[1:3], zip(ref[:2], err[:2])):
            assert_within(o, rr, ee, f"replay {r} dG, dU")
        assert_within(got[3], ref[2], err[2], f"replay {r} dX")
        for o, rr, e0, e1 in ((got[4], ref[3], err[3], err[0]), (got[5], ref[4], err[4], err[1])):
            assert_within(o.t(), rr, e0 + host[0].t().abs() @ e1, f"replay {r} dW")
        step()
        torch.cuda.synchronize()
        assert torch.allclose(H, got[0], rtol=1e-4, atol=1e-4)


def test_side_stream():
    M, K, F = 64, 128, 96
    X, Wg, Wu, host = operands(M, K, F, False, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        H = rs.glu(X, Wg, Wu)
    side.synchronize()
    ref, err = glu64("silu", *host)
    assert_within(H, ref[0], err[0])


def test_run_to_run():
    X, Wg, Wu, _ = operands(300, 500, 400, False, seed=13)
    dH = torch.randn((300, 400), device="cuda")
    first = None
    for _ in range(3):
        H, G, U = rs.glu(X, Wg, Wu, act="gelu", save=True)
        got = (H, G, U, *rs.glu_backward(dH, X, Wg, Wu, G, U, act="gelu"))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_refusals():
    M, K, F = 6, 12, 10
    X, Wg, Wu, _ = operands(M, K, F, False, seed=1)
    with pytest.raises(ValueError, match="shape"):
        rs.glu(X, Wg, Wu, transw=True)
    with pytest.raises(ValueError, match="row stride"):
        rs.glu(X, Wg, Wu.contiguous())
    with pytest.raises(ValueError, match="column stride"):
        rs.glu(torch.randn((K, M), device="cuda").t(), Wg, Wu)
    with pytest.raises(ValueError, match="row stride"):
        rs.glu(X, Wg[:1].expand(K, F), Wu[:1].expand(K, F))
    with pytest.raises(TypeError):
        rs.glu(X.half(), Wg, Wu)
    with pytest.raises(ValueError, match="GPU"):
        rs.glu(X, Wg.cpu(), Wu.cpu())
    with pytest.raises(ValueError, match="shape"):
        rs.glu(X, Wg, Wu, out=torch.empty((M, F + 1), device="cuda"))
    buf = torch.zeros((M, 2 * F), device="cuda")
    with pytest.raises(rs.SgemmError) as e:
        rs.glu(X, Wg, Wu, out=buf[:, :F], save=(buf[:, 1:F + 1], buf[:, F:]))
    assert e.value.status == 5  # SGEMM_ERR_ALIAS
    H, G, U = rs.glu(X, Wg, Wu, save=True)
    with pytest.raises(ValueError, match="beta"):
        rs.glu_backward(H, X, Wg, Wu, G, U, beta=1.0)
    with pytest.raises(ValueError, match="shape"):
        rs.glu_backward(H[:, :F - 1], X, Wg, Wu, G, U)
    with pytest.raises(rs.SgemmError) as e:
        rs.glu_backward(H, X, Wg, Wu, G, U, dX=X)
    assert e.value.status == 5


def test_same_rows_twice_and_shared_weights():
    """One tensor as both weights, and dH, G and U as one tensor: inputs may
    overlap."""
    M, K, F = 20, 48, 36
    X, Wg, _, host = operands(M, K, F, False, seed=2, kind="separate")
    H, G, U = rs.glu(X, Wg, Wg, act="relu", save=True)
    ref, err = glu64("relu", host[0], host[1], host[1])
    for o, r, e in zip((H, G, U), ref, err):
        assert_within(o, r, e)
    assert torch.equal(G, U)
    dX, dWg, dWu = rs.glu_backward(G, X, Wg, Wg, G, G, act="relu")
    g = G.cpu().double()
    ref, err = glu_backward64("relu", host[0], host[1], host[1], g, g, g)
    for o, r, e in zip((dX, dWg, dWu), ref[2:], err[2:]):
        assert_within(o, r, e)


@pytest.mark.parametrize("rows", [3, 24])
def test_two_streams_at_once(rows):
    """Calls that pack (a workspace) on two streams together."""
    M, K, F = 700 + rows, 515, 771
    sets = [operands(M, K, F, False, seed=s) for s in (1, 2)]
    want = [rs.glu(X, Wg, Wu, act="gelu") for X, Wg, Wu, _ in sets]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in sets], []
    for _ in range(4):
        for st, (X, Wg, Wu, _) in zip(streams, sets):
            with torch.cuda.stream(st):
                outs.append(rs.glu(X, Wg, Wu, act="gelu"))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


def test_offsets_past_32_bits():
    """More than 2^31 results, rows from both ends and the middle checked."""
    M, K, F = 66000, 16, 33000
    X, Wg, Wu, host = operands(M, K, F, True, seed=3, kind="separate")
    H = rs.glu(X, Wg, Wu, transw=True)
    rows = torch.tensor([0, 1, 32767, 40001, M - 2, M - 1])
    ref, err = glu64("silu", host[0][rows], host[1], host[2])
    assert_within(H[rows.cuda()], ref[0], err[0])

"""Orthogonalised updates on the GPU: one step against an elementwise bound,
all steps against a bound of the whole error, both in 64 bits."""
import pytest
import torch

import roofline_sgemm_f32_amd as rs
from tests.adapt_util import MUON, ortho64, ortho_norm_bound, ortho_step64
from tests.ff_util import HALF_STEP, TYPES, Guarded, assert_within, rounded

pytestmark = pytest.mark.gpu
CUBIC = (1.5, -0.5, 0.0)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rs.load()


def gradient(gen, m, n, dtype):
    g = torch.randn((m, n), generator=gen) + 2 * torch.randn((m, 1), generator=gen) * torch.randn((1, n), generator=gen)
    return (1e-3 * g).to(dtype)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (5, 4096), (2000, 16), (31, 33), (64, 64), (65, 63), (64, 1000),
          (127, 129), (128, 128), (200, 72), (256, 256), (257, 300), (300, 511), (520, 136), (384, 700)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_one_step(shape, t):
    gen = torch.Generator().manual_seed(sum(shape))
    G = gradient(gen, *shape, TYPES[t])
    out = Guarded(*shape, TYPES[t], gap=sum(shape) % 3)
    rs.orthogonalize(G.cuda(), steps=1, out=out.view)
    ref, err = ortho_step64(G, MUON)
    assert_within(out.view, ref, rounded(ref, err, TYPES[t]))
    assert out.intact()


@pytest.mark.parametrize("coef", [MUON, CUBIC, ((4.0, -7.0, 4.0), MUON, CUBIC)], ids=["muon", "cubic", "each"])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", [(1, 5), (16, 300), (96, 64), (130, 257), (300, 300)], ids=lambda s: "x".join(map(str, s)))
def test_all_steps(shape, t, coef):
    gen = torch.Generator().manual_seed(sum(shape))
    G = gradient(gen, *shape, TYPES[t])
    steps = [tuple(coef)] * 5 if not isinstance(coef[0], tuple) else list(coef)
    got = rs.orthogonalize(G.cuda(), coefficients=coef).cpu().double()
    ref = ortho64(G, steps)
    bound = ortho_norm_bound(G, steps) + HALF_STEP[TYPES[t]] * float(ref.norm())
    assert float((got - ref).norm()) <= bound


# Stacks that take each tile of each product in turn: (count, rows, columns) and the
# tiles of S (with its shares), of P and of P X.
STACKS = [(1, 65, 1030), (12, 640, 400), (16, 130, 2601), (16, 4097, 130), (12, 701, 699), (3, 770, 4096),
          (16, 900, 905), (3, 1100, 4099), (12, 1300, 1299), (2, 2048, 3001), (16, 1031, 1500)]


@pytest.mark.parametrize("shape", STACKS, ids=lambda s: "x".join(map(str, s)))
def test_every_tile(shape):
    """64/7 64 64; 64 64 128; 64/2 64 192; 64/2 64 256; 128 128 64; 128/3 64 256;
    192 192 256; 192/4 64 256; 256 256 192; 256/3 64 256: one step elementwise, two
    steps by norm, in float64 on the GPU."""
    i = STACKS.index(shape)
    gen = torch.Generator(device="cuda").manual_seed(i)
    dt = list(TYPES.values())[i % 3]
    b, m, n = shape
    G = torch.randn(shape, generator=gen, device="cuda")
    G += 2 * torch.randn((b, m, 1), generator=gen, device="cuda") * torch.randn((b, 1, n), generator=gen, device="cuda")
    G = (1e-3 * G).to(dt)
    one, two = rs.orthogonalize(G, steps=1), rs.orthogonalize(G, steps=2, coefficients=CUBIC)
    for k in {0, b // 2, b - 1}:
        ref, err = ortho_step64(G[k], MUON, device="cuda")
        d = (one[k].double() - ref).abs()
        assert bool((d <= rounded(ref, err, dt)).all()), k
        ref = ortho64(G[k], [CUBIC] * 2, device="cuda")
        bound = ortho_norm_bound(G[k], [CUBIC] * 2, device="cuda") + HALF_STEP[dt] * float(ref.norm())
        assert float((two[k].double() - ref).norm()) <= bound, k


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shape", [(3, 70, 40), (5, 16, 520), (2, 200, 136)], ids=lambda s: "x".join(map(str, s)))
def test_stacks_views_and_in_place(shape, t):
    """A stack with gaps everywhere gives what its matrices give alone, bit for
    bit, also in place and from a view at an odd offset."""
    gen = torch.Generator().manual_seed(7)
    dt = TYPES[t]
    b, m, n = shape
    G = torch.stack([gradient(gen, m, n, dt) * 10.0 ** i for i in range(b)]).cuda()
    alone = [rs.orthogonalize(g.contiguous()) for g in G]
    assert all(torch.equal(a, o) for a, o in zip(alone, rs.orthogonalize(G)))
    wide = torch.full((b, m + 2, n + 5), float("nan"), dtype=dt, device="cuda")
    view = wide[:, 1:-1, 3:-2]
    view.copy_(G)
    assert rs.orthogonalize(view, out=view) is view
    assert all(torch.equal(a, o) for a, o in zip(alone, view))
    keep = wide.clone()
    keep[:, 1:-1, 3:-2] = float("nan")
    assert bool(torch.isnan(keep).all())
    # The same matrix in every place.
    same = rs.orthogonalize(G[1:2].expand(b, m, n))
    assert all(torch.equal(alone[1], o) for o in same)


@pytest.mark.parametrize("shape", [(40, 70), (90, 70), (70, 1100)], ids=lambda s: "x".join(map(str, s)))
def test_zeros_and_what_is_not_finite(shape):
    for t in TYPES.values():
        G = torch.zeros((3, *shape), dtype=t, device="cuda")
        assert not rs.orthogonalize(G).any()
        assert not rs.orthogonalize(G, eps=0.0).any()
        for bad in (float("nan"), float("inf"), -float("inf")):
            G = torch.ones((3, *shape), dtype=t, device="cuda")
            G[:, 0] = 2
            G[1, 5, 6] = bad
            O = rs.orthogonalize(G)
            assert bool(torch.isnan(O[1]).all()), bad
            assert bool(torch.isfinite(O[0]).all()) and torch.equal(O[0], O[2])


@pytest.mark.parametrize("rows", [50, 100])
@pytest.mark.parametrize("factor", [2.0 ** -100, 2.0 ** 100])
def test_scale_of_the_gradient_does_not_matter(factor, rows):
    """Squares outside float's range; without eps a power of two changes no bit."""
    gen = torch.Generator().manual_seed(1)
    G = gradient(gen, rows, 80, torch.float32).cuda()
    assert torch.equal(rs.orthogonalize(G * factor, eps=0.0), rs.orthogonalize(G, eps=0.0))


@pytest.mark.parametrize("shape", [(40, 60), (100, 90)], ids=lambda s: "x".join(map(str, s)))
def test_one_large_element(shape):
    """All of the norm in one place: the small ones keep their own precision (their
    parts are below float16's normal numbers)."""
    gen = torch.Generator().manual_seed(2)
    G = torch.randn(shape, generator=gen) * 1e-4
    G[3, 4] = 1.0
    ref, err = ortho_step64(G, MUON)
    assert_within(rs.orthogonalize(G.cuda(), steps=1), ref, rounded(ref, err, torch.float32))


def test_same_bits_in_a_graph_and_on_two_streams():
    gen = torch.Generator().manual_seed(4)
    Gs = [gradient(gen, m, n, torch.float32).cuda() for m, n in ((136, 200), (64, 520))]
    want = [rs.orthogonalize(G) for G in Gs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [rs.orthogonalize(G) for G in Gs]
    for _ in range(3):
        for t in got:
            t.fill_(float("nan"))
        rs.orthogonalize(Gs[1][:40])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    streams = [torch.cuda.Stream() for _ in Gs]
    outs = [[], []]
    for _ in range(6):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(rs.orthogonalize(Gs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(want[i], o) for o in outs[i])


def test_empty():
    for shape in ((0, 4), (4, 0), (0, 3, 4), (2, 0, 3)):
        G = torch.zeros(shape, device="cuda")
        assert rs.orthogonalize(G).shape == G.shape


def test_refusals():
    G = torch.ones((4, 6), device="cuda")
    with pytest.raises(ValueError, match="unit column stride"):
        rs.orthogonalize(G.t())
    with pytest.raises(ValueError, match="out"):
        rs.orthogonalize(G, out=G[:3])
    with pytest.raises(TypeError, match="out"):
        rs.orthogonalize(G, out=G.half())
    with pytest.raises(ValueError, match="out"):
        rs.orthogonalize(G, out=G.cpu())
    with pytest.raises(rs.SgemmError, match="ALIAS"):
        buf = torch.ones((4, 7), device="cuda")
        rs.orthogonalize(buf[:, :6], out=buf[:, 1:])
    for coef in ((100.0, 0.0, 0.0), (float("nan"), 0.0, 0.0)):
        with pytest.raises(rs.SgemmError, match="ARG"):
            rs.orthogonalize(G, coefficients=coef)
    for steps in (0, 65):
        with pytest.raises((rs.SgemmError, ValueError)):
            rs.orthogonalize(G, steps=steps)

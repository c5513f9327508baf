"""The largest tiles of the Newton-Schulz products where they are ragged, and a
weight's results in calls that deal it out differently."""
import pytest

from gpu_checks import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
A0, B0, C0 = 3.4445, -4.7750, 2.0315
# 1550, 1551, 6299 and 6301 are no multiples of 320, 256, 128 or 32; the third weight's last tiles are mostly empty
SHAPES = [(1550, 6301), (6299, 1551), (300, 500)]


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def cdiv(a, b):
    return -(-a // b)


def tiles(shapes, bm, bn):
    return sum(cdiv(min(s), bm) * cdiv(max(s), bn) for s in shapes)


def iterate(G, steps=5):
    X = G.double() / (G.double().norm() + 1e-7)
    X = X.t().contiguous() if G.shape[0] > G.shape[1] else X
    for _ in range(steps):
        A = X @ X.t().contiguous()
        X = A0 * X + (B0 * A + C0 * (A @ A)) @ X
    return X.t() if G.shape[0] > G.shape[1] else X


def bound(precise):
    """Full rank, five steps: the two kinds of operands' statements in the header."""
    return 1e-5 if precise else 5 * 6e-4


def draw(seed, shapes, scale=1e-3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(*s, generator=gen, device="cuda") * scale for s in shapes]


def test_these_weights_get_the_large_tiles():
    """The kernels' rules on the CUs of this card: 320 x 256 of fp16 operands, 128 x 256 in two parts."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    squares = tiles(SHAPES, 128, 128)
    assert cdiv(tiles(SHAPES, 320, 256), cus) * 25 * cus < squares * 6
    assert cdiv(tiles(SHAPES, 128, 256), cus) * 12 < cdiv(squares, cus) * 7


@pytest.mark.parametrize("precise", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_orthogonalize(sp, precise, dtype):
    Gs = draw(1, SHAPES)
    outs = [Guarded(s, dtype, fill=0xFF) for s in SHAPES]
    arr = (sp.OrthoJob * 3)(*[sp.OrthoJob(0, 0, *s) for s in SHAPES])
    ws = Guarded((sp.lib().sp24_orthogonalize_workspace(arr, 3),), torch.uint8, fill=0x7F)
    sp.sp24_orthogonalize_batch(Gs, dtype=dtype, outs=[o.t for o in outs], workspace=ws.t, precise=precise)
    ws.check("workspace")
    for G, o in zip(Gs, outs):
        o.check()
        want = iterate(G)
        err = ((o.t.double() - want).norm() / want.norm()).item()
        assert err <= bound(precise) + (2.0 ** -11 if dtype == torch.float16 else 0.0)


@pytest.mark.parametrize("precise", [True, False])
def test_optimiser_step(sp, precise):
    G, M0, P0 = draw(2, SHAPES), draw(3, SHAPES, 1e-2), draw(4, SHAPES, 0.02)
    M, P, W = ([Guarded(s, t) for s in SHAPES] for t in (torch.float32, torch.float32, torch.float16))
    for g, t in zip(M + P, M0 + P0):
        g.t.copy_(t)
    sp.sp24_muon_step(G, [m.t for m in M], [p.t for p in P], [w.t for w in W], [0.5] * 3, decays=[0.01] * 3, precise=precise)
    for k in range(3):
        for g in (M[k], P[k], W[k]):
            g.check()
        m = 0.95 * M0[k].double() + G[k].double()
        X = iterate(G[k].double() + 0.95 * m)
        # momentum in fp32, 0.95 and 0.99 as fp32 numbers; the update's direction to 2^-22
        assert ((M[k].t.double() - m).abs() <= 4 * 2.0 ** -24 * (M0[k].double().abs() + G[k].double().abs() + m.abs())).all()
        err = (P[k].t.double() - (0.99 * P0[k].double() - 0.5 * X)).norm()
        assert err <= bound(precise) * 0.5 * X.norm() + 3 * 2.0 ** -24 * (P0[k].double().norm() + 0.5 * X.norm())
        assert torch.equal(W[k].t, P[k].t.half())


@pytest.mark.parametrize("precise", [True, False])
def test_alone_and_beside_others_to_the_same_accuracy(sp, precise):
    """The tiles and the split of a reduction are chosen for a call's weights together, so a weight's bits
    may differ between calls; its accuracy does not, and the same call gives the same bits."""
    shapes = [(1600, 6400), (6400, 1600), (200, 330)]
    Gs = draw(5, shapes)
    for batch in ([0], [0, 1], [0, 1, 2], [2, 0]):
        got = sp.sp24_orthogonalize_batch([Gs[k] for k in batch], dtype=torch.float32, precise=precise)
        again = sp.sp24_orthogonalize_batch([Gs[k] for k in batch], dtype=torch.float32, precise=precise)
        for k, x, y in zip(batch, got, again):
            want = iterate(Gs[k])
            assert torch.equal(x, y)
            assert ((x.double() - want).norm() / want.norm()).item() <= bound(precise)

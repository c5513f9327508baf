"""GPU checks of the two kinds of operands that the orthogonalised updates and
the optimiser step take: fp32's accuracy unless the caller asks for fp16
operands, whatever the results' type."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# all steps in one workgroup in either mode; with fp16 operands only; a chain of launches, wide and tall
SHAPES = [(64, 64), (128, 160), (300, 900), (1001, 357)]


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def gauss(seed, *shape):
    return torch.from_numpy(np.random.default_rng([seed, *shape]).standard_normal(shape).astype(np.float32) * 1e-2).cuda()


@pytest.mark.parametrize("shape", SHAPES)
def test_fp16_results_are_fp32_ones_rounded_once(sp, shape):
    """The same products, so the same bits: an fp16 result has the error of its rounding and no other."""
    G = gauss(1, *shape)
    assert torch.equal(sp.sp24_orthogonalize(G), sp.sp24_orthogonalize(G, dtype=torch.float32).half())
    fast = sp.sp24_orthogonalize(G, dtype=torch.float32, precise=False)
    assert torch.equal(sp.sp24_orthogonalize(G, precise=False), fast.half())
    assert not torch.equal(fast, sp.sp24_orthogonalize(G, dtype=torch.float32))


@pytest.mark.parametrize("shape", SHAPES)
def test_the_optimiser_is_precise_unless_told_otherwise(sp, shape):
    from structured_sparse_transformer_amd.muon import Muon
    G, P0 = gauss(2, *shape), gauss(3, *shape).half().float()

    def step(**kw):
        M, P, W = torch.zeros_like(G), P0.clone(), P0.half()
        sp.sp24_muon_step([G], [M], [P], [W], [0.5], **kw)
        return P

    precise = step(precise=True)
    assert torch.equal(step(), precise)
    assert not torch.equal(step(precise=False), precise)
    of_class = Muon([P0.half()], lr=0.1)
    of_class.step([G])
    told = Muon([P0.half()], lr=0.1, precise=True)
    told.step([G])
    assert torch.equal(of_class.masters[0], told.masters[0])


# Accuracy, normwise against float64, in the units of the header's statement.
#   Growth: X's 22 bits and the fp32 sums leave some 1e-6 of a rank-one result's
#   norm a step (in quadrature (a + |b| + c) 2^-23 / sqrt(3) three times over,
#   over the step's a + b + c = 0.70: 1.7e-6), which every later step multiplies
#   by a where the update has nothing; the steps' shares add up geometrically, to
#   1.4 times the first's.  Stated as 3e-6 a^(steps - 1).
#   fp16 operands: A, B and X are rounded to 2^-12 / sqrt(3) in the mean square,
#   times |b| + 2 c, 1 and |B| <= 2.8: sqrt(8.8^2 + 2.8^2 + 2.8^2) 1.4e-4 = 1.4e-3
#   of a singular value near 1 in the one step that takes it there and less in
#   the others; 5e-4 a step where 128 rows or more average it out, and five times
#   that below.
GROWTH, A0 = 3e-6, 3.4445


def bound(shape, steps, precise):
    each = 0.0 if precise else 5e-4 if min(shape) >= 128 else 2.5e-3
    return GROWTH * A0 ** (steps - 1) + steps * each


def spectrum(kind, R, C):
    rng = np.random.default_rng([7, R, C])
    m = min(R, C)
    if kind.startswith("rank"):
        k, noise = kind[4:].split("+")
        k = min(int(k), m)
        x = rng.standard_normal((R, k)) @ rng.standard_normal((k, C)) / np.sqrt(k) + float(noise) * rng.standard_normal((R, C))
    else:
        i = np.arange(1.0, m + 1)
        s = {"i^-1": 1 / i, "i^-2": i ** -2, "exp": np.exp(-i / 10), "flat": np.ones(m)}[kind]
        x = (np.linalg.qr(rng.standard_normal((R, m)))[0] * s) @ np.linalg.qr(rng.standard_normal((C, m)))[0].T
    return (x * 1e-2).astype(np.float32)


def iterate(X, steps, a=A0, b=-4.7750, c=2.0315):
    """In float64, on whatever X is (an array or a tensor), m <= n or not."""
    if X.shape[0] > X.shape[1]:
        return iterate(X.T, steps, a, b, c).T
    X = X / ((X ** 2).sum() ** 0.5 + 1e-7)
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


@pytest.mark.parametrize("kind", ["rank1+0", "rank16+0", "rank32+0", "rank16+1e-3", "rank20+0.05", "i^-1", "i^-2", "exp", "flat"])
@pytest.mark.parametrize("shape", [(20, 30), (64, 64), (128, 160), (300, 900), (900, 130)])
def test_accuracy_over_spectra_and_steps(sp, shape, kind):
    G = spectrum(kind, *shape)
    for steps in (1, 2, 5, 6, 8):
        want = iterate(G.astype(np.float64), steps)
        for precise in (True, False):
            got = sp.sp24_orthogonalize(torch.from_numpy(G).cuda(), steps, dtype=torch.float32, precise=precise)
            err = np.linalg.norm(got.cpu().numpy() - want) / np.linalg.norm(want)
            assert err <= bound(shape, steps, precise), (steps, precise, err)
        got = sp.sp24_orthogonalize(torch.from_numpy(G).cuda(), steps, precise=False).cpu().numpy().astype(np.float64)
        assert np.linalg.norm(got - want) <= (bound(shape, steps, False) + 2.0 ** -11) * np.linalg.norm(want)


@pytest.mark.parametrize("rank", [1, 64, 1600])
def test_accuracy_at_the_widest_layer(sp, rank):
    gen = torch.Generator(device="cuda").manual_seed(rank)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    G = (rand(1600, rank) @ rand(rank, 6400)).float()
    for steps in (5, 8):
        want = iterate(G.double(), steps)
        for precise in (True, False):
            got = sp.sp24_orthogonalize(G, steps, dtype=torch.float32, precise=precise).double()
            assert ((got - want).norm() / want.norm()).item() <= bound(G.shape, steps, precise)


@pytest.mark.parametrize("precise", [True, False])
def test_first_step_on_a_low_rank_gradient(sp, precise):
    """The optimiser's first step on the gradient of 24 tokens: momentum is that gradient alone."""
    G, P0, lr = spectrum("rank24+0", 256, 400), spectrum("flat", 256, 400), 0.5
    M, P = torch.zeros(256, 400, device="cuda"), torch.from_numpy(P0).cuda()
    sp.sp24_muon_step([torch.from_numpy(G).cuda()], [M], [P], [None], [lr], precise=precise)
    X = iterate(1.95 * G.astype(np.float64), 5)
    err = np.linalg.norm(P.cpu().numpy() - (P0.astype(np.float64) - lr * X))
    # and the roundings of P's three operations
    assert err <= bound((256, 400), 5, precise) * lr * np.linalg.norm(X) + 3 * 2.0 ** -24 * (np.linalg.norm(P0) + lr * np.linalg.norm(X))


@pytest.mark.parametrize("precise", [True, False])
@pytest.mark.parametrize("shape", [(1, 1), (40, 70), (300, 400)])
def test_coefficients_at_the_edge_of_the_range(sp, shape, precise):
    """A rank-one update's singular value goes 1 -> 3.9 -> -10.9, its square and X itself just inside
    fp16's range.  Three roundings of 2^-22 (or 2^-12) at most, each times (1 + 2 * 3.8) 3.9 / 10.9 = 3,
    and the fp32 sums'."""
    rng = np.random.default_rng([9, *shape])
    G = (rng.standard_normal((shape[0], 1)) @ rng.standard_normal((1, shape[1]))).astype(np.float32)
    rows = [(3.9, 0.0, 0.0), (1.0, -0.25, 0.0)]
    got = sp.sp24_orthogonalize(torch.from_numpy(G).cuda(), 2, rows, dtype=torch.float32, precise=precise)
    X = float(np.float32(3.9)) * G.astype(np.float64) / (np.linalg.norm(G.astype(np.float64)) + 1e-7)
    want = X - 0.25 * (X @ X.T @ X)
    err = np.linalg.norm(got.cpu().numpy() - want) / np.linalg.norm(want)
    assert err <= (1e-5 if precise else 9 * 2.0 ** -12)

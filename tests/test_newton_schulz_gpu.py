"""GPU checks of the orthogonalised updates and the optimiser step against
float64 Newton-Schulz iterations.

Tolerances, normwise.  A step rounds X, A and B once each, to u relative at
most: u = 2^-12 (half an ulp of 11 bits) for fp16 operands, 2^-22 for
operands in two parts with fp32 sums of K terms (sums by blocks of 16: about
sqrt(K / 16) 2^-24).  An error in one of the three reaches X' times at most
a + |b| + c = 10.25, and errors of the 3 steps-fold roundings are independent,
so the result's is taken as 10.25 sqrt(3 steps) u.  (Early errors grow with
the small singular values; what the lo part does not take of that stays below
the same bound.)  The result's own rounding adds 2^-11 or 2^-24.
"""
import math

import numpy as np
import pytest

from gpu_checks import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
COEFFS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def tol(dtype, shape, steps=5):
    u = 2.0 ** -12 if dtype == torch.float16 else 2.0 ** -22 + 2.0 ** -24 * math.sqrt(max(shape) / 16 + 4)
    return 10.25 * math.sqrt(3 * steps) * u + (2.0 ** -11 if dtype == torch.float16 else 2.0 ** -24)


def iterate(G, steps=5, coeffs=COEFFS, eps=1e-7):
    X = np.asarray(G, np.float64)
    X = X / (np.sqrt((X ** 2).sum()) + eps)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    rows = [coeffs] * steps if np.ndim(coeffs) == 1 else coeffs
    for a, b, c in rows:
        A = X @ X.T
        X = a * X + (b * A + c * A @ A) @ X
    return X.T if tall else X


def rel(got, want):
    n = np.linalg.norm(want)
    d = np.linalg.norm(got.double().cpu().numpy() - want)
    return d / n if n else d


def update(seed, R, C, kind="mixed"):
    rng = np.random.default_rng([seed, R, C])
    x = rng.standard_normal((R, C))
    if kind == "lowrank":
        k = max(1, min(R, C) // 16)
        x = rng.standard_normal((R, k)) @ rng.standard_normal((k, C)) / math.sqrt(k) + 0.05 * x
    elif kind == "mixed":
        x *= np.exp(rng.standard_normal((R, 1))) * np.exp(0.5 * rng.standard_normal((1, C)))
    return (x * 1e-2).astype(np.float32)


SHAPES = [(1, 1), (1, 9), (9, 1), (16, 16), (64, 64), (65, 63), (31, 200), (128, 128), (129, 130), (357, 1001), (1001, 357),
          (128, 640), (700, 96), (500, 500), (192, 1600)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
@pytest.mark.parametrize("g", [torch.float16, torch.float32])
def test_orthogonalize(sp, R, C, out, g):
    G = torch.from_numpy(update(1, R, C)).to(g)
    o = Guarded((R, C), out, fill=0xFF)
    arr = (sp.OrthoJob * 1)(sp.OrthoJob(0, 0, R, C))
    ws = Guarded((sp.lib().sp24_orthogonalize_workspace(arr, 1),), torch.uint8, fill=0x7F)
    sp.sp24_orthogonalize(G.cuda(), dtype=out, out=o.t, workspace=ws.t)
    o.check()
    ws.check("workspace")
    assert rel(o.t, iterate(G.numpy())) <= tol(out, (R, C))


@pytest.mark.parametrize("kind", ["gauss", "lowrank"])
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_spectra(sp, kind, out):
    G = update(2, 300, 900, kind)
    assert rel(sp.sp24_orthogonalize(torch.from_numpy(G).cuda(), dtype=out), iterate(G)) <= tol(out, G.shape)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
def test_steps_with_their_own_coefficients(sp, steps):
    G = update(3, 100, 260)
    rows = [(3.4445 - 0.1 * k, -4.7750 + 0.1 * k, 2.0315 - 0.05 * k) for k in range(steps)]
    for out in (torch.float16, torch.float32):
        got = sp.sp24_orthogonalize(torch.from_numpy(G).cuda(), steps, rows, dtype=out)
        assert rel(got, iterate(G, steps, rows)) <= tol(out, G.shape, steps)


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e25])
def test_scale_of_the_update_does_not_matter(sp, scale):
    G = update(4, 70, 150) * 100
    got = sp.sp24_orthogonalize(torch.from_numpy((G * np.float32(scale))).cuda(), eps=0.0, dtype=torch.float32)
    # the inputs' own rounding: relative 2^-24, and 2^-149 in units of 1e-30 among subnormals
    assert rel(got, iterate(G * np.float32(scale), eps=0.0)) <= tol(torch.float32, G.shape)


def test_zero_update_gives_zeros_and_small_rows_survive(sp):
    z = torch.zeros(40, 90, device="cuda")
    assert (sp.sp24_orthogonalize(z) == 0).all()
    G = update(5, 40, 90)
    G[7] = 0
    G[:, 11] = 0
    got = sp.sp24_orthogonalize(torch.from_numpy(G).cuda(), dtype=torch.float32)
    assert (got[7] == 0).all() and (got[:, 11] == 0).all()
    assert rel(got, iterate(G)) <= tol(torch.float32, G.shape)


def test_batch_of_shapes_equals_single_calls(sp):
    shapes = [(64, 64), (200, 77), (16, 300), (0, 5), (129, 128), (1, 1), (333, 40), (250, 260)]
    Gs = [torch.from_numpy(update(6, *s)).cuda() if s[0] else torch.empty(s, device="cuda") for s in shapes]
    for out in (torch.float16, torch.float32):
        for got, G in zip(sp.sp24_orthogonalize_batch(Gs, dtype=out), Gs):
            assert torch.equal(got, sp.sp24_orthogonalize(G, dtype=out))


def test_in_place_twice_the_same_and_in_a_graph(sp):
    for R, C in ((40, 50), (260, 300)):
        G = torch.from_numpy(update(7, R, C)).cuda()
        want = sp.sp24_orthogonalize(G, dtype=torch.float32)
        assert torch.equal(sp.sp24_orthogonalize(G, dtype=torch.float32), want)
        H = G.clone()
        assert torch.equal(sp.sp24_orthogonalize(H, dtype=torch.float32, out=H), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = sp.sp24_orthogonalize(G, dtype=torch.float32, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        arr = (sp.OrthoJob * 1)(sp.OrthoJob(0, 0, R, C))
        ws = torch.empty(sp.lib().sp24_orthogonalize_workspace(arr, 1), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(G)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sp.sp24_orthogonalize(G, dtype=torch.float32, out=out, workspace=ws)
        # the matrix units' sums are not the same bits for negated operands, so
        # each sign is compared with its own eager result
        minus = sp.sp24_orthogonalize(-G, dtype=torch.float32)
        for k in range(4):
            G.mul_(-1)
            ws.fill_(0x55)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want if k % 2 else minus)


def muon_ref(G, M, P, lr, decay, mu, nesterov):
    G, M, P = (np.asarray(v, np.float64) for v in (G, M, P))
    M = mu * M + G
    X = iterate(G + mu * M if nesterov else M)
    return M, (1 - decay) * P - lr * X, lr * np.linalg.norm(X)


@pytest.mark.parametrize("shapes", [[(64, 64)], [(256, 64), (64, 256)], [(300, 1000), (1000, 300), (33, 47)], [(7, 500)]])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("precise", [False, True])
def test_muon_step(sp, shapes, nesterov, precise):
    Gs = [update(8, *s) for s in shapes]
    Ms = [update(9, *s) for s in shapes]
    Ps = [update(10, *s, "gauss") for s in shapes]
    d = lambda v: [torch.from_numpy(x).cuda() for x in v]  # noqa: E731
    G, lrs, decays = d(Gs), [0.02 + 0.01 * k for k in range(len(shapes))], [0.1 * k for k in range(len(shapes))]
    M, P, W = ([Guarded(s, t) for s in shapes] for t in (torch.float32, torch.float32, torch.float16))
    for g, x in zip(M + P, Ms + Ps):
        g.t.copy_(torch.from_numpy(x))
    Wt = [w.t for w in W]
    Wt[-1] = None if len(W) > 1 else Wt[-1]
    sp.sp24_muon_step(G, [m.t for m in M], [p.t for p in P], Wt, lrs, decays, momentum=0.9, nesterov=nesterov, precise=precise)
    for g in M + P + W:
        g.check()
    for k, s in enumerate(shapes):
        assert torch.equal(G[k].cpu(), torch.from_numpy(Gs[k]))
        m, p, step = muon_ref(Gs[k], Ms[k], Ps[k], np.float32(lrs[k]), np.float32(decays[k]), np.float32(0.9), nesterov)
        got_m = M[k].t.cpu().numpy()
        assert (np.abs(got_m - m) <= 3 * 2.0 ** -24 * (np.abs(m) + np.abs(Gs[k]) + np.abs(Ms[k]))).all()
        # the update's own tolerance, and the roundings of P's three operations
        err = np.linalg.norm(P[k].t.cpu().numpy() - p)
        t = tol(torch.float32 if precise else torch.float16, s)
        assert err <= t * step + 3 * 2.0 ** -24 * (np.linalg.norm(Ps[k]) + step)
        if Wt[k] is not None:
            assert torch.equal(Wt[k], P[k].t.half())


def test_steps_of_the_ffn_weights_size(sp):
    """The widest layer's W2, a gated layer's W1, a long thin matrix and two ragged ones,
    each against float64 on the GPU."""
    for R, C in ((1600, 6400), (3200, 1600), (130, 70001), (2503, 4100), (5000, 2049)):
        gen = torch.Generator(device="cuda").manual_seed(R)
        G = torch.randn(R, C, generator=gen, device="cuda") * 1e-3
        X = G.double() / (G.double().norm() + 1e-7)
        X = X.t().contiguous() if R > C else X
        for _ in range(5):
            A = X @ X.t().contiguous()
            X = COEFFS[0] * X + (COEFFS[1] * A + COEFFS[2] * (A @ A)) @ X
        X = X.t() if R > C else X
        for out in (torch.float16, torch.float32):
            err = ((sp.sp24_orthogonalize(G, dtype=out).double() - X).norm() / X.norm()).item()
            assert err <= tol(out, (R, C))


def test_two_large_weights_of_one_call(sp):
    """Large tiles for the two together, and their steps: against single calls' float64."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    shapes = [(1600, 6400), (6400, 1600), (40, 70)]
    G, M, P = ([torch.randn(*s, generator=gen, device="cuda") * f for s in shapes] for f in (1e-3, 1e-2, 0.02))
    P0 = [p.double() for p in P]
    U = [g.double() + 0.95 * (0.95 * m.double() + g.double()) for g, m in zip(G, M)]
    W = [torch.empty_like(p, dtype=torch.float16) for p in P]
    sp.sp24_muon_step(G, M, P, W, [0.5] * 3, decays=[0.01] * 3, momentum=0.95)
    for u, p0, p, w, s in zip(U, P0, P, W, shapes):
        X = u / (u.norm() + 1e-7)
        X = X.t().contiguous() if s[0] > s[1] else X
        for _ in range(5):
            A = X @ X.t().contiguous()
            X = COEFFS[0] * X + (COEFFS[1] * A + COEFFS[2] * (A @ A)) @ X
        X = X.t() if s[0] > s[1] else X
        step = 0.5 * X.norm()
        err = (p.double() - (0.99 * p0 - 0.5 * X)).norm()
        # momentum and nesterov in fp32: the update's direction to 2^-22
        assert err <= tol(torch.float16, s) * step + 3 * 2.0 ** -24 * (p0.norm() + step)
        assert torch.equal(w, p.half())

"""GPU checks of the 2:4 products with bias, activation and residual, of the
input gradient through an activation with the bias gradient, and of the bias
gradient alone, against their formulas in float64.

Tolerances, from how each value comes about.  A sum of n products of fp16
values in fp32 is within n 2^-23 of the sum of magnitudes (2^-23 and not 2^-24:
a matrix instruction may truncate), n here K/2 + 2.  An activation passes an
error on by its slope (largest slopes: 1.13 for the smooth ones) and is itself
within 2^-19 (1 + |u|) of the exact value in absolute and, for u near 0 and
large, 2^-19 in relative terms; a slope is within 2^-18 (1 + |u|).  Results are
rounded once to fp16: 2^-11 relative, 2^-25 among subnormals.  Sums over T
tokens are within T 2^-23 of the sum of magnitudes of their terms, each of
which has its own error.
"""
import math

import pytest

from gpu_checks import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ACTS = ["none", "relu", "relu2", "gelu", "gelu_tanh", "silu"]
HALF, SUB, SUM, ACT, SLOPE = 2.0 ** -11, 2.0 ** -25, 2.0 ** -23, 2.0 ** -19, 2.0 ** -18


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def weight(sp, R, C, seed):
    """A weight, its forms, and its kept entries as a dense float64 matrix."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn(R, C, generator=gen, device="cuda") * (C / 2) ** -0.5).half()
    forms = sp.sp24_search_compress(W)
    bits = torch.tensor(sp.sp24_pattern_table(), device="cuda")[forms["idx"].long()]
    keep = (bits[:, :, None] >> torch.arange(16, device="cuda") & 1).reshape(R // 4, C // 4, 4, 4)
    keep = keep.transpose(1, 2).reshape(R, C).bool()
    return forms, torch.where(keep, W, 0).double(), gen


def act64(name, u):
    return {"none": lambda: u, "relu": lambda: torch.relu(u), "relu2": lambda: torch.relu(u).square(),
            "gelu": lambda: u * 0.5 * torch.erfc(-u * math.sqrt(0.5)), "silu": lambda: u * torch.sigmoid(u),
            "gelu_tanh": lambda: u * torch.sigmoid(math.sqrt(8 / math.pi) * (u + 0.044715 * u ** 3))}[name]()


def slope64(name, u):
    u = u.detach().requires_grad_()
    with torch.enable_grad():
        g, = torch.autograd.grad(act64(name, u).sum(), u)
    return g


def far(got, want, tol):
    """What is off by more than its tolerance, by how much at worst."""
    over = (got.double() - want).abs() / tol
    return float(over.max()) if over.numel() else 0.0


def check_fwd(sp, T, R, C, act, bias, residual, keep, seed=0, scale=1.0):
    forms, Ws, gen = weight(sp, R, C, seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    X = (rand(T, C) * scale).half()
    b = rand(R) if bias else None
    res = rand(T, R).half() if residual else None
    Y, U = Guarded((T, R), torch.float16), Guarded((T, R), torch.float16) if keep else None
    y, u = sp.sp24_spmm_fwd_act(X, forms["vals_row"], forms["meta_row"], R, C, act=act, bias=b, residual=res,
                                U=U.t if keep else False, out=Y.t)
    assert y.data_ptr() == Y.t.data_ptr() and (u is None) == (not keep)
    Y.check("Y")
    X, zero = X.double(), torch.zeros(1, dtype=torch.float64, device="cuda")
    b, res = (zero if v is None else v.double() for v in (b, res))
    want = X @ Ws.t() + b
    sum_err = (C / 2 + 2) * SUM * (X.abs() @ Ws.abs().t() + b.abs())
    if keep:
        U.check("U")
        assert far(u, want, sum_err + HALF * (want.abs() + sum_err) + SUB) <= 1
    a = act64(act, want)
    if act == "relu2":
        err = (2 * want.abs() + sum_err) * sum_err + SUM * a
    else:
        err = 1.13 * sum_err + (ACT * (1 + want.abs()) if act not in ("none", "relu") else 0)
    err = err + SUM * (a.abs() + res.abs())
    assert far(y, a + res, err + HALF * ((a + res).abs() + err) + SUB) <= 1


def check_bwd(sp, T, R, C, act, sums=True, seed=0):
    forms, Ws, gen = weight(sp, R, C, seed)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dY, U = rand(T, R).half(), (2 * rand(T, C)).half()
    dU, db = Guarded((T, C), torch.float16), Guarded((C,), torch.float32)
    got, gotb = sp.sp24_spmm_bwd_input_act(dY, forms["vals_col"], forms["meta_col"], R, C, None if act == "none" else U,
                                           act=act, dbias=db.t if sums else False, out=dU.t)
    dU.check("dU")
    dY, U = dY.double(), U.double()
    D = dY @ Ws
    sum_err = (R / 2 + 2) * SUM * (dY.abs() @ Ws.abs())
    slope = slope64(act, U)
    exact = act in ("none", "relu", "relu2")
    slope_err = SUM * slope.abs() if exact else SLOPE * (1 + U.abs())
    want = D * slope
    err = sum_err * (slope.abs() + slope_err) + D.abs() * slope_err + SUM * want.abs()
    assert far(got, want, err + HALF * (want.abs() + err) + SUB) <= 1
    if not sums:
        assert gotb is None
        return
    db.check("dbias")
    assert far(gotb, want.sum(0), err.sum(0) + T * SUM * (want.abs() + err).sum(0) + 1e-30) <= 1


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,R,C", [(1, 64, 64), (7, 48, 80), (16, 16, 16), (33, 320, 208), (200, 256, 1600)])
def test_forward(sp, act, T, R, C):
    check_fwd(sp, T, R, C, act, True, True, True)


@pytest.mark.parametrize("T,R,C", [(1, 1600, 6400), (1, 6400, 1600), (17, 1600, 6400), (24, 80, 4096), (32, 6400, 1600),
                                   (64, 112, 6400), (65, 1024, 320), (127, 64, 1616), (129, 336, 64), (257, 272, 128),
                                   (300, 6400, 192), (1000, 128, 48), (1021, 1024, 4096), (2500, 528, 656),
                                   (8192, 2064, 336)])
def test_forward_sizes(sp, T, R, C):
    check_fwd(sp, T, R, C, "gelu", True, False, T % 2 == 0, seed=T)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("T", [5, 600])
def test_forward_parts(sp, bias, residual, keep, T):
    check_fwd(sp, T, 272, 320, "silu", bias, residual, keep, seed=1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,R,C", [(1, 64, 64), (7, 80, 48), (16, 16, 16), (33, 208, 320), (200, 1600, 256)])
def test_backward(sp, act, T, R, C):
    check_bwd(sp, T, R, C, act)


@pytest.mark.parametrize("T,R,C", [(1, 1600, 6400), (19, 1616, 6400), (64, 64, 1600), (65, 320, 1024), (129, 64, 336),
                                   (257, 128, 272), (1021, 1024, 4096), (1000, 48, 128), (2500, 656, 528), (24, 6416, 528), (150, 6400, 80),
                                   (8100, 336, 2064)])
def test_backward_sizes(sp, T, R, C):
    check_bwd(sp, T, R, C, "gelu", seed=T)
    check_bwd(sp, T, R, C, "relu", sums=False, seed=T)


def test_products_alone_are_the_plain_calls(sp):
    """Without bias, activation and residual: the same products as sp24_spmm_fwd
    and sp24_spmm_bwd_input give, within two roundings."""
    for T in (3, 400):
        forms, Ws, gen = weight(sp, 512, 320, 5)
        X, dY = (torch.randn(T, n, generator=gen, device="cuda").half() for n in (320, 512))
        a, _ = sp.sp24_spmm_fwd_act(X, forms["vals_row"], forms["meta_row"], 512, 320)
        b = sp.sp24_spmm_fwd(X, forms["vals_row"], forms["meta_row"], 512, 320)
        assert far(a, b.double(), 2 * HALF * b.double().abs() + 1e-4) <= 1
        a, _ = sp.sp24_spmm_bwd_input_act(dY, forms["vals_col"], forms["meta_col"], 512, 320, None)
        b = sp.sp24_spmm_bwd_input(dY, forms["vals_col"], forms["meta_col"], 512, 320)
        assert far(a, b.double(), 2 * HALF * b.double().abs() + 1e-4) <= 1


@pytest.mark.parametrize("act", ACTS[1:])
def test_activations_over_their_range(sp, act):
    """A weight that copies its input (one kept value of 1 a row, the other 0),
    so U is any fp16 number; the backward with dY = 1 gives the slopes."""
    n = 16384
    u = torch.cat([torch.linspace(-12, 12, n - 2048), torch.linspace(-0.01, 0.01, 2048 - 8),
                   torch.tensor([0.0, -0.0, 6e-8, -6e-8, 200.0, -200.0, 65504.0, -65504.0])]).half().cuda()
    X = torch.zeros(n, 16, dtype=torch.float16, device="cuda")
    X[:, 0] = u
    W = torch.zeros(16, 16, dtype=torch.float16, device="cuda")
    W[0, 0] = 1.0
    f = sp.sp24_search_compress(W)
    Y, U = sp.sp24_spmm_fwd_act(X, f["vals_row"], f["meta_row"], 16, 16, act=act, U=True)
    assert torch.equal(U[:, 0], u + 0.0)   # a sum: -0 becomes 0
    want = act64(act, u.double())
    big = want.abs() > 65504 * (1 + 2.0 ** -12)
    assert torch.isinf(Y[:, 0][big]).all()
    # relative all over the range, far negative u too, where GELU and SILU vanish
    tol = (HALF + 2.0 ** -16) * want.abs() + SUB + 2.0 ** -30
    assert far(Y[:, 0][~big], want[~big], tol[~big]) <= 1
    dY = torch.zeros(n, 16, dtype=torch.float16, device="cuda")
    dY[:, 0] = 1.0
    Uin = torch.zeros(n, 16, dtype=torch.float16, device="cuda")
    Uin[:, 0] = u
    dU, _ = sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], 16, 16, Uin, act=act)
    want = slope64(act, u.double()).nan_to_num()
    fine = want.abs() < 65504
    tol = HALF * want.abs() + SUB + SLOPE * (1 + u.double().abs().clamp(max=16))
    assert far(dU[:, 0][fine], want[fine], tol[fine]) <= 1


def test_slopes_match_differences(sp):
    """(act(u + h) - act(u - h)) / 2h through the forward call's fp16 results is
    too coarse; in float64 the slopes' reference is held to its differences."""
    u = torch.linspace(-6, 6, 1001, dtype=torch.float64, device="cuda")
    h = 1e-5
    for act in ACTS:
        near = (act64(act, u + h) - act64(act, u - h)) / (2 * h)
        keep = u.abs() > 2 * h if act in ("relu", "relu2") else torch.ones_like(u, dtype=torch.bool)
        assert (near - slope64(act, u))[keep].abs().max() < 1e-8


def test_infinite_and_nan(sp):
    f, Ws, gen = weight(sp, 64, 64, 9)
    for T in (4, 300):
        X = torch.randn(T, 64, generator=gen, device="cuda").half()
        X[1, 5] = float("nan")
        X[2] = float("inf")
        for act in ACTS:
            Y, _ = sp.sp24_spmm_fwd_act(X, f["vals_row"], f["meta_row"], 64, 64, act=act)
            used = (Ws[:, 5] != 0)
            assert torch.isnan(Y[1][used]).all()
            others = torch.tensor([t for t in range(T) if t not in (1, 2)], device="cuda")
            assert torch.isfinite(Y[others]).all()
    bias = torch.zeros(64, device="cuda")
    bias[:3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    zero = torch.zeros(2, 64, dtype=torch.float16, device="cuda")
    for act, low in zip(ACTS, (-math.inf, 0.0, 0.0, 0.0, math.nan, math.nan)):
        Y, _ = sp.sp24_spmm_fwd_act(zero, f["vals_row"], f["meta_row"], 64, 64, act=act, bias=bias)
        got = Y[0, :3].tolist()
        assert got[0] == math.inf and math.isnan(got[2])
        assert math.isnan(got[1]) if math.isnan(low) else got[1] == low


def test_slopes_at_infinities_and_nan(sp):
    """What the backward makes of U where the forward gave inf or NaN: no NaN of U
    is lost, and no infinity turns one activation's limit into another's."""
    R, C = 64, 64
    f, Ws, gen = weight(sp, R, C, 9)
    for T in (3, 40, 40000):   # thin, shared and whole tiles
        dY = torch.ones(T, R, dtype=torch.float16, device="cuda")
        U = torch.zeros(T, C, dtype=torch.float16, device="cuda")
        U[:, 0], U[:, 1], U[:, 2] = math.nan, math.inf, -math.inf
        d, _ = sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], R, C, None)
        assert torch.isfinite(d).all() and (d[0, :3] != 0).all()
        for act in ACTS[1:]:
            got, db = sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], R, C, U, act=act)
            if act == "relu":
                assert torch.equal(got[:, 0], d[:, 0])
            else:
                assert torch.isnan(got[:, 0]).all() and torch.isnan(db[0])
            if act in ("relu", "gelu"):
                assert torch.equal(got[:, 1], d[:, 1]) and (got[:, 2] == 0).all()
            elif act == "relu2":
                assert torch.isinf(got[:, 1]).all() and (got[:, 2] == 0).all()
            else:
                assert torch.isnan(got[:, 1:3]).all()
            assert torch.isfinite(got[:, 3:]).all() and torch.isfinite(db[3:]).all()


def test_no_tokens_and_no_width(sp):
    f, _, _ = weight(sp, 64, 32, 2)
    Y, U = sp.sp24_spmm_fwd_act(torch.empty(0, 32, dtype=torch.float16, device="cuda"), f["vals_row"], f["meta_row"], 64,
                                32, act="gelu", U=True)
    assert Y.shape == (0, 64) and U.shape == (0, 64)
    db = torch.full((32,), 7.0, device="cuda")
    sp.sp24_spmm_bwd_input_act(torch.empty(0, 64, dtype=torch.float16, device="cuda"), f["vals_col"], f["meta_col"], 64,
                               32, torch.empty(0, 32, dtype=torch.float16, device="cuda"), act="gelu", dbias=db)
    assert (db == 0).all()
    db = sp.sp24_bias_grad(torch.empty(0, 48, dtype=torch.float16, device="cuda"), dbias=torch.ones(48, device="cuda"))
    assert (db == 0).all()
    # a reduction of no entries leaves the bias and the residual
    none = [torch.empty(32, 0, dtype=d, device="cuda") for d in (torch.float16, torch.int16)]
    bias, res = torch.arange(32.0, device="cuda"), torch.ones(3, 32, dtype=torch.float16, device="cuda")
    Y, _ = sp.sp24_spmm_fwd_act(torch.empty(3, 0, dtype=torch.float16, device="cuda"), *none, 32, 0, bias=bias, residual=res)
    assert torch.equal(Y, (bias + 1).half().expand(3, 32))


@pytest.mark.parametrize("T,R,C", [(9, 320, 256), (700, 320, 256), (40, 1024, 1024)])
def test_in_place(sp, T, R, C):
    f, _, gen = weight(sp, R, C, 3)
    X, dY, res, U = (torch.randn(T, n, generator=gen, device="cuda").half() for n in (C, R, R, C))
    want, _ = sp.sp24_spmm_fwd_act(X, f["vals_row"], f["meta_row"], R, C, act="relu", residual=res)
    got, _ = sp.sp24_spmm_fwd_act(X, f["vals_row"], f["meta_row"], R, C, act="relu", residual=res, out=res)
    assert torch.equal(got, want)
    want, wb = sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], R, C, U, act="silu")
    got, gb = sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], R, C, U, act="silu", out=U)
    assert torch.equal(got, want) and torch.equal(gb, wb)


def test_workspace(sp):
    """A call writes nothing past the workspace that it asked for."""
    T, R, C = 150, 528, 6416
    f, _, gen = weight(sp, R, C, 6)
    X, dY, U, long = (torch.randn(t, n, generator=gen, device="cuda").half() for t, n in ((T, C), (T, R), (T, C), (2000, R)))
    for need, call in (
            (sp.lib().sp24_spmm_fwd_act_workspace(T, R, C),
             lambda w: sp.sp24_spmm_fwd_act(X, f["vals_row"], f["meta_row"], R, C, act="gelu", workspace=w)),
            (sp.lib().sp24_spmm_bwd_input_act_workspace(T, R, C),
             lambda w: sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], R, C, U, act="gelu", workspace=w)),
            (sp.lib().sp24_bias_grad_workspace(2000, R), lambda w: (sp.sp24_bias_grad(long, workspace=w),))):
        assert need > 0
        ws = Guarded((need,), torch.uint8)
        got = call(ws.t)
        ws.check("workspace")
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, call(None)))
        with pytest.raises(ValueError):
            call(ws.t[:need - 16])


@pytest.mark.parametrize("T,R", [(1, 16), (1, 6400), (63, 48), (64, 512), (65, 528), (517, 1600), (1024, 80), (1025, 80), (4096, 1024),
                                 (16384, 6400), (100000, 16)])
def test_bias_grad(sp, T, R):
    gen = torch.Generator(device="cuda").manual_seed(T + R)
    dY = torch.randn(T, R, generator=gen, device="cuda").half()
    db = Guarded((R,), torch.float32)
    got = sp.sp24_bias_grad(dY, dbias=db.t)
    db.check()
    assert far(got, dY.double().sum(0), T * 2.0 ** -24 * dY.double().abs().sum(0)) <= 1
    assert torch.equal(got, sp.sp24_bias_grad(dY))


def test_streams_and_graphs(sp):
    """Another stream, and a captured pass replayed over new inputs with eager
    work between, give the eager bits."""
    T, d, h = 700, 256, 1024
    (f1, _, gen), (f2, _, _) = weight(sp, h, d, 1), weight(sp, d, h, 2)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    X, dY, b1, b2 = rand(T, d).half(), rand(T, d).half(), rand(h), rand(d)

    def both(x):
        H, U = sp.sp24_spmm_fwd_act(x, f1["vals_row"], f1["meta_row"], h, d, act="gelu", bias=b1, U=True)
        Y, _ = sp.sp24_spmm_fwd_act(H, f2["vals_row"], f2["meta_row"], d, h, bias=b2, residual=x)
        dU, db1 = sp.sp24_spmm_bwd_input_act(dY, f2["vals_col"], f2["meta_col"], d, h, U, act="gelu")
        return H, Y, dU, db1, sp.sp24_bias_grad(dY)

    want = both(X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(X)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = X.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(x)
    for k in range(4):
        x.copy_(X * (k + 1))
        graph.replay()
        eager = both(x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), k


def test_many_tokens(sp):
    """Offsets past 2^31 bytes of the inputs and outputs."""
    T, R, C = 350_000, 64, 6400
    forms, Ws, gen = weight(sp, R, C, 4)
    U = torch.randn(T, C, generator=gen, device="cuda").half()
    dY = torch.randn(T, R, generator=gen, device="cuda").half()
    dU, db = sp.sp24_spmm_bwd_input_act(dY, forms["vals_col"], forms["meta_col"], R, C, U, act="relu")
    Y, _ = sp.sp24_spmm_fwd_act(U, forms["vals_row"], forms["meta_row"], R, C)
    total = torch.zeros(C, dtype=torch.float64, device="cuda")
    mag = torch.zeros(C, dtype=torch.float64, device="cuda")
    for a in range(0, T, 50_000):
        s = slice(a, a + 50_000)
        D = (dY[s].double() @ Ws) * (U[s] > 0)
        err = (R / 2 + 2) * SUM * (dY[s].double().abs() @ Ws.abs())
        assert far(dU[s], D, err + HALF * (D.abs() + err) + SUB) <= 1
        total += D.sum(0)
        mag += (D.abs() + err).sum(0)
        want = U[s].double() @ Ws.t()
        err = (C / 2 + 2) * SUM * (U[s].double().abs() @ Ws.abs().t())
        assert far(Y[s], want, err + HALF * (want.abs() + err) + SUB) <= 1
    assert far(db, total, (T + R / 2 + 2) * SUM * mag) <= 1

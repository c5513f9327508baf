"""The plain 2:4 layer (SparseFFN), AdamW over a model's tensors and the step from
token ids to new weights around them (TokenMLP): each against the same
composition in float64 on what the calls before it returned, whole steps
captured and replayed, and a short training run.

Tolerances.  fp16 outputs: 2^-11 of the value, 2^-25 among subnormals, and the
sums' errors, n 2^-23 of the magnitudes for n terms; GELU passes an error on by
at most 1.13 and adds 2^-19 (1 + |u|), its slope 2^-18 (1 + |u|).
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
HALF, SUB, SUM = 2.0 ** -11, 2.0 ** -25, 2.0 ** -23


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def pruned(sp, W):
    R, C = W.shape
    bits = torch.tensor(sp.sp24_pattern_table(), device="cuda")[sp.sp24_mask_search(W).long()]
    keep = (bits[:, :, None] >> torch.arange(16, device="cuda") & 1).reshape(R // 4, C // 4, 4, 4)
    return torch.where(keep.transpose(1, 2).reshape(R, C).bool(), W, 0).double()


def parts(gen, V, d, h):
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return (rand(V, d), (rand(h, d) * d ** -0.5).half(), rand(h) * 0.1, (rand(d, h) * h ** -0.5).half(), rand(d) * 0.1)


def near(got, want, err):
    err = err + HALF * (want.abs() + err) + SUB
    assert ((got.double() - want).abs() <= err).all(), float(((got.double() - want).abs() / err).max())


def gelu(u):
    return u * 0.5 * torch.erfc(-u * math.sqrt(0.5))


def slope(u):
    return 0.5 * torch.erfc(-u * math.sqrt(0.5)) + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("T,d,h,residual", [(1, 64, 256, True), (77, 80, 208, False), (600, 128, 512, True),
                                            (1500, 320, 1280, True)])
def test_layer(sp, T, d, h, residual):
    from structured_sparse_transformer_amd.ffn import SparseFFN
    gen = torch.Generator(device="cuda").manual_seed(T)
    _, W1, b1, W2, b2 = parts(gen, 1, d, h)
    layer = SparseFFN(W1, b1, W2, b2, residual=residual, decay=0.25)
    with pytest.raises(RuntimeError):
        layer(torch.zeros(T, d, dtype=torch.float16, device="cuda"))
    layer.refresh()
    X, dY = (torch.randn(T, d, generator=gen, device="cuda").half() for _ in range(2))
    Y, saved = layer.forward(X)
    assert torch.equal(layer(X), Y)
    P1, P2, x, dy = pruned(sp, W1), pruned(sp, W2), X.double(), dY.double()
    U = x @ P1.t() + b1.double()
    err = (d / 2 + 2) * SUM * (x.abs() @ P1.abs().t() + b1.double().abs())
    near(saved.U, U, err)
    near(saved.Hg, gelu(U), 1.13 * err + 2.0 ** -19 * (1 + U.abs()))
    H = saved.Hg.double()
    want = H @ P2.t() + b2.double() + (x if residual else 0)
    near(Y, want, (h / 2 + 3) * SUM * (H.abs() @ P2.abs().t() + b2.double().abs() + x.abs()))
    dX, dW1, db1, dW2, db2 = layer.backward(dY, saved)
    assert torch.equal(db2, sp.sp24_bias_grad(dY))
    u = saved.U.double()
    dU, kept = sp.sp24_spmm_bwd_input_act(dY, layer.forms[1]["vals_col"], layer.forms[1]["meta_col"], d, h, saved.U, act="gelu")
    assert torch.equal(kept, db1)
    near(dU, (dy @ P2) * slope(u), (d / 2 + 2) * SUM * (dy.abs() @ P2.abs()) * 1.13 + (dy @ P2).abs() * 2.0 ** -18 * (1 + u.abs()))
    D = dU.double()
    near(dX, D @ P1 + (dy if residual else 0), (h / 2 + 3) * SUM * (D.abs() @ P1.abs() + dy.abs()))
    for dW, a, b, W, P in ((dW1, D, x, W1, P1), (dW2, dy, H, W2, P2)):
        want = a.t() @ b + 0.25 * (W.double() - P)
        assert ((dW.double() - want).abs() <= (T + 2) * SUM * (a.abs().t() @ b.abs() + W.double().abs())).all()


def test_refusals(sp):
    from structured_sparse_transformer_amd.adamw import AdamW
    from structured_sparse_transformer_amd.ffn import SparseFFN
    gen = torch.Generator(device="cuda").manual_seed(0)
    _, W1, b1, W2, b2 = parts(gen, 1, 64, 128)
    for bad in ((W1, b2, W2, b1), (W1, b1, W1, b2)):
        with pytest.raises(ValueError):
            SparseFFN(*bad)
    with pytest.raises(ValueError):
        SparseFFN(W1, b1, W2, b2, act="tanh")
    with pytest.raises(ValueError):
        AdamW([b1], bits=16)
    opt = AdamW([b1, b2], max_norm=1.0)
    with pytest.raises(ValueError):
        opt.step([b1])
    assert int(opt.control.abs().sum()) == 0
    with pytest.raises(ValueError):
        AdamW([b1]).step([b2])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("guard", [dict(), dict(max_norm=0.5), dict(loss_scale=8.0), dict(max_norm=1e9, loss_scale=2.0)])
def test_optimiser(sp, bits, guard):
    """Three steps against the formulas in float64, from the states as held."""
    from structured_sparse_transformer_amd.adamw import AdamW
    gen = torch.Generator(device="cuda").manual_seed(bits)
    shapes = [(50, 70), (7,), (64, 64), (0,), (1, 1)]
    P = [torch.randn(*s, generator=gen, device="cuda") for s in shapes]
    W = [p.half() if k % 2 == 0 else None for k, p in enumerate(P)]
    opt = AdamW(P, W, lr=1e-2, weight_decay=0.1, bits=bits, **guard)
    for t in range(1, 4):
        if t == 3:
            opt.set_lr(3e-3)
        lr = 1e-2 if t < 3 else 3e-3
        G = [torch.randn(*s, generator=gen, device="cuda") for s in shapes]
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in G)) / guard.get("loss_scale", 1.0)
        factor = min(1.0, guard.get("max_norm", math.inf) / norm) / guard.get("loss_scale", 1.0)
        if bits == 32:
            held = [(m.double().clone(), v.double().clone()) for m, v in opt.states]
        else:
            held = [(sp.sp24_state8_values(a, b).double(), sp.sp24_state8_values(c, e, root=True).double().square())
                    for a, b, c, e in opt.states]
        before = [p.double().clone() for p in P]
        opt.step(G)
        for p, p0, w, g, (m, v) in zip(P, before, W, G, held):
            g = g.double() * factor
            m, v = 0.9 * m + 0.1 * g, 0.999 * v + 0.001 * g * g
            step = lr * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
            scale = lr / (1 - 0.9 ** t) / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
            # 6 roundings of M's terms (|m| + 0.2 |g| bounds them), 30 of the step's, 3 of P's
            tol = 2.0 ** -24 * (6 * scale * (m.abs() + 0.2 * g.abs()) + 30 * step.abs() + 3 * p0.abs())
            assert ((p.double() - ((1 - lr * 0.1) * p0 - step)).abs() <= tol).all()
            assert w is None or torch.equal(w, p.half())


@pytest.mark.parametrize("guard", [{}, {"max_norm": 1.0}])
def test_a_refused_step_is_not_counted(sp, guard):
    from structured_sparse_transformer_amd.adamw import AdamW
    P = [torch.zeros(70, device="cuda"), torch.zeros(5, 3, device="cuda")]
    optimizer = AdamW(P, **guard)
    good = [torch.ones_like(p) for p in P]
    for bad in (good[:1], [good[0], good[1][:4]], [good[0], good[1].half()], [g.cpu() for g in good], good[::-1]):
        with pytest.raises(ValueError):
            optimizer.step(bad)
    steps = lambda: int(sp.control_values(optimizer.control)["step"]) if guard else optimizer.steps  # noqa: E731
    assert steps() == 0 and not any(p.any() for p in P)
    optimizer.step(good)
    assert steps() == 1 and all(p.all() for p in P)


def test_a_captured_step_counts_on(sp):
    """Refused where t would be a constant of the graph; with no more than an
    infinite max_norm it counts, and gives the eager steps' bits."""
    from structured_sparse_transformer_amd.adamw import AdamW
    ends = []
    G = [torch.ones(70, device="cuda")]
    for how in ("eager", "captured", "plain"):
        P = [torch.zeros(70, device="cuda")]
        optimizer = AdamW(P, max_norm=None if how == "plain" else math.inf)
        graph = torch.cuda.CUDAGraph()
        if how == "plain":
            with torch.cuda.graph(graph):
                G[0].add_(0.0)
                with pytest.raises(RuntimeError, match="captured"):
                    optimizer.step(G)
            assert optimizer.steps == 0
            continue
        if how == "captured":
            with torch.cuda.graph(graph):
                optimizer.step(G)
        for _ in range(4):
            graph.replay() if how == "captured" else optimizer.step(G)
            torch.cuda.synchronize()
        assert int(sp.control_values(optimizer.control)["step"]) == 4
        ends.append(P[0])
    assert torch.equal(*ends)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_captured_and_replayed(sp, bits):
    """Whole steps, tokens to new weights, captured and replayed over new tokens
    with eager work between: the eager steps' bits."""
    from structured_sparse_transformer_amd.token_step import TokenMLP
    V, d, h, T = 300, 64, 256, 500
    ends = []
    for captured in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(5)
        model = TokenMLP(*parts(gen, V, d, h), lr=1e-2, bits=bits, max_norm=1.0, loss_scale=4.0)
        ids = torch.zeros(T, dtype=torch.int64, device="cuda")
        target = torch.zeros(T, d, dtype=torch.float16, device="cuda")

        def step():
            Y, saved = model.forward(ids)
            model.update(model.backward(ids, (4.0 * (Y.float() - target.float()) / T).half(), saved))

        step()   # the streams and forms exist before the capture
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for k in range(5):
            ids.copy_(torch.randint(-1, V, (T,), generator=gen, device="cuda"))
            target.copy_(torch.randn(T, d, generator=gen, device="cuda").half())
            if k == 3:
                target[7, 7] = math.nan   # a step that is left out
            graph.replay() if captured else step()
            model.layer(target[:3])
            torch.cuda.synchronize()
        assert int(sp.control_values(model.optimizer.control)["step"]) == 5
        ends.append([t for part in model.optimizer.plan.tensors for t in part if t is not None] + [model.layer.flips])
    assert all(torch.equal(a, b) for a, b in zip(*ends))
    assert all(torch.isfinite(t.float()).all() for t in ends[0])


def test_training_learns(sp):
    from structured_sparse_transformer_amd.token_step import train_plain
    for bits in (8, 32):
        losses = train_plain(steps=30, bits=bits)
        assert all(math.isfinite(v) for v in losses)


def test_gradients_match_differences(sp):
    """The loss's differences along random directions of b1 and b2, in fp16
    outputs' precision, against the gradients."""
    from structured_sparse_transformer_amd.ffn import SparseFFN
    gen = torch.Generator(device="cuda").manual_seed(9)
    _, W1, b1, W2, b2 = parts(gen, 1, 64, 256)
    layer = SparseFFN(W1, b1, W2, b2)
    layer.refresh()
    X, dY = (torch.randn(400, 64, generator=gen, device="cuda").half() for _ in range(2))
    _, saved = layer.forward(X)
    _, _, db1, _, db2 = layer.backward(dY, saved)
    loss = lambda: float((layer(X).double() * dY.double()).sum())  # noqa: E731
    for b, db in ((b1, db1), (b2, db2)):
        way = torch.randn(b.shape, generator=gen, device="cuda")
        start, eps = b.clone(), 2.0 ** -4
        b.copy_(start + eps * way)
        up = loss()
        b.copy_(start - eps * way)
        down = loss()
        b.copy_(start)
        slope_ = float((db.double() * way.double()).sum())
        # 25600 outputs of about unit size, each rounded to fp16 twice (its own rounding, and H's over 128 terms of
        # size 256^-0.5): noise 1.5 (400 64)^0.5 2^-12 / eps; the third derivative's part, eps^2 / 6 of terms as large
        noise = 6 * 1.5 * 160 * 2.0 ** -12 / eps
        assert abs((up - down) / (2 * eps) - slope_) <= noise + eps * eps * float((dY.double().abs().sum()) * 0.1)

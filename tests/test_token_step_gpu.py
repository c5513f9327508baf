"""The step from token ids to new weights (token_step.py): its gradients and new
weights against the same composition in float64 on what the layer returned, and
a short training run."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def newton_schulz(G, steps=5, a=3.4445, b=-4.7750, c=2.0315):
    X = G.double().cpu()
    X = X / (X.norm() + 1e-7)
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    for _ in range(steps):
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    return X.t() if tall else X


def test_one_step():
    from structured_sparse_transformer_amd.token_step import TokenFFN
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    V, d, h, T = 300, 64, 96, 500
    table, W1, W2 = rand(V, d), (rand(2 * h, d) * 0.1).half(), (rand(d, h) * 0.1).half()
    start = [w.float().cpu().double() for w in (W1, W2)]
    m = TokenFFN(table, W1, W2, scale=0.5, decay=0.01, lr=1e-2, momentum=0.9, weight_decay=0.1, precise=True)
    ids = torch.randint(-1, V, (T,), generator=gen, device="cuda")
    Y, saved = m.forward(ids)
    # the embedding's rows: one fp32 product, rounded to fp16
    ok = ids >= 0
    want = torch.where(ok[:, None], table[ids.clamp(min=0)].double() * 0.5, 0.0)
    assert ((saved.X.double() - want).abs() <= (2.0 ** -11 + 2.0 ** -24) * want.abs() + 2.0 ** -25).all()
    dY = rand(T, d).half()
    dX, dW1, dW2 = m.layer.backward(dY, saved)
    grads = m.backward(ids, dY, saved)
    assert torch.equal(grads[0], dW1) and torch.equal(grads[1], dW2)
    # the table's gradient: fp32 sums of at most T terms
    ref, mag = torch.zeros(V, d, dtype=torch.float64, device="cuda"), torch.zeros(V, d, dtype=torch.float64, device="cuda")
    ref.index_add_(0, ids[ok], dX[ok].double() * 0.5)
    mag.index_add_(0, ids[ok], dX[ok].double().abs() * 0.5)
    assert ((m.dtable.double() - ref).abs() <= (T + 2) * 2.0 ** -24 * mag).all()
    before, dtable = table.clone(), m.dtable.clone()
    m.update(grads, table_lr=0.25)
    assert torch.equal(table, before.add(dtable, alpha=-0.25)) and (m.dtable == 0).all()
    # the first step's momentum is the gradient, the update that of 1.9 G
    for P, W, G, w0 in zip(m.optimizer.masters, (W1, W2), grads, start):
        lr = 1e-2 * 0.2 * math.sqrt(max(G.shape))
        X = newton_schulz(G.double() * (1 + float(torch.tensor(0.9))))
        want = (1 - 1e-3) * w0 - lr * X
        # orthogonalised to fp32 accuracy (at most 3e-5 of the update's norm), P's own roundings
        err = (P.cpu().double() - want).norm()
        assert err <= 3e-5 * lr * X.norm() + 3 * 2.0 ** -24 * (w0.norm() + lr * X.norm())
        assert torch.equal(W, P.half())
    # the layer runs on the new weights' masks
    from structured_sparse_transformer_amd import sp24
    for W, forms in zip((W1, W2), m.layer.forms):
        assert torch.equal(forms["idx"], sp24.sp24_mask_search(W))


def test_more_weights_than_a_call_takes():
    from structured_sparse_transformer_amd.muon import Muon
    gen = torch.Generator(device="cuda").manual_seed(4)
    shapes = [(32, 16 * (k + 1)) for k in range(11)]
    weights = [(torch.randn(*s, generator=gen, device="cuda") * 0.1).half() for s in shapes]
    singles = [w.clone() for w in weights]
    grads = [torch.randn(*s, generator=gen, device="cuda") for s in shapes]
    Muon(weights, lr=0.01).step(grads)
    for w, one, g in zip(weights, singles, grads):
        Muon([one], lr=0.01).step([g])
        assert torch.equal(w, one)


def test_training_learns():
    from structured_sparse_transformer_amd.token_step import train
    losses = train(steps=60)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * losses[0]

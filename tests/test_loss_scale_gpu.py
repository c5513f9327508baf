"""The masked decay term of the plain layer's gradients beside a loss scale: the
term is of the unscaled gradient (dW = dY^T H + decay (1 - M) W), so in the
gradients of a loss multiplied by s it stands as s decay (1 - M) W, and after an
update nothing of s is left.

Tolerances.  Without a gradient from the outputs, dW is one product of the decay,
rounded to fp32, and an fp16 entry: 2^-24 for either rounding.  Otherwise a sum
of T products in fp32 and that term, (T + 2) 2^-23 of the magnitudes.  Scales by
a power of two are exact everywhere.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
V, D, H, T = 50, 64, 256, 150


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def masked(sp, W):
    """(1 - M) W in float64."""
    R, C = W.shape
    bits = torch.tensor(sp.sp24_pattern_table(), device="cuda")[sp.sp24_mask_search(W).long()]
    keep = (bits[:, :, None] >> torch.arange(16, device="cuda") & 1).reshape(R // 4, C // 4, 4, 4)
    return torch.where(keep.transpose(1, 2).reshape(R, C).bool(), 0, W).double()


def model_of(**more):
    from structured_sparse_transformer_amd.token_step import TokenMLP
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    model = TokenMLP(rand(V, D), (rand(H, D) * D ** -0.5).half(), rand(H), (rand(D, H) * H ** -0.5).half(), rand(D),
                     lr=1e-2, weight_decay=0.0, **more)
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    return model, ids, rand(T, D)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 10, 1000.0])
def test_gradients_hold_the_scaled_term(sp, scale):
    model, ids, dY = model_of(decay=0.25, loss_scale=scale)
    terms = [masked(sp, model.layer.W1), masked(sp, model.layer.W2)]
    _, saved = model.forward(ids)
    _, dW1, db1, dW2, db2 = model.backward(ids, torch.zeros(T, D, dtype=torch.float16, device="cuda"), saved)
    assert not db1.any() and not db2.any()
    for dW, term in zip((dW1, dW2), terms):
        want = scale * 0.25 * term
        assert ((dW.double() - want).abs() <= 2.0 ** -23 * want.abs()).all()
    dY = (dY * 0.01 * scale).half()
    _, _, _, dW2, _ = model.backward(ids, dY, saved)
    a, b = dY.double(), saved.Hg.double()
    err = (T + 2) * 2.0 ** -23 * (a.abs().t() @ b.abs() + scale * 0.25 * terms[1].abs())
    assert ((dW2.double() - (a.t() @ b + scale * 0.25 * terms[1])).abs() <= err).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_an_update_has_nothing_of_the_scale(sp, bits, max_norm):
    """The term alone makes the gradients: masters, copies and states after three
    updates are the unscaled run's, bit for bit."""
    ends = []
    for scale in (1.0, 2.0 ** 10):
        model, ids, _ = model_of(decay=0.25, loss_scale=scale, bits=bits, max_norm=max_norm)
        start = [W.clone() for W in (model.layer.W1, model.layer.W2)]
        for _ in range(3):
            _, saved = model.forward(ids)
            model.update(model.backward(ids, torch.zeros(T, D, dtype=torch.float16, device="cuda"), saved))
        assert not any(torch.equal(W, W0) for W, W0 in zip((model.layer.W1, model.layer.W2), start))
        ends.append([t for part in model.optimizer.plan.tensors for t in part if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*ends))


def test_the_layer_alone(sp):
    """The layer takes the scale of the loss that its dY is of."""
    model, ids, _ = model_of(decay=0.25)
    _, saved = model.forward(ids)
    zero = torch.zeros(T, D, dtype=torch.float16, device="cuda")
    once, eight = model.layer.backward(zero, saved), model.layer.backward(zero, saved, loss_scale=8.0)
    for a, b in zip(once, eight):
        assert torch.equal(a * 8.0, b)
    assert once[1].any() and once[3].any()

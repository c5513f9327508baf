"""The short training run of the plain layer, step by step: every one of its steps
is counted, scales and clips the gradients as their norm says, and moves every
parameter by AdamW's formula from the states as held; the fp16 copies are the
masters rounded, and the layer's 2:4 forms are of the new copies.

Tolerances of a parameter: 6 roundings of M's terms (|m| + 0.2 |g| bounds them) over
the root, 30 of the step's, 3 of P's, 2^-24 each.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
LR, B1, B2, DECAY, SCALE, MOST = 1e-2, 0.9, 0.999, 0.01, 2.0 ** 10, 1.0


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


@pytest.mark.parametrize("bits", [32, 8])
def test_every_step_is_taken(sp, bits, monkeypatch):
    from structured_sparse_transformer_amd import token_step
    counts = []

    class Checked(token_step.TokenMLP):
        def update(self, grads):
            opt = self.optimizer
            t = len(counts) + 1
            before = [p.double() for p in opt.params]
            if bits == 32:
                held = [(m.double(), v.double()) for m, v in opt.states]
            else:
                held = [(sp.sp24_state8_values(a, b).double(), sp.sp24_state8_values(c, e, root=True).double().square())
                        for a, b, c, e in opt.states]
            super().update(grads)
            counts.append(int(sp.control_values(opt.control)["step"]))
            assert int(sp.control_values(opt.control)["skip"]) == 0
            norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads)) / SCALE
            assert norm > 0 and all(g.any() for g in grads)
            factor = min(1.0, MOST / norm) / SCALE
            for p, p0, w, g, (m, v), decay in zip(opt.params, before, opt.copies, grads, held, (0, DECAY, 0, DECAY, 0)):
                g = g.double() * factor
                m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
                scale = LR / (1 - B1 ** t) / ((v / (1 - B2 ** t)).sqrt() + 1e-8)
                step = scale * m
                tol = 2.0 ** -24 * (6 * scale * (m.abs() + 0.2 * g.abs()) + 30 * step.abs() + 3 * p0.abs())
                assert ((p.double() - ((1 - LR * decay) * p0 - step)).abs() <= tol).all()
                assert not torch.equal(p.double(), p0) and (w is None or torch.equal(w, p.half()))
            for W, forms in zip((self.layer.W1, self.layer.W2), self.layer.forms):
                fresh = sp.sp24_search_compress(W)
                assert all(torch.equal(fresh[k], forms[k]) for k in ("idx", "vals_row", "meta_row", "vals_col", "meta_col"))

    monkeypatch.setattr(token_step, "TokenMLP", Checked)
    losses = token_step.train_plain(steps=6, bits=bits)
    assert counts == [1, 2, 3, 4, 5, 6] and len(losses) == 6 and all(math.isfinite(v) for v in losses)

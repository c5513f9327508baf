"""The optimiser over more weights than one call takes: a gradient that is
refused leaves every weight as it was."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BAD = {"type": lambda g: g.half(), "shape": lambda g: g[:-1], "strides": lambda g: torch.cat([g, g], 1)[:, ::2],
       "alignment": lambda g: torch.cat([g.flatten()[:1], g.flatten()])[1:].view_as(g), "host": lambda g: g.cpu(),
       "none": lambda g: None}


@pytest.mark.parametrize("fault", BAD)
def test_a_refused_gradient_changes_nothing(fault):
    from structured_sparse_transformer_amd.muon import Muon
    gen = torch.Generator(device="cuda").manual_seed(6)
    weights = [(torch.randn(32, 48, generator=gen, device="cuda") * 0.1).half() for _ in range(11)]
    grads = [torch.randn(32, 48, generator=gen, device="cuda") for _ in weights]
    m = Muon(weights, lr=0.01)
    m.step(grads)
    before = [t.clone() for t in m.weights + m.masters + m.momenta]
    wrong = list(grads)
    wrong[9] = BAD[fault](grads[9])
    with pytest.raises(ValueError):
        m.step(wrong)
    assert all(torch.equal(a, b) for a, b in zip(before, m.weights + m.masters + m.momenta))
    m.step(grads)
    assert not any(torch.equal(a, b) for a, b in zip(before, m.weights + m.masters + m.momenta))

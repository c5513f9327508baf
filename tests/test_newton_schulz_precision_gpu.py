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

"""Where U <= 0 the backward through RELU and RELU2 is 0 whatever the product is,
also an infinite or NaN one; where U > 0, and through the other activations, such a
product comes through, into the bias gradient too."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


@pytest.mark.parametrize("T", [3, 40, 40000])   # thin, shared and whole tiles
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_products_that_are_not_finite(sp, T, bad):
    W = torch.ones(64, 64, dtype=torch.float16, device="cuda")   # two of four of each kept, none zero
    f = sp.sp24_search_compress(W)
    dY = torch.ones(T, 64, dtype=torch.float16, device="cuda")
    dY[1] = bad
    U = torch.ones(T, 64, dtype=torch.float16, device="cuda")
    U[:, 1::2] = -1.0
    U[:, 3] = 0.0
    others = torch.arange(T, device="cuda") != 1
    for act in ("relu", "relu2", "gelu", "gelu_tanh", "silu"):
        dU, db = sp.sp24_spmm_bwd_input_act(dY, f["vals_col"], f["meta_col"], 64, 64, U, act=act)
        assert torch.isfinite(dU[others]).all()
        assert not torch.isfinite(dU[1, ::2]).any() and not torch.isfinite(db[::2]).any()
        if act in ("relu", "relu2"):
            assert (dU[:, 1::2] == 0).all() and (db[1::2] == 0).all()
        else:
            assert not torch.isfinite(dU[1, 1::2]).any() and not torch.isfinite(db[1::2]).any()

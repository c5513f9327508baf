"""What no AdamW step can run with is refused where the optimiser or its plan is
made: a guarded step's norm counts it on the device before the step itself is
checked, and a step that was refused after that would be counted all the same."""
import math
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sp():
    from structured_sparse_transformer_amd import build, sp24
    if not os.path.exists(sp24.LIB_PATH):
        build.build()
    sp24.lib()
    return sp24


SETTINGS = [dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)), dict(betas=(math.nan, 0.9)), dict(eps=-1e-8), dict(eps=math.nan)]


@pytest.mark.parametrize("setting", SETTINGS)
def test_settings(sp, setting):
    from structured_sparse_transformer_amd.adamw import AdamW
    with pytest.raises(ValueError, match="betas"):
        AdamW([torch.zeros(5)], max_norm=1.0, **setting)


@pytest.mark.parametrize("which", range(4))
def test_alignment(sp, which):
    """Of values, states and copies; a tensor without entries may lie anywhere."""
    for state in (torch.float32, torch.uint8):
        whole = [torch.zeros(9, dtype=d) for d in (torch.float32, state, state, torch.float16)]
        tensors = [[t[1:] if k == which else t[:8]] for k, t in enumerate(whole)]
        exps = [torch.zeros(2, dtype=torch.uint8)[1:] for _ in range(2)]
        more = dict(M_exps=exps[:1], V_exps=exps[1:]) if state == torch.uint8 else {}
        with pytest.raises(ValueError, match="aligned"):
            sp.sp24_adamw_plan(*tensors, **more)
    sp.sp24_adamw_plan(*([t[8:]] for t in (torch.zeros(9)[1:], torch.zeros(9)[1:], torch.zeros(9)[1:])))


@pytest.mark.gpu
def test_nothing_is_counted(sp):
    from structured_sparse_transformer_amd.adamw import AdamW
    whole = torch.ones(101, device="cuda")
    with pytest.raises(ValueError, match="aligned"):
        AdamW([whole[1:]], max_norm=1.0)
    optimizer = AdamW([whole], betas=[0, 0.5], eps=0, max_norm=1.0)
    with pytest.raises(sp.Sp24Error):   # the gradient 4 bytes past a multiple of 16: refused by the norm
        optimizer.step([torch.ones(102, device="cuda")[1:]])
    assert int(sp.control_values(optimizer.control)["step"]) == 0 and (whole == 1).all()
    optimizer.step([torch.ones(101, device="cuda")])
    assert int(sp.control_values(optimizer.control)["step"]) == 1 and (whole < 1).all()

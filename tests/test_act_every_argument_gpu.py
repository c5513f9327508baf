"""The products' activations and slopes over every finite fp16 argument, as the
kernels round them (the CPU emulation covers their arithmetic alone).

Tolerances: an activation is rounded to fp16 (2^-11, 2^-25 among subnormals) from
a value within 2^-16 relative of the exact one or 2^-30; a slope within 2^-18 (1 +
|u|), |u| up to 16 where the smooth ones still change.
"""
import pytest
from test_spmm_act_gpu import ACTS, HALF, SLOPE, SUB, act64, far, slope64, sp  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("whole", [True, False])
def test_every_argument(sp, act, whole):  # noqa: F811
    """In one call over all of them (whole tiles), and in calls of 16 (thin)."""
    every = torch.arange(1 << 16, device="cuda").to(torch.int16).view(torch.float16)
    u = every[torch.isfinite(every)]
    assert len(u) == 63488
    if not whole:
        u = u[:: 31][:2048]
    W = torch.zeros(16, 64, dtype=torch.float16, device="cuda")
    W[0, 0] = 1.0
    f = sp.sp24_search_compress(W)
    col = lambda v, n: torch.cat([v[:, None], torch.zeros(len(v), n - 1, dtype=v.dtype, device="cuda")], 1)  # noqa: E731
    parts = [u] if whole else list(u.split(16))
    Y = torch.cat([sp.sp24_spmm_fwd_act(col(v, 64), f["vals_row"], f["meta_row"], 16, 64, act=act)[0][:, 0] for v in parts])
    want = act64(act, u.double())
    big = want.abs() > 65504 * (1 + 2.0 ** -12)
    assert torch.isinf(Y[big]).all()
    # between the largest number and half a step past it a value may go either way
    fits = want.abs() <= 65504
    assert far(Y[fits], want[fits], ((HALF + 2.0 ** -16) * want.abs() + SUB + 2.0 ** -30)[fits]) <= 1
    W = torch.zeros(64, 16, dtype=torch.float16, device="cuda")
    W[0, 0] = 1.0
    f = sp.sp24_search_compress(W)
    D = torch.cat([sp.sp24_spmm_bwd_input_act(col(torch.ones_like(v), 64), f["vals_col"], f["meta_col"], 64, 16, col(v, 16),
                                              act=act)[0][:, 0] for v in parts])
    want = slope64(act, u.double())
    fits = want.abs() < 65504
    assert far(D[fits], want[fits], (HALF * want.abs() + SUB + SLOPE * (1 + u.double().abs().clamp(max=16)))[fits]) <= 1

"""GPU checks of 8-bit AdamW states at a tensor's end: the last, partly filled
group of 64 is its own, whatever the other groups hold.

Where a group turned non-finite, the others' steps are compared with a run
without it bit for bit: nothing of one group enters another's arithmetic.
"""
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


def steps(sp, n, bad, count=4):
    """`count` steps of a tensor of n entries, whose first gradient holds `bad`."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    P = torch.randn(n, generator=gen, device="cuda")
    M, V = sp.state8(P), sp.state8(P)
    plan = sp.sp24_adamw_plan([P], [M[0]], [V[0]], M_exps=[M[1]], V_exps=[V[1]])
    for t in range(1, count + 1):
        G = torch.randn(n, generator=gen, device="cuda")
        if t == 1:
            for at, value in bad:
                G[at] = value
        sp.sp24_adamw_step(plan, [G], step=t, seed=5)
    return P, M, V


# the last group full, of 1, 8, 60 and 63 entries; in the first group's wave, in another wave, in another workgroup
@pytest.mark.parametrize("n", [65, 124, 128, 200, 255, 256, 257, 1000, 4096 + 8, 3 * 4096 + 64 + 33])
@pytest.mark.parametrize("value", [math.nan, 1e30])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_a_group_that_is_not_finite_stays_alone(sp, n, value, place):
    group = {"first": 0, "middle": (n - 1) // 128, "last": (n - 1) // 64}[place]
    P, M, V = steps(sp, n, [(64 * group, value)])
    wantP, wantM, wantV = steps(sp, n, [])
    lost = torch.arange(n, device="cuda") // 64 == group
    kept = torch.arange(len(M[1]), device="cuda") != group
    for got, want in ((M, wantM), (V, wantV)):
        assert torch.equal(got[0][~lost], want[0][~lost]) and torch.equal(got[1][kept], want[1][kept])
    # 1e30 squared overflows: V's group is lost then, and the root of it is infinite where the entry is
    assert int(V[1][group]) == 255 and (int(M[1][group]) == 255) == math.isnan(value)
    assert torch.equal(P[~lost], wantP[~lost]) and torch.isfinite(P[~lost]).all()
    assert torch.isnan(P[lost]).all()
    m, r = sp.sp24_state8_values(*M), sp.sp24_state8_values(*V, root=True)
    assert torch.isfinite(m[~lost]).all() and torch.equal(torch.isnan(r), lost)

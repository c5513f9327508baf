"""Arguments of the orthogonalisation and the optimiser step that choose and
bound their arithmetic: checked on the host, so all of this runs without a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

SHAPE, UNSUPPORTED, WORKSPACE = 2, 5, 7
A = 0x1000          # 16-byte aligned, never dereferenced
F16, F32, I32 = 0, 1, 2
FP16_OPERANDS = 16
USUAL = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def sp():
    from structured_sparse_transformer_amd import build, sp24
    import os
    if not os.path.exists(sp24.LIB_PATH):
        build.build()
    sp24.lib()
    return sp24


def orthogonalize(sp, rows, out=F16, steps=None):
    """The status of a call with too small a workspace: WORKSPACE when everything else is accepted."""
    coef = (ctypes.c_float * 96)(*[v for r in rows for v in r])
    job = (sp.OrthoJob * 1)(sp.OrthoJob(A, A, 64, 32))
    return sp.lib().sp24_orthogonalize(job, 1, F32, out, coef, len(rows) if steps is None else steps, 1e-7, A, 1, None)


def test_operands_are_chosen_beside_the_result_type(sp):
    assert sp.FP16_OPERANDS == FP16_OPERANDS
    for out in (F16, F32, F16 | FP16_OPERANDS, F32 | FP16_OPERANDS):
        assert orthogonalize(sp, [USUAL] * 5, out) == WORKSPACE
    for out in (I32, I32 | FP16_OPERANDS, 8, 32, 2 * FP16_OPERANDS | F32):
        assert orthogonalize(sp, [USUAL] * 5, out) == UNSUPPORTED


def muon(sp, rows, precise):
    coef = (ctypes.c_float * 96)(*[v for r in rows for v in r])
    job = (sp.MuonJob * 1)(sp.MuonJob(A, A, A, A, 64, 32, 0.1, 0.0))
    return sp.lib().sp24_muon_step(job, 1, 0.95, 1, precise, coef, len(rows), 1e-7, A, 1, None)


def largest(rows, split):
    """The largest of what X, A and B reach, from a fine grid of singular values."""
    import numpy as np
    top, s = 0.0, 1.0
    for a, b, c in rows:
        v = np.linspace(0, s, 200001)
        q = b * v ** 2 + c * v ** 4
        s = np.abs(v * (a + q)).max()
        top = max(top, v[-1] ** 2, np.abs(q + (a if split else 0)).max(), s)
    return top


ACCEPTED = [[USUAL] * 32, [(1.5, -0.5, 0.0)] * 32, [(1.875, -1.25, 0.375)] * 32, [(0.0, 0.0, 0.0)] * 5, [(1.0, 0.0, 0.0)] * 3,
            [(3.4445 - 0.1 * k, -4.7750 + 0.1 * k, 2.0315 - 0.05 * k) for k in range(8)],
            [(8.3, -23.6, 17.3), (4.1, -2.95, 0.545)], [(3.9, 0.0, 0.0), (1.0, -0.25, 0.0)], [(15.4, -14.4, 0.0)],
            [(3.0, -15.4, 13.0)]]
# a singular value of 2.5 whose B would be 42; a I alone past 16 (B's diagonal); X past 16; A past
# 16; B's vertex past -16 between ends that are within
REFUSED = [[(2.5, 0.0, 0.0), (1.0, -4.775, 1.828)], [(17.0, 0.0, 0.0)], [(3.0, 0.0, 14.0)], [(4.1, 0.0, 0.0), (0.1, 0.0, 0.0)],
           [(1.0, -70.0, 70.0)], [USUAL, (1.0, 1.0, 40.0)], [(3.5, 0.0, 0.0), (1.5, 0.0, 0.0), (1.0, 0.0, 0.0)]]


@pytest.mark.parametrize("rows", ACCEPTED)
def test_coefficients_within_range_are_taken(sp, rows):
    for fast in (0, FP16_OPERANDS):
        assert largest(rows, not fast) <= 15.5
        assert orthogonalize(sp, rows, F32 | fast) == WORKSPACE
        assert muon(sp, rows, int(not fast)) == WORKSPACE


@pytest.mark.parametrize("rows", REFUSED)
def test_coefficients_past_fp16s_range_are_refused(sp, rows):
    for fast in (0, FP16_OPERANDS):
        assert largest(rows, not fast) > 15.5
        assert orthogonalize(sp, rows, F32 | fast) == UNSUPPORTED
        assert muon(sp, rows, int(not fast)) == UNSUPPORTED


def test_coefficients_that_only_two_part_operands_cannot_hold(sp):
    rows = [(15.6, -15.1, 0.0)]    # a I is in B then; X itself stays below 7
    assert largest(rows, False) <= 15.5 < largest(rows, True)
    assert orthogonalize(sp, rows, F16) == UNSUPPORTED and orthogonalize(sp, rows, F16 | FP16_OPERANDS) == WORKSPACE
    assert muon(sp, rows, 1) == UNSUPPORTED and muon(sp, rows, 0) == WORKSPACE


def test_random_coefficients_against_a_grid(sp):
    import random
    rng = random.Random(5)
    seen = [0, 0]
    for _ in range(300):
        rows = [tuple(rng.uniform(-f, f) for f in (4, 8, 8)) for _ in range(rng.randint(1, 3))]
        rows = [tuple(float(ctypes.c_float(v).value) for v in r) for r in rows]
        top = largest(rows, True)
        if abs(top - 15.5) < 0.01:
            continue               # the grid's own error
        assert (orthogonalize(sp, rows) == WORKSPACE) == (top < 15.5)
        seen[int(top < 15.5)] += 1
    assert min(seen) > 20


def test_forms_of_coefficients_that_the_binding_takes(sp):
    import numpy as np
    want = [float(ctypes.c_float(v).value) for v in USUAL]
    for one in (None, USUAL, list(USUAL), np.array(USUAL), torch.tensor(USUAL, dtype=torch.float64)):
        assert list(sp._coeffs(one, 3)) == want * 3
    for each in ([USUAL] * 3, np.array([USUAL] * 3), torch.tensor([USUAL] * 3, dtype=torch.float64), iter([USUAL] * 3)):
        assert list(sp._coeffs(each, 3)) == want * 3
    for bad in ([], [()], [USUAL] * 2, [USUAL, USUAL, USUAL[:2]], USUAL[:2], np.zeros((0, 3))):
        with pytest.raises(ValueError):
            sp._coeffs(bad, 3)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_coefficients_that_are_no_numbers_are_refused(sp, bad):
    for k in range(3):
        row = list(USUAL)
        row[k] = bad
        assert orthogonalize(sp, [USUAL, row]) == UNSUPPORTED and muon(sp, [row], 1) == UNSUPPORTED

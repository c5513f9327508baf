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

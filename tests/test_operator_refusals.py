"""Argument checks of the embedding, orthogonalisation and optimiser entry
points: every refusal comes back before any device call, so all of this runs
without a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, TOO_LARGE, WORKSPACE = 0, 1, 2, 3, 5, 6, 7
A = 0x1000          # 16-byte aligned, never dereferenced
MIS = 0x1008
F16, F32, I32, I64 = 0, 1, 2, 3


@pytest.fixture(scope="module")
def sp():
    from structured_sparse_transformer_amd import build, sp24
    import os
    if not os.path.exists(sp24.LIB_PATH):
        build.build()
    sp24.lib()
    return sp24


def test_status_strings(sp):
    assert sp.lib().sp24_status_str(WORKSPACE) == b"workspace too small"
    assert sp.STATUS_NAMES[WORKSPACE] == "ERR_WORKSPACE"


def test_embed_fwd(sp):
    f = sp.lib().sp24_embed_fwd

    def call(ids=A, id_type=I64, T=4, table=A, table_type=F16, V=10, d=8, out=A):
        return f(ids, id_type, T, table, table_type, V, d, 1.0, out, None)

    assert call(id_type=F16) == UNSUPPORTED and call(id_type=9) == UNSUPPORTED and call(table_type=I32) == UNSUPPORTED
    assert call(T=-1) == SHAPE and call(V=-1) == SHAPE and call(d=-8) == SHAPE
    assert call(T=2 ** 31) == TOO_LARGE and call(V=2 ** 31) == TOO_LARGE and call(d=2 ** 31) == TOO_LARGE
    assert call(T=2 ** 30, d=2 ** 10) == TOO_LARGE and call(V=2 ** 30, d=2 ** 10) == TOO_LARGE
    assert call(T=2 ** 31 - 1, d=128 + 8, V=1) == TOO_LARGE        # over 2^34 chunks of 8 entries
    assert call(ids=None) == NULL and call(table=None) == NULL and call(out=None) == NULL
    assert call(ids=MIS) == ALIGN and call(table=MIS) == ALIGN and call(out=MIS) == ALIGN
    assert call(T=0, ids=None, out=None) == OK and call(d=0, out=None, table=None) == OK


def test_embed_bwd(sp):
    f, size = sp.lib().sp24_embed_bwd, sp.lib().sp24_embed_bwd_workspace
    need = size(4, 10, 8)
    assert need > 0

    def call(ids=A, id_type=I64, T=4, dout=A, V=10, d=8, acc=0, dtable=A, ws=A, n=need):
        return f(ids, id_type, T, dout, V, d, 1.0, acc, dtable, ws, n, None)

    assert call(id_type=F32) == UNSUPPORTED
    assert call(T=-1) == SHAPE and call(V=-1) == SHAPE and call(d=-1) == SHAPE
    assert call(T=2 ** 28) == TOO_LARGE and call(d=2 ** 24) == TOO_LARGE and call(V=2 ** 31) == TOO_LARGE
    for k in ("ids", "dout", "dtable", "ws"):
        assert call(**{k: None}) == NULL and call(**{k: MIS}) == ALIGN
    assert call(n=need - 1) == WORKSPACE
    assert call(V=0, dtable=None, ws=None, n=0) == OK and call(d=0, dtable=None, ws=None, n=0) == OK
    assert call(T=0, acc=1, ids=None, dout=None, dtable=None, ws=None, n=0) == OK
    assert call(T=0, ids=None, dout=None, ws=None) == NULL     # every row is still to be cleared
    assert size(2 ** 28, 10, 8) == -1 and size(-1, 10, 8) == -1


def test_embed_bwd_stays_within_a_launch(sp):
    # a launch has 2^32 work-items along x (clearing takes 256 for 16 rows, placing
    # 512 for 2048 ids) and 65535 workgroups along y (joining takes 256 columns each)
    size = sp.lib().sp24_embed_bwd_workspace
    assert size(10, 2 ** 27 - 1, 1) > 0 and size(10, 2 ** 27, 1) == -1 and size(10, 2 ** 28, 1) == -1
    assert (2 ** 22 + 2 ** 27 // 16) * 256 < 2 ** 32 and (2 ** 28 // 64) * 512 < 2 ** 32
    assert size(10, 10, 2 ** 24 - 257) > 0 and size(10, 10, 2 ** 24 - 256) == -1
    assert -(-(2 ** 24 - 257) // 256) <= 65535


def ortho_jobs(sp, *jobs):
    return (sp.OrthoJob * len(jobs))(*[sp.OrthoJob(*j) for j in jobs])


def test_orthogonalize(sp):
    f, size = sp.lib().sp24_orthogonalize, sp.lib().sp24_orthogonalize_workspace
    good = (A, A, 64, 32)
    need = size(ortho_jobs(sp, good), 1)
    coef = (ctypes.c_float * 96)()

    def call(*jobs, count=None, g=F32, o=F16, c=coef, steps=5, eps=1e-7, ws=A, n=need):
        jobs = jobs or (good,)
        return f(ortho_jobs(sp, *jobs), len(jobs) if count is None else count, g, o, c, steps, eps, ws, n, None)

    assert f(None, 1, F32, F16, coef, 5, 1e-7, A, need, None) == NULL
    assert call(count=0) == SHAPE and call(*[good] * 9) == SHAPE
    assert call(g=I32) == UNSUPPORTED and call(o=7) == UNSUPPORTED
    assert call(steps=0) == SHAPE and call(steps=33) == SHAPE and call(c=None) == NULL
    assert call(eps=-1.0) == UNSUPPORTED and call(eps=float("nan")) == UNSUPPORTED
    assert call((A, A, -1, 32)) == SHAPE and call((A, A, 64, 2 ** 31)) == TOO_LARGE
    assert call((A, A, 2 ** 15, 2 ** 15)) == TOO_LARGE and call((A, A, 1, 2 ** 23)) == TOO_LARGE
    assert call((None, A, 64, 32)) == NULL and call((A, None, 64, 32)) == NULL and call(ws=None) == NULL
    assert call((MIS, A, 64, 32)) == ALIGN and call((A, MIS, 64, 32)) == ALIGN and call(ws=MIS) == ALIGN
    assert call(n=need - 1) == WORKSPACE and call(good, good) == WORKSPACE
    assert call((None, None, 0, 32), ws=None, n=0) == OK
    assert size(None, 1) == -1 and size(ortho_jobs(sp, (A, A, 2 ** 15, 2 ** 15)), 1) == -1


def test_muon_step(sp):
    f, size = sp.lib().sp24_muon_step, sp.lib().sp24_muon_workspace
    coef = (ctypes.c_float * 96)()

    def jobs(*j):
        return (sp.MuonJob * len(j))(*[sp.MuonJob(*x, 0.1, 0.0) for x in j])

    good = (A, A, A, A, 64, 32)
    need = size(jobs(good), 1)

    def call(*j, c=coef, steps=5, eps=1e-7, ws=A, n=need):
        j = j or (good,)
        return f(jobs(*j), len(j), 0.95, 1, 0, c, steps, eps, ws, n, None)

    assert f(None, 1, 0.95, 1, 0, coef, 5, 1e-7, A, need, None) == NULL
    assert call(*[good] * 9) == SHAPE and call(steps=0) == SHAPE and call(c=None) == NULL and call(eps=-1.0) == UNSUPPORTED
    for k in range(3):
        bad = list(good)
        bad[k] = None
        assert call(tuple(bad)) == NULL
    for k in range(4):
        bad = list(good)
        bad[k] = MIS
        assert call(tuple(bad)) == ALIGN
    assert call(good[:4] + (64, -1)) == SHAPE and call(good[:4] + (2 ** 15, 2 ** 15)) == TOO_LARGE
    assert call(ws=None) == NULL and call(n=need - 1) == WORKSPACE
    assert call((None, None, None, None, 0, 32), ws=None, n=0) == OK
    assert size(jobs(good), 0) == -1


def test_binding_refuses_before_the_library(sp):
    f32, f16 = lambda *s: torch.zeros(*s), lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    ids = torch.zeros(4, dtype=torch.int64)
    for bad in (lambda: sp.sp24_embed_fwd(ids.float(), f16(8, 16)), lambda: sp.sp24_embed_fwd(ids, f16(8)),
                lambda: sp.sp24_embed_fwd(ids, f32(8, 16).double()),
                lambda: sp.sp24_embed_fwd(ids, f16(8, 16), out=f32(4, 16)),
                lambda: sp.sp24_embed_bwd(ids, f32(4, 16), 8), lambda: sp.sp24_embed_bwd(ids, f16(5, 16), 8),
                lambda: sp.sp24_embed_bwd(ids, f16(4, 16), 8, accumulate=True),
                lambda: sp.sp24_embed_bwd(ids, f16(4, 16), 8, dtable=f32(9, 16)),
                lambda: sp.sp24_embed_bwd(ids, f16(4, 16), 8, workspace=torch.zeros(16, dtype=torch.uint8)),
                lambda: sp.sp24_embed_bwd(ids, f16(4, 16), -8),
                lambda: sp.sp24_orthogonalize(f32(8)), lambda: sp.sp24_orthogonalize(f32(8, 8).double()),
                lambda: sp.sp24_orthogonalize(f32(8, 8), dtype=torch.bfloat16),
                lambda: sp.sp24_orthogonalize(f32(8, 8), steps=0), lambda: sp.sp24_orthogonalize(f32(8, 8), steps=33),
                lambda: sp.sp24_orthogonalize(f32(8, 8), steps=5, coeffs=[(1, 2, 3)] * 4),
                lambda: sp.sp24_orthogonalize(f32(8, 8), coeffs=(1, 2)),
                lambda: sp.sp24_orthogonalize_batch([f32(8, 8), f16(8, 8)]), lambda: sp.sp24_orthogonalize_batch([]),
                lambda: sp.sp24_orthogonalize(f32(8, 8), out=f32(8, 8)),
                lambda: sp.sp24_muon_step([f16(8, 8)], [f32(8, 8)], [f32(8, 8)], [None], [0.1]),
                lambda: sp.sp24_muon_step([f32(8, 8)], [f32(8, 9)], [f32(8, 8)], [None], [0.1]),
                lambda: sp.sp24_muon_step([f32(8, 8)], [f32(8, 8)], [f32(8, 8)], [f32(8, 8)], [0.1]),
                lambda: sp.sp24_muon_step([f32(8, 8)], [f32(8, 8)], [f32(8, 8)], [None], [])):
        with pytest.raises(ValueError):
            bad()
    for call in (lambda: sp.sp24_embed_fwd(ids, f16(8, 16)), lambda: sp.sp24_embed_bwd(ids, f16(4, 16), 8),
                 lambda: sp.sp24_orthogonalize(f32(8, 8)),
                 lambda: sp.sp24_muon_step([f32(8, 8)], [f32(8, 8)], [f32(8, 8)], [None], [0.1])):
        with pytest.raises(ValueError, match="on the GPU"):
            call()

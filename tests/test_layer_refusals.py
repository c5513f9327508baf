"""Argument checks of the products with an epilogue, the bias gradient, the
gradients' norm and AdamW: every refusal comes back before any device call, so
all of this runs without a GPU."""
import ctypes
import math
import os

import pytest

torch = pytest.importorskip("torch")

OK, NULL, SHAPE, ALIGN, UNSUPPORTED, TOO_LARGE, WORKSPACE = 0, 1, 2, 3, 5, 6, 7
A, MIS = 0x1000, 0x1008     # never dereferenced
F16, F32, I32, BF16, STATE8 = 0, 1, 2, 4, 5


@pytest.fixture(scope="module")
def sp():
    from structured_sparse_transformer_amd import build, sp24
    if not os.path.exists(sp24.LIB_PATH):
        build.build()
    sp24.lib()
    return sp24


def test_fwd_act(sp):
    f, size = sp.lib().sp24_spmm_fwd_act, sp.lib().sp24_spmm_fwd_act_workspace
    need = size(100, 32, 8192)
    assert need > 0 and size(0, 32, 64) == 0 and size(1, 32, 64) == 0
    assert size(-1, 32, 64) == -1 and size(4, 24, 64) == -1 and size(4, 2 ** 27, 64) == -1 and size(2 ** 31, 32, 64) == -1

    def call(X=A, vals=A, meta=A, T=100, R=32, C=8192, bias=A, act=3, residual=A, U=A, Y=A, ws=A, n=need):
        return f(X, vals, meta, T, R, C, bias, act, residual, U, Y, ws, n, None)

    assert call(act=-1) == UNSUPPORTED and call(act=6) == UNSUPPORTED
    assert call(T=-1) == SHAPE and call(R=24) == SHAPE and call(C=72) == SHAPE and call(R=-16) == SHAPE
    assert call(T=2 ** 31) == TOO_LARGE and call(R=2 ** 27) == TOO_LARGE and call(T=2 ** 30, C=2 ** 10) == TOO_LARGE
    for k in ("X", "vals", "meta", "Y", "ws"):
        assert call(**{k: None}) == NULL
    for k in ("X", "vals", "meta", "Y", "bias", "residual", "U", "ws"):
        assert call(**{k: MIS}) == ALIGN
    assert call(n=need - 1) == WORKSPACE
    assert call(T=0, X=None, Y=None, bias=MIS, ws=None) == OK and call(R=0, Y=None, ws=None) == OK


def test_bwd_input_act(sp):
    f, size = sp.lib().sp24_spmm_bwd_input_act, sp.lib().sp24_spmm_bwd_input_act_workspace
    need = size(1000, 32, 64)
    assert need > 0 and size(0, 32, 64) == 0

    def call(dY=A, vals=A, meta=A, T=1000, R=32, C=64, act=3, U=A, dU=A, dbias=A, ws=A, n=need):
        return f(dY, vals, meta, T, R, C, act, U, dU, dbias, ws, n, None)

    assert call(act=9) == UNSUPPORTED
    assert call(T=-1) == SHAPE and call(R=24) == SHAPE and call(C=72) == SHAPE
    assert call(T=2 ** 31) == TOO_LARGE and call(C=2 ** 27) == TOO_LARGE
    assert size(-1, 32, 64) == -1 and size(4, 24, 64) == -1 and size(4, 32, 2 ** 27) == -1 and size(2 ** 31, 32, 64) == -1
    for k in ("dY", "vals", "meta", "dU", "U", "ws"):
        assert call(**{k: None}) == NULL
    for k in ("dY", "vals", "meta", "dU", "U", "dbias", "ws"):
        assert call(**{k: MIS}) == ALIGN
    assert call(n=need - 1) == WORKSPACE
    assert call(C=0, dU=None, dbias=None) == OK


def test_bias_grad(sp):
    f, size = sp.lib().sp24_bias_grad, sp.lib().sp24_bias_grad_workspace
    need = size(5000, 32)
    assert need > 0 and size(0, 32) == 0 and size(1, 32) == 0

    def call(dY=A, T=5000, R=32, dbias=A, ws=A, n=need):
        return f(dY, T, R, dbias, ws, n, None)

    assert call(T=-1) == SHAPE and call(R=24) == SHAPE and call(R=-16) == SHAPE
    assert call(T=2 ** 31) == TOO_LARGE and call(R=2 ** 27) == TOO_LARGE and call(T=2 ** 30, R=2 ** 10) == TOO_LARGE
    assert size(1, 2 ** 27) == -1 and size(-1, 32) == -1 and size(4, 24) == -1 and size(2 ** 31, 16) == -1
    for k in ("dY", "dbias", "ws"):
        assert call(**{k: None}) == NULL and call(**{k: MIS}) == ALIGN
    assert call(n=need - 1) == WORKSPACE and call(R=0, dY=None, dbias=None, ws=None) == OK


def test_grad_norm(sp):
    f, size = sp.lib().sp24_grad_norm, sp.lib().sp24_grad_norm_workspace

    def call(ptrs=(A, A), sizes=(10, 20), g=F32, scale=1.0, most=1.0, control=A, ws=A, n=None, count=None):
        p, s = (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(sizes))(*sizes)
        count = len(sizes) if count is None else count
        need = size(ctypes.cast(s, ctypes.c_void_p), count)
        return f(ctypes.cast(p, ctypes.c_void_p), ctypes.cast(s, ctypes.c_void_p), count, g, scale, most, control, ws,
                 need if n is None else n, None)

    assert call(g=I32) == UNSUPPORTED and call(g=BF16) == UNSUPPORTED
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == UNSUPPORTED
    for most in (0.0, -1.0, math.nan):
        assert call(most=most) == UNSUPPORTED
    assert call(sizes=(10, -1)) == SHAPE and call(count=-1) == SHAPE and call(sizes=(10, 2 ** 34)) == TOO_LARGE
    assert call(control=None) == NULL and call(control=MIS) == ALIGN
    assert call(ptrs=(A, None)) == NULL and call(ptrs=(A, MIS)) == ALIGN
    assert call(ws=None) == NULL and call(ws=MIS) == ALIGN and call(n=15) == WORKSPACE
    assert f(None, None, 2, F32, 1.0, 1.0, A, A, 100, None) == NULL
    assert size(None, 0) == 0 and size(None, 1) == -1


def test_adamw(sp):
    f = sp.lib().sp24_adamw_step

    def call(g=F32, state=F32, b1=0.9, b2=0.999, eps=1e-8, step=1, control=None, count=2, jobs=True, **fields):
        base = dict(G=A, P=A, M=A, V=A, M_exps=A, V_exps=A, W=None, n=64, lr=0.1, decay=0.0)
        arr = (sp.AdamwJob * 2)(sp.AdamwJob(n=0), sp.AdamwJob(**{**base, **fields}))
        return f(ctypes.cast(arr, ctypes.c_void_p) if jobs else None, count, g, state, b1, b2, eps, step, control, 0, None)

    assert call(jobs=False) == NULL and call(count=-1) == SHAPE
    assert call(g=I32) == UNSUPPORTED and call(state=F16) == UNSUPPORTED and call(g=STATE8) == UNSUPPORTED
    for b in (-0.1, 1.0, math.nan):
        assert call(b1=b) == UNSUPPORTED and call(b2=b) == UNSUPPORTED
    assert call(eps=-1.0) == UNSUPPORTED and call(eps=math.nan) == UNSUPPORTED
    assert call(step=0) == SHAPE and call(control=MIS) == ALIGN
    assert call(n=-1) == SHAPE and call(n=2 ** 34) == TOO_LARGE
    for k in ("G", "P", "M", "V"):
        assert call(**{k: None}) == NULL and call(**{k: MIS}) == ALIGN
    assert call(W=MIS) == ALIGN
    assert call(state=STATE8, M_exps=None) == NULL and call(state=STATE8, V_exps=None) == NULL
    assert call(n=0, G=None) == OK and call(count=0, jobs=False) == OK


def test_state8_values(sp):
    f = sp.lib().sp24_state8_values

    def call(codes=A, exps=A, n=64, root=0, kind=F32, out=A):
        return f(codes, exps, n, root, kind, out, None)

    assert call(kind=F16) == UNSUPPORTED and call(n=-1) == SHAPE and call(n=2 ** 34) == TOO_LARGE
    for k in ("codes", "exps", "out"):
        assert call(**{k: None}) == NULL
    assert call(codes=MIS) == ALIGN and call(out=MIS) == ALIGN and call(n=0, codes=None, exps=None, out=None) == OK


def test_binding(sp):
    """What the binding refuses before it asks for the GPU."""
    half = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    vals, meta = half(32, 32), torch.zeros(32, 4, dtype=torch.int16)
    X = half(5, 64)
    for bad in (dict(act="swish"), dict(bias=torch.zeros(31)), dict(bias=half(32)), dict(residual=half(5, 31)),
                dict(out=half(5, 33)), dict(U=torch.zeros(5, 32))):
        with pytest.raises(ValueError):
            sp.sp24_spmm_fwd_act(X, vals, meta, 32, 64, **bad)
    with pytest.raises(ValueError):
        sp.sp24_spmm_fwd_act(X.float(), vals, meta, 32, 64)
    cols, cmeta = half(64, 16), torch.zeros(64, 2, dtype=torch.int16)
    for U, more in ((None, dict(act="gelu")), (half(5, 63), dict(act="gelu")), (half(5, 64), dict(dbias=half(64))),
                    (half(5, 64), dict(act="tanh"))):
        with pytest.raises(ValueError):
            sp.sp24_spmm_bwd_input_act(half(5, 32), cols, cmeta, 32, 64, U, **more)
    with pytest.raises(ValueError):
        sp.sp24_bias_grad(torch.zeros(5, 32))
    with pytest.raises(ValueError):
        sp.sp24_grad_norm([torch.zeros(5, dtype=torch.int32)])
    P = torch.zeros(70)
    for args in (([P], [P], [P[:69]]), ([P], [P], [P], [P]), ([P], [P, P], [P]), ([P.half()], [P], [P])):
        with pytest.raises(ValueError):
            sp.sp24_adamw_plan(*args)
    with pytest.raises(ValueError):
        sp.sp24_adamw_plan([P], [P], [P], M_exps=[torch.zeros(2, dtype=torch.uint8)])
    c, e = sp.state8(P)
    assert c.dtype == e.dtype == torch.uint8 and len(e) == 2
    with pytest.raises(ValueError):
        sp.sp24_adamw_plan([P], [c], [c], M_exps=[e], V_exps=[e[:1]])
    plan = sp.AdamwPlan((sp.AdamwJob * 1)(), ([P],), [70], False)
    for kw in (dict(), dict(step=1, control=P)):
        with pytest.raises(ValueError):
            sp.sp24_adamw_step(plan, [P], **kw)
    with pytest.raises(ValueError):
        sp.sp24_adamw_step(plan, [P[:3]], step=1)
    with pytest.raises(ValueError):
        sp.sp24_state8_values(c, e[:1])


def test_a_plan_takes_no_memory_twice(sp):
    """A tied weight listed twice, one state for two tensors, or parts of one
    buffer that overlap: two workgroups would write the same entries."""
    P, M, V, Q, N, U = (torch.zeros(70) for _ in range(6))
    both = torch.zeros(139)
    for args in (([P, P], [M, N], [V, U]), ([P, Q], [M, M], [V, U]), ([P], [M], [M]), ([P], [P], [V]),
                 ([both[:70], both[69:]], [M, N], [V, U])):
        with pytest.raises(ValueError, match="share memory"):
            sp.sp24_adamw_plan(*args)
    c, d, e = (torch.zeros(70, dtype=torch.uint8) for _ in range(3))
    with pytest.raises(ValueError, match="share memory"):
        sp.sp24_adamw_plan([P], [c], [d], M_exps=[e[:2]], V_exps=[e[1:3]])

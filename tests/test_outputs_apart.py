"""Outputs of the products with an epilogue that share memory with what other
workgroups still read are refused before the GPU is asked: a product in place on
its own input, the residual's memory where that is the input too, one tensor for
two outputs, parts of one buffer that overlap."""
import os

import pytest

torch = pytest.importorskip("torch")
T, N = 5, 64


@pytest.fixture(scope="module")
def sp():
    from structured_sparse_transformer_amd import build, sp24
    if not os.path.exists(sp24.LIB_PATH):
        build.build()
    sp24.lib()
    return sp24


def half(*s):
    return torch.zeros(*s, dtype=torch.float16)


FORM = (half(N, N // 2), torch.zeros(N, N // 16, dtype=torch.int16))


@pytest.fixture()
def tensors():
    buffer = half(2 * T * N)
    return dict(X=buffer[: T * N].view(T, N), Y=half(T, N), res=half(T, N), late=buffer[T * N // 2: T * N // 2 + T * N].view(T, N))


@pytest.mark.parametrize("residual,out,U", [("X", "X", None), (None, "X", None), ("res", "X", None), ("res", "Y", "Y"),
                                            ("res", None, "res"), ("res", None, "X"), (None, "late", None), (None, "Y", "late"),
                                            ("late", "late", None)])
def test_forward(sp, tensors, residual, out, U):
    get = lambda k: None if k is None else tensors[k]  # noqa: E731
    with pytest.raises(ValueError, match="shares memory"):
        sp.sp24_spmm_fwd_act(tensors["X"], *FORM, N, N, residual=get(residual), out=get(out), U=get(U))


@pytest.mark.parametrize("U,out", [("X", "X"), ("res", "X"), ("res", "late"), (None, "X")])
def test_backward(sp, tensors, U, out):
    get = lambda k: None if k is None else tensors[k]  # noqa: E731
    with pytest.raises(ValueError, match="shares memory"):
        sp.sp24_spmm_bwd_input_act(tensors["X"], *FORM, N, N, get(U), act="gelu" if U else "none", out=get(out))


def test_backward_sums(sp, tensors):
    with pytest.raises(ValueError, match="shares memory"):
        sp.sp24_spmm_bwd_input_act(tensors["X"], *FORM, N, N, tensors["res"], act="gelu", out=tensors["Y"],
                                   dbias=tensors["Y"].view(-1).view(torch.float32)[:N])


def test_what_may_be_in_place(sp, tensors):
    """Neighbours in one buffer, the residual's and U's own memory (a view of it
    too) come as far as the GPU's own check."""
    both = half(2 * T * N)
    for call in (lambda: sp.sp24_spmm_fwd_act(tensors["X"], *FORM, N, N, residual=tensors["res"], out=tensors["res"].view(T, N)),
                 lambda: sp.sp24_spmm_fwd_act(tensors["X"], *FORM, N, N, out=both[: T * N].view(T, N), U=both[T * N:].view(T, N)),
                 lambda: sp.sp24_spmm_bwd_input_act(tensors["X"], *FORM, N, N, tensors["res"], act="gelu", out=tensors["res"])):
        with pytest.raises(ValueError, match="must be on the GPU"):
            call()

"""The learning rate of a captured AdamW step is a constant of its graph: a change
of it is warned of, replays keep the rate they were captured with, and a step
captured again takes the new one.

Gradients of ones, no decay, no clipping: M and the root of V are 1 - b^t each, up
to their roundings, so every step takes lr off P, within 40 roundings of lr and
one of P.
"""
import math
import warnings

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def test_a_captured_rate(sp):
    from structured_sparse_transformer_amd.adamw import AdamW
    P, G = torch.zeros(70, device="cuda"), torch.ones(70, device="cuda")
    optimizer = AdamW([P], lr=0.5, weight_decay=0.0, max_norm=math.inf)

    def moved(run, lr):
        start = P.clone()
        run()
        torch.cuda.synchronize()
        assert ((start - P - lr).abs() <= 2.0 ** -24 * (40 * lr + start.abs() + lr)).all()

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            optimizer.step([G])
        return graph

    eager = lambda: optimizer.step([G])  # noqa: E731
    with warnings.catch_warnings():
        warnings.simplefilter("error")   # nothing is captured yet
        moved(eager, 0.5)
        optimizer.set_lr(0.25)
        moved(eager, 0.25)
        old = capture()
    moved(old.replay, 0.25)
    with pytest.warns(RuntimeWarning, match="capture it again"):
        optimizer.set_lr(0.125)
    moved(old.replay, 0.25)
    new = capture()
    for _ in range(3):
        moved(new.replay, 0.125)
        moved(eager, 0.125)
        moved(old.replay, 0.25)
    assert int(sp.control_values(optimizer.control)["step"]) == 13


def test_no_more_than_once(sp):
    from structured_sparse_transformer_amd.adamw import AdamW
    P = torch.zeros(70, device="cuda")
    optimizer = AdamW([P], max_norm=1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        optimizer.step([torch.ones_like(P)])
    with pytest.warns(RuntimeWarning):
        optimizer.set_lr(1e-4)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        optimizer.set_lr(1e-5)

"""GPU checks of the token embedding and its gradient against plain float64
sums.

Tolerances.  Forward: one fp32 product and one rounding to fp16, so within
half an fp16 ulp (relative 2^-11, absolute 2^-25 among subnormals) and the
product's own 2^-24.  Gradient: a sum of n fp16 values held in fp32, in parts
of up to 64 and then over the parts, is within n 2^-24 sum |x| of the exact
sum; the scale's product and the addition to an old value add one rounding
each.
"""
import numpy as np
import pytest

from gpu_checks import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def draw_ids(rng, T, V, kind):
    if kind == "uniform":
        ids = rng.integers(0, V, T)
    elif kind == "skewed":
        ids = np.minimum(np.exp(rng.random(T) * np.log(V + 1)).astype(np.int64) - 1, V - 1)
    elif kind == "one":
        ids = np.full(T, V - 1)
    elif kind == "runs64":           # runs that end exactly where the chunks of 64 do
        ids = (np.arange(T) // 64) % V
    elif kind == "padding":
        ids = np.full(T, -1)
    ids = ids.astype(np.int64)
    if kind in ("uniform", "skewed") and T > 8:
        ids[rng.integers(0, T, T // 8)] = -1
        ids[rng.integers(0, T, 2)] = V           # one past the end is padding too
    return ids


def ref_fwd(ids, table, scale):
    out = np.zeros((len(ids), table.shape[1]))
    ok = (ids >= 0) & (ids < len(table))
    out[ok] = table[ids[ok]].astype(np.float64) * float(np.float32(scale))
    return out


def ref_bwd(ids, dout, V, scale):
    """The sums, and the sums of magnitudes and the counts that bound their rounding."""
    ok = (ids >= 0) & (ids < V)
    s, a, n = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1])), np.zeros(V)
    x = dout.astype(np.float64)
    np.add.at(s, ids[ok], x[ok])
    np.add.at(a, ids[ok], np.abs(x[ok]))
    np.add.at(n, ids[ok], 1)
    f = float(np.float32(scale))
    return s * f, a * abs(f), n


@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (1, 50257, 1600), (3, 7, 8), (63, 1025, 67), (130, 1024, 16),
                                   (257, 3001, 1000), (1000, 500, 2056), (5, 40, 4097)])
@pytest.mark.parametrize("ids32", [False, True])
@pytest.mark.parametrize("table32", [False, True])
def test_forward(sp, T, V, d, ids32, table32):
    rng = np.random.default_rng([T, V, d])
    ids = draw_ids(rng, T, V, "uniform")
    table = rng.standard_normal((V, d)).astype(np.float32 if table32 else np.float16)
    out = Guarded((T, d), torch.float16)
    sp.sp24_embed_fwd(dev(ids.astype(np.int32) if ids32 else ids), dev(table), 1.7, out=out.t)
    out.check()
    ref = ref_fwd(ids, table, 1.7)
    got = out.t.cpu().numpy().astype(np.float64)
    assert (np.abs(got - ref) <= (2.0 ** -11 + U32) * np.abs(ref) + 2.0 ** -25).all()


def test_forward_is_a_copy_at_scale_one_and_takes_any_id(sp):
    rng = np.random.default_rng(5)
    table = (rng.standard_normal((100, 24)) * 2.0 ** -16).astype(np.float16)     # subnormals among them
    ids = np.array([[0, 99, 100, -1], [-2 ** 40, 2 ** 40, 2 ** 32, 50]])
    out = sp.sp24_embed_fwd(dev(ids), dev(table))
    assert tuple(out.shape) == (2, 4, 24)
    got = out.cpu().numpy().view(np.uint16)
    want = np.zeros((2, 4, 24), np.uint16)
    for at in ((0, 0), (0, 1), (1, 3)):
        want[at] = table[ids[at]].view(np.uint16)
    assert (got == want).all()


def test_forward_keeps_what_padding_rows_would_read_out(sp):
    """A table of infinities and NaN: only the rows asked for are read into the output."""
    table = np.full((4, 8), np.inf, np.float16)
    table[1] = np.nan
    table[2] = 3
    out = sp.sp24_embed_fwd(dev(np.array([2, -1, 4, 0, 1])), dev(table), 2.0).cpu().numpy()
    assert (out[0] == 6).all() and (out[1:3] == 0).all() and np.isposinf(out[3]).all() and np.isnan(out[4]).all()


CASES = [(1, 1, 1, "uniform"), (1, 50257, 1600, "uniform"), (517, 1003, 67, "skewed"), (64, 3, 8, "one"),
         (65, 3, 8, "one"), (129, 1024, 32, "runs64"), (640, 1025, 72, "runs64"), (4096, 2049, 24, "skewed"),
         (4097, 1023, 40, "skewed"), (9000, 5000, 16, "one"), (20000, 1, 8, "one"), (300, 20, 2056, "skewed"),
         (300, 20, 515, "skewed"), (1000, 3000, 8, "padding"), (200000, 70000, 8, "skewed"),
         (140000, 300, 3, "skewed"), (5000, 4000, 130, "uniform")]


@pytest.mark.parametrize("T,V,d,kind", CASES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(sp, T, V, d, kind, accumulate):
    rng = np.random.default_rng([T, V, d])
    ids = draw_ids(rng, T, V, kind)
    dout = rng.standard_normal((T, d)).astype(np.float16)
    old = rng.standard_normal((V, d)).astype(np.float32)
    out = Guarded((V, d), torch.float32, fill=0xFF)     # NaN unless written
    if accumulate:
        out.t.copy_(dev(old))
    need = sp.sp24_embed_bwd_workspace(T, V, d)
    ws = Guarded((need,), torch.uint8, fill=0x7F)
    sp.sp24_embed_bwd(dev(ids.astype(np.int32) if d % 2 else ids), dev(dout), V, 0.3, dtable=out.t,
                      accumulate=accumulate, workspace=ws.t)
    out.check()
    ws.check("workspace")
    ref, mag, n = ref_bwd(ids, dout, V, 0.3)
    got = out.t.cpu().numpy().astype(np.float64)
    bound = (n[:, None] + 2) * U32 * mag
    if accumulate:
        ref = ref + old
        bound = bound + U32 * (np.abs(ref) + bound)
        assert (got[n == 0] == old[n == 0]).all()       # rows of absent ids are left alone
    else:
        assert (got[n == 0] == 0).all()
    assert (np.abs(got - ref) <= 1.01 * bound).all()


def test_gradient_is_that_of_the_forward_by_differences(sp):
    """Small whole numbers and a power of two as scale keep every value exact, so the
    change of sum(out * dout) under a change of one table entry is the gradient itself."""
    rng = np.random.default_rng(11)
    V, d, ids = 9, 5, dev(np.array([0, 3, 3, -1, 8, 3, 0, 9]))
    table, dout = dev(rng.integers(-8, 9, (V, d)).astype(np.float32)), dev(rng.integers(-8, 9, (8, d)).astype(np.float16))

    def f(t):
        return (sp.sp24_embed_fwd(ids, t, 0.5).double() * dout.double()).sum().item()

    grad = sp.sp24_embed_bwd(ids, dout, V, 0.5).cpu().numpy()
    base = f(table)
    for v in range(V):
        for c in range(d):
            t = table.clone()
            t[v, c] += 2
            assert (f(t) - base) / 2 == grad[v, c]


def test_no_tokens_and_no_rows(sp):
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert sp.sp24_embed_fwd(none, torch.ones(3, 8, device="cuda")).shape == (0, 8)
    out = torch.full((300, 8), float("nan"), device="cuda")
    sp.sp24_embed_bwd(none, torch.empty(0, 8, dtype=torch.float16, device="cuda"), 300, dtable=out)
    assert (out == 0).all()
    some = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert (sp.sp24_embed_fwd(some, torch.empty(0, 8, device="cuda")) == 0).all()
    assert sp.sp24_embed_bwd(some, torch.ones(4, 8, dtype=torch.float16, device="cuda"), 0).shape == (0, 8)
    assert sp.sp24_embed_bwd(some, torch.ones(4, 0, dtype=torch.float16, device="cuda"), 5).shape == (5, 0)


def test_same_bits_on_every_run_on_another_stream_and_in_a_graph(sp):
    rng = np.random.default_rng(3)
    T, V, d = 6000, 700, 136
    ids, dout = dev(draw_ids(rng, T, V, "skewed")), dev(rng.standard_normal((T, d)).astype(np.float16))
    want = sp.sp24_embed_bwd(ids, dout, V, 1.0).clone()
    for _ in range(3):
        assert torch.equal(sp.sp24_embed_bwd(ids, dout, V, 1.0), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sp.sp24_embed_bwd(ids, dout, V, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    ws = torch.empty(sp.sp24_embed_bwd_workspace(T, V, d), dtype=torch.uint8, device="cuda")
    out = torch.empty(V, d, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sp.sp24_embed_bwd(ids, dout, V, 1.0, dtable=out, workspace=ws)
    for k in range(4):
        dout.mul_(-1)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want if k % 2 else -want)


def test_offsets_past_32_bits(sp):
    """A table of 4.3e9 entries: rows beyond 2^32 entries and bytes."""
    V, d = 70000, 62000
    ids = dev(np.array([V - 1, 0, 69500, V - 1, 69273, -1]))
    table = torch.zeros(V, d, dtype=torch.float16, device="cuda")
    rows = torch.randn(3, d, device="cuda").half()
    at = torch.tensor([V - 1, 69500, 69273], device="cuda")
    table[at] = rows
    out = sp.sp24_embed_fwd(ids, table)
    zero = torch.zeros(d, dtype=torch.float16, device="cuda")
    for k, want in enumerate((rows[0], zero, rows[1], rows[0], rows[2], zero)):
        assert torch.equal(out[k], want)
    del table
    dout = torch.randn(6, d, device="cuda").half()
    grad = torch.full((V, d), float("nan"), device="cuda")
    sp.sp24_embed_bwd(ids, dout, V, dtable=grad)
    assert torch.equal(grad[V - 1], dout[0].float() + dout[3].float())
    assert torch.equal(grad[69500], dout[2].float()) and torch.equal(grad[69273], dout[4].float())
    assert torch.equal(grad[0], dout[1].float())
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[ids[:5]] = False
    for lo in range(0, V, 7000):
        part = grad[lo:lo + 7000]
        assert (part[rest[lo:lo + 7000]] == 0).all()

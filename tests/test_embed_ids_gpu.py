"""Ids as a training loop has them: parts of a token stream that start anywhere,
and views of a batch."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sp():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from structured_sparse_transformer_amd import sp24
    sp24.lib()
    return sp24


VIEWS = {"from 1": lambda t: t[1:65], "from 2": lambda t: t[2:66], "from 3": lambda t: t[3:4], "from 4": lambda t: t[4:68],
         "inputs": lambda t: t.view(10, 30)[:, :-1], "targets": lambda t: t.view(10, 30)[:, 1:],
         "transposed": lambda t: t.view(10, 30).t(), "every other": lambda t: t[::2], "one id for all": lambda t: t[5:6].expand(40)}


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("other_stream", [False, True])
def test_views_of_ids(sp, view, dtype, other_stream):
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(-1, 50, (300,), generator=gen, device="cuda").to(dtype)
    table = torch.randn(50, 24, generator=gen, device="cuda")
    ids = VIEWS[view](tokens)
    dout = torch.randn(*ids.shape, 24, generator=gen, device="cuda").half()
    keep = tokens.clone()
    plain = ids.clone(memory_format=torch.contiguous_format)
    want = sp.sp24_embed_fwd(plain, table, 0.5), sp.sp24_embed_bwd(plain, dout, 50, 0.5)
    real = (plain >= 0).unsqueeze(-1)
    assert torch.equal(want[0], torch.where(real, 0.5 * table[plain.clamp(min=0).long()], 0.0).half())
    stream = torch.cuda.Stream() if other_stream else None
    if other_stream:
        stream.wait_stream(torch.cuda.current_stream())
    got = sp.sp24_embed_fwd(ids, table, 0.5, stream=stream), sp.sp24_embed_bwd(ids, dout, 50, 0.5, stream=stream)
    if other_stream:
        torch.cuda.current_stream().wait_stream(stream)
    assert got[0].shape == (*ids.shape, 24)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(tokens, keep)

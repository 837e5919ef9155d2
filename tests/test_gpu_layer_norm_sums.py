"""GPU layer norm backward: the column sums of many long rows (over 16384
columns, the pass of their own)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def test_long_chains_lose_nothing(gq):
    """A large value in each of the first 64 rows and ones behind it, which are
    half of its last place: one long chain would lose all of them.  A sum of
    chains of c additions is off by c 2^-24 times the magnitudes: 64 rows
    added by themselves, one more addition per 4096 rows, then the 64 parts."""
    rows, cols = 64 * 1500, 16392
    a = gq.act(rows, cols, torch.bfloat16)
    dy = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    dy[:64] = 2.0 ** 24
    # x - mean = 1 and 1 / std = 1 in every place, so both sums are dy's
    x = torch.full((rows, cols), 3.0, dtype=torch.bfloat16, device="cuda")
    mean, rstd = torch.full((rows,), 2.0, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    gq.gq_layer_norm_backward(a, dy, x, mean, rstd, None, x, dw, db,
                              workspace=gq.alloc_workspace(gq.gq_layer_norm_workspace(a)))
    want = 64 * 2.0 ** 24 + rows - 64
    bound = (64 + rows / 4096 + 1 + 64) * U32 * want
    for got in (dw, db):
        assert float((got.double() - want).abs().max()) <= bound
    del dy, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 4095, 4097, 4200])
def test_whole_numbers(gq, rows):
    """Sums of whole numbers are exact, whatever the split."""
    cols = 16393
    a = gq.act(rows, cols, torch.float16)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    dy = torch.randint(-8, 9, (rows, cols), generator=gen, device="cuda").half()
    x = torch.randint(-8, 9, (rows, cols), generator=gen, device="cuda").half()
    mean, rstd = torch.ones(rows, device="cuda"), torch.full((rows,), 2.0, device="cuda")
    dx = torch.empty_like(x)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    gq.gq_layer_norm_backward(a, dy, x, mean, rstd, None, dx, dw, db,
                              workspace=gq.alloc_workspace(gq.gq_layer_norm_workspace(a)))
    d = dy.double()
    assert torch.equal(db.double(), d.sum(0))
    assert torch.equal(dw.double(), (d * (x.double() - 1) * 2).sum(0))

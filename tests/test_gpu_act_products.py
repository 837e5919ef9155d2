"""GPU weight gradient: how exact its products are in each type.  fp16 takes one
exact product per token; fp32 takes three, whose terms end at 2^-133."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES, U32, values, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def run(gq, dy, codes, steps, cols, dtype, group=0):
    rows, out = dy.shape
    a = gq.act(rows, cols, TYPES[dtype], group)
    dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
    gq.gq_act_wgrad(a, torch.as_tensor(dy).to(TYPES[dtype]).cuda(), torch.as_tensor(codes).cuda(),
                    torch.as_tensor(steps).cuda(), dw, db,
                    workspace=gq.alloc_workspace(gq.gq_act_wgrad_workspace(a, out)))
    return dw, db


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,group", [(50, 60, 70, 0), (300, 200, 130, 32),
                                                 (1500, 104, 260, 64), (4000, 48, 64, 0)])
def test_one_product_per_token(gq, dtype, rows, out, cols, group):
    """n exact products: n additions, each off by at most 2^-23 (it may round
    towards zero), and 64 more that join splits and lanes."""
    x, dy = values(rows, rows, cols, dtype), values(out, rows, out, dtype)
    codes, steps = A.pack(x, group, dtype)
    dw, db = run(gq, dy, codes, steps, cols, dtype, group)
    xr = A.unpack(codes, steps, cols, group)
    ww, wb = A.wgrad(dy, xr)
    k = 2 * (rows + 64) * U32
    within(dw, ww, k * (np.abs(dy).T @ np.abs(xr)))
    within(db, wb, k * np.abs(dy).sum(axis=0))
    # as a whole: n roundings add up like a random walk
    got = dw.double().cpu().numpy()
    assert np.linalg.norm(got - ww) / np.linalg.norm(ww) <= 4 * np.sqrt(rows) * U32


@pytest.mark.parametrize("exp", [-100, -109, -111, -120, -126, -130])
def test_the_smallest_fp32_gradients(gq, exp):
    """One token: below 2^-110 the third term is cut at 2^-133, above nothing is;
    the three terms' additions round twice."""
    rng = np.random.default_rng([16, -exp])
    dy = ((1 + rng.random((1, 64))) * 2.0 ** exp).astype(np.float32).astype(np.float64)
    codes = np.zeros((1, 16), np.int8)
    codes[0, :3] = 1, -64, 127
    steps = np.full((1, 1), 2.0 ** 100, np.float32)
    dw, db = run(gq, dy, codes, steps, 3, "f32")
    xr = A.unpack(codes, steps, 3)
    want = dy.T @ xr
    cut = 2.0 ** -133 if exp < -110 else 0.0
    within(dw, want, 2 * 2 * U32 * np.abs(want) + cut * np.abs(xr))
    assert np.array_equal(db.double().cpu().numpy(), dy[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_infinite_gradients_show_where_they_are_used(gq, dtype):
    rng = np.random.default_rng(17)
    dy = rng.integers(-4, 5, (90, 24)).astype(np.float64)
    dy[50, 7] = np.inf
    codes, steps = A.pack(rng.standard_normal((90, 40)), 0, dtype)
    codes[50, :40] = np.where(codes[50, :40] == 0, 1, codes[50, :40])
    dw, db = run(gq, dy, codes, steps, 40, dtype)
    bad = ~torch.isfinite(dw).cpu().numpy()
    assert np.array_equal(bad, np.arange(24)[:, None] == np.full((1, 40), 7))
    assert np.array_equal(torch.isinf(db).cpu().numpy(), np.arange(24) == 7)
    if dtype != "f32":                   # fp32 in three terms: NaN
        sign = np.sign(codes[50, :40])
        assert np.array_equal(dw[7].cpu().numpy(), sign * np.inf)

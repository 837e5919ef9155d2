"""Long sums of the product from 8-bit floating point forms: terms of one sign, where
cuts all go one way, and terms that cancel, where what was cut stands beside a small
result.  The bounds are those of test_gpu_block_linear.py: 16-bit results are off by
at most 2^-10 of the sum of the terms' magnitudes before their rounding, eight cuts of
up to 2^-13 of the largest of eight; fp32 results by the additions' roundings.  How far
they are off is printed (pytest -s)."""
import numpy as np
import pytest
import torch

from oracle import step as S
from tests.act_util import TYPES, rounding, within
from tests.test_gpu_block_linear import d8, dev

pytestmark = pytest.mark.gpu
COLS, OUT, STEP = 16384, 70, 2.0 ** -9


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def operands(kind, rows):
    """Codes of all sizes, so that products lie far apart; for terms that cancel the
    second half of a row's columns, in another order for all rows and weights alike,
    is the first with the other sign in x, but for 16 columns."""
    rng = np.random.default_rng([30, rows])
    x = rng.integers(0, 0x7f, (rows, COLS)).astype(np.uint8)
    w = rng.integers(0, 0x7f, (OUT, COLS)).astype(np.uint8)
    if kind == "cancelling":
        half = COLS // 2
        x[:, half:], w[:, half:] = x[:, :half] | 0x80, w[:, :half]
        x[:, half:half + 16] = 0
        order = rng.permutation(COLS)
        x, w = x[:, order], w[:, order]
    return np.ascontiguousarray(x), np.ascontiguousarray(w)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["same sign", "cancelling"])
@pytest.mark.parametrize("rows", [20, 200])
def test_sums(gq, rows, kind, dtype):
    x, w = operands(kind, rows)
    a = gq.act(rows, COLS, TYPES[dtype], 128)
    y = torch.empty(rows, OUT, dtype=TYPES[dtype], device="cuda")
    steps = torch.full((rows, a.groups), STEP, device="cuda")
    gq.gq_block_linear(a, d8(x), steps, d8(w), steps[:1], None, y,
                       workspace=gq.alloc_workspace(gq.gq_block_linear_workspace(a, OUT)))
    xv, wv = S.values(x) * STEP, S.values(w) * STEP
    want, mag = xv @ wv.T, np.abs(xv) @ wv.T
    off = np.abs(y.double().cpu().numpy() - want)
    print(f"off by {(off / mag).max():.2g} of the magnitudes at most, in the 2-norm "
          f"{np.linalg.norm(off) / np.linalg.norm(want):.2g} of the results")
    tol = ((COLS + 2) * 2.0 ** -23 + (0.0 if dtype == "f32" else 2.0 ** -10)) * mag
    within(y, want, tol + rounding(np.abs(want) + tol, dtype))

"""GPU 8-bit integer linear layer against the CPU form: the integer sum is
exact, so a result is off by four fp32 roundings of its terms and one of its
type."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES, U32, matrix, rounding, untouched, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def operands(seed, rows, out, cols, low=-127, high=127):
    rng = np.random.default_rng([6, seed])

    def codes(n):
        c = np.zeros((n, A.pitch(cols)), np.int8)
        c[:, :cols] = rng.integers(low, high + 1, (n, cols))
        return c

    f = lambda *s: np.exp(rng.standard_normal(s)).astype(np.float32)  # noqa: E731
    return (codes(rows), f(rows, 1) / 100, codes(out), f(out) / 100,
            rng.standard_normal(out).astype(np.float32))


def check(gq, rows, out, cols, dtype, bias=True, pad=0, lead=0, seed=0, ops=None):
    c, s, wc, ws, b = ops or operands(seed, rows, out, cols)
    a = gq.act(rows, cols, TYPES[dtype])
    y, buf, mask = matrix(np.zeros((rows, out)), TYPES[dtype], pad, lead)
    work = gq.alloc_workspace(gq.gq_act_linear_workspace(a, out))
    if work is not None:
        work.fill_(0x55)
    d = lambda v: torch.as_tensor(v).cuda()  # noqa: E731
    gq.gq_act_linear(a, d(c), d(s), d(wc), d(ws), d(b) if bias else None, y, workspace=work)
    want = A.linear(c, s, wc, ws, b if bias else None, cols)
    prod = A.linear(c, s, wc, ws, None, cols)
    tol = 4 * U32 * (np.abs(prod) + np.abs(want))
    within(y, want, tol + rounding(np.abs(want) + tol, dtype))
    assert untouched(buf, mask)
    return y


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,pad,lead", [
    (1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (1, 4096, 4096, 0, 0), (1, 1001, 777, 0, 1),
    (2, 130, 16, 1, 3), (3, 33, 1030, 0, 0), (16, 512, 2048, 0, 0), (17, 511, 100, 1, 1),
    (31, 65, 129, 0, 0), (33, 257, 513, 3, 2), (64, 128, 128, 0, 0), (65, 200, 260, 0, 0),
    (129, 131, 4100, 1, 1), (200, 520, 1000, 0, 0), (300, 300, 64, 0, 0)])
def test_sizes(gq, dtype, rows, out, cols, pad, lead):
    check(gq, rows, out, cols, dtype, pad=pad, lead=lead, seed=rows)
    check(gq, rows, out, cols, dtype, bias=False, seed=cols)


@pytest.mark.parametrize("rows", [1, 5, 16, 32, 48, 64, 80, 128, 256, 257])
@pytest.mark.parametrize("cols", [48, 1024, 6000])
def test_row_counts(gq, rows, cols):
    check(gq, rows, 272, cols, "bf16", seed=rows)


def test_large_tiles(gq):
    check(gq, 2049, 4100, 300, "bf16")
    check(gq, 4096, 2048, 256, "f16")
    check(gq, 2500, 2500, 129, "f32")


def test_long_sums_are_split(gq):
    """Few tiles and a long sum: split and joined."""
    a = gq.act(1111, 16000, torch.bfloat16)
    assert gq.gq_act_linear_workspace(a, 1000) > 0
    check(gq, 1111, 1000, 16000, "bf16", pad=3, lead=1)
    check(gq, 1100, 1001, 15001, "f32", bias=False)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_extreme_codes(gq, rows):
    """All codes at the ends, over the longest sum that 32 bits hold."""
    cols, out = 131071, 48
    for x, w in ((-128, -128), (-128, 127), (127, 127)):
        c = np.full((rows, A.pitch(cols)), x, np.int8)
        wc = np.full((out, A.pitch(cols)), w, np.int8)
        c[:, cols:] = wc[:, cols:] = 0
        check(gq, rows, out, cols, "f32", bias=False,
              ops=(c, np.ones((rows, 1), np.float32), wc, np.ones(out, np.float32),
                   np.zeros(out, np.float32)))


def test_tokens_that_are_not_finite_stay_alone(gq):
    c, s, wc, ws, b = operands(1, 70, 140, 200)
    s[3], s[69] = np.nan, np.inf
    ws[7] = np.nan
    c[3] = 0
    wc[7] = 0
    check(gq, 70, 140, 200, "bf16", ops=(c, s, wc, ws, b))


def test_single_tokens_equal_the_batch(gq):
    """The same token gives the same bits alone and in any batch."""
    ops = operands(2, 300, 500, 1500)
    c, s, wc, ws, b = ops
    batch = check(gq, 300, 500, 1500, "f32", ops=ops)
    for lo, n in ((0, 1), (299, 1), (10, 16), (100, 70)):
        part = check(gq, n, 500, 1500, "f32", ops=(c[lo:lo + n], s[lo:lo + n], wc, ws, b))
        assert torch.equal(part, batch[lo:lo + n])


def test_no_rows(gq):
    a = gq.act(0, 64, torch.bfloat16)
    c, s = gq.alloc_act(a)
    w = torch.zeros(8, 64, dtype=torch.int8, device="cuda")
    gq.gq_act_linear(a, c, s, w, torch.ones(8, device="cuda"), None,
                     torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"))

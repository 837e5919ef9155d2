"""GPU 8-bit activation operators at the ends of their buffers: matrices with
nothing behind them, and matrices with values behind them that would show.
Whole numbers, so the sums are exact."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def at_the_end(values, dtype):
    """A contiguous device matrix whose last value is its buffer's last."""
    n = values.size
    size = -(-n // 512) * 512                # whole blocks of the allocator
    buf = torch.full((size,), float("nan"), dtype=dtype, device="cuda")
    m = buf[size - n:].view(values.shape)
    m.copy_(torch.as_tensor(values))
    return m


def before(values, dtype, poison, rows=200):
    """A contiguous device matrix with `rows` more rows of poison behind it."""
    buf = torch.full((values.shape[0] + rows, values.shape[1]), poison, dtype=dtype,
                     device="cuda")
    buf[:values.shape[0]] = torch.as_tensor(values)
    return buf[:values.shape[0]]


def numbers(seed, rows, out, cols, group):
    rng = np.random.default_rng([12, seed])
    dy = rng.integers(-4, 5, (rows, out)).astype(np.float64)
    codes = np.zeros((rows, A.pitch(cols)), np.int8)
    codes[:, :cols] = rng.integers(-127, 128, (rows, cols))
    steps = 2.0 ** rng.integers(0, 3, (rows, A.groups(cols, group))).astype(np.float32)
    assert rows * 4 * 127 * 4 < 2 ** 24
    return dy, codes, steps


def wgrad(gq, dy, codes, steps, cols, dtype, group, place):
    rows, out = dy.shape
    a = gq.act(rows, cols, TYPES[dtype], group)
    dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
    work = gq.alloc_workspace(gq.gq_act_wgrad_workspace(a, out))
    if place == "end":
        d = at_the_end(dy, TYPES[dtype])
        c, s = torch.as_tensor(codes).cuda(), torch.as_tensor(steps).cuda()
    else:
        d = before(dy, TYPES[dtype], float("nan"))
        c, s = before(codes, torch.int8, 127), before(steps, torch.float32, float("nan"))
    gq.gq_act_wgrad(a, d, c, s, dw, db, workspace=work)
    ww, wb = A.wgrad(dy, A.unpack(codes, steps, cols, group))
    assert np.array_equal(dw.double().cpu().numpy(), ww)
    assert np.array_equal(db.double().cpu().numpy(), wb)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", [1, 2, 3, 4, 5, 6, 7, 9])
def test_weight_gradient_of_few_features_at_the_end_of_memory(gq, dtype, out):
    for rows in (33, 35, 38, 64, 65, 70, 129, 1000):
        dy, codes, steps = numbers(rows, rows, out, 40, 32)
        wgrad(gq, dy, codes, steps, 40, dtype, 32, "end")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 15, 31, 63, 65, 100, 200, 2011])
@pytest.mark.parametrize("out,cols,group", [(8, 16, 0), (24, 100, 32), (130, 48, 0),
                                            (264, 260, 64)])
def test_weight_gradient_reads_zeros_behind_the_last_row(gq, dtype, rows, out, cols, group):
    wgrad(gq, *numbers(rows, rows, out, cols, group), cols, dtype, group, "before")


@pytest.mark.parametrize("rows", [1, 17, 33, 50, 65, 130, 300])
@pytest.mark.parametrize("out,cols", [(1, 16), (17, 100), (40, 64), (63, 1000), (131, 272)])
def test_integer_product_reads_zeros_behind_the_last_rows(gq, rows, out, cols):
    rng = np.random.default_rng([13, rows, out])
    _, x, _ = numbers(rows, rows, 1, cols, 0)
    _, w, _ = numbers(out, out, 1, cols, 0)
    s = 2.0 ** rng.integers(0, 3, (rows, 1)).astype(np.float32)
    v = 2.0 ** rng.integers(-3, 0, out).astype(np.float32)
    b = rng.integers(-9, 9, out).astype(np.float32)
    a = gq.act(rows, cols, torch.float32)
    y = torch.full((rows + 9, out), 77.0, device="cuda")
    nan = float("nan")
    gq.gq_act_linear(
        a, before(x, torch.int8, 127), before(s, torch.float32, nan),
        before(w, torch.int8, 127), before(v[:, None], torch.float32, nan).view(-1),
        before(b[:, None], torch.float32, nan).view(-1), y[:rows],
        workspace=gq.alloc_workspace(gq.gq_act_linear_workspace(a, out)))
    # sums below 1000 * 127^2 < 2^24 times powers of two: only the bias rounds
    want = A.linear(x, s, w, v, b, cols)
    off = np.abs(y[:rows].double().cpu().numpy() - want)
    assert (off <= 2 * 2.0 ** -24 * (np.abs(want) + np.abs(b))).all()
    assert (y[rows:] == 77.0).all()

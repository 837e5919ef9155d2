"""GPU weight and bias gradient from the 8-bit form against the CPU form.

Products are exact, so with small whole numbers the sums are exact too and
have to be equal; otherwise a sum of n products is off by at most 2 n 2^-24
times the sum of their magnitudes (n counts each term that a value is split
into, three for fp32 and up to two for fp16; an accumulation may round towards
zero, hence the 2)."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES, U32, matrix, untouched, values, within

pytestmark = pytest.mark.gpu
TERMS = {"bf16": 1, "f16": 2, "f32": 3}


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def run(gq, dy, codes, steps, cols, dtype, group, pad=0, lead=0, beta=0.0, bias=True):
    rows, out = dy.shape
    a = gq.act(rows, cols, TYPES[dtype], group)
    dyt, _, _ = matrix(dy, TYPES[dtype], pad, lead)
    n = out * cols
    flat = torch.full((n + out + 9,), 77.0, device="cuda")    # odd places of a flat gradient
    dw, db = flat[3:3 + n], flat[6 + n:6 + n + out]
    rng = np.random.default_rng([7, out])
    old = rng.integers(-8, 9, n + out).astype(np.float32)
    dw.copy_(torch.as_tensor(old[:n]))
    db.copy_(torch.as_tensor(old[n:]))
    work = gq.alloc_workspace(gq.gq_act_wgrad_workspace(a, out))
    if work is not None:
        work.fill_(0xFF)                                     # NaN
    gq.gq_act_wgrad(a, dyt, torch.as_tensor(codes).cuda(), torch.as_tensor(steps).cuda(), dw,
                    db if bias else None, beta=beta, workspace=work)
    edge = torch.cat([flat[:3], flat[3 + n:6 + n], flat[6 + n + out:]])
    assert (edge == 77.0).all()
    return (dw.view(out, cols), db, old[:n].reshape(out, cols).astype(np.float64),
            old[n:].astype(np.float64))


def exact(gq, rows, out, cols, dtype, group=0, pad=0, lead=0, beta=0.0, bias=True, seed=0):
    """Whole numbers whose sums are exact in fp32."""
    rng = np.random.default_rng([8, seed])
    dy = rng.integers(-4, 5, (rows, out)).astype(np.float64)
    codes = np.zeros((rows, A.pitch(cols)), np.int8)
    codes[:, :cols] = rng.integers(-127, 128, (rows, cols))
    steps = 2.0 ** rng.integers(0, 3, (rows, A.groups(cols, group))).astype(np.float32)
    assert rows * 4 * 127 * 4 < 2 ** 24
    dw, db, ow, ob = run(gq, dy, codes, steps, cols, dtype, group, pad, lead, beta, bias)
    ww, wb = A.wgrad(dy, A.unpack(codes, steps, cols, group))
    assert np.array_equal(dw.double().cpu().numpy(), ww + beta * ow)
    assert np.array_equal(db.double().cpu().numpy(), wb + beta * ob if bias else ob)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,pad,lead", [
    (1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (31, 7, 5, 1, 1), (32, 128, 128, 0, 0),
    (33, 129, 131, 3, 2), (64, 256, 256, 0, 0), (65, 260, 272, 4, 0), (100, 1, 300, 0, 0),
    (257, 40, 1001, 0, 3), (1000, 300, 70, 0, 0), (513, 512, 512, 8, 8), (129, 640, 257, 0, 0),
    (700, 1030, 1040, 2, 0)])
def test_whole_numbers(gq, dtype, rows, out, cols, pad, lead):
    exact(gq, rows, out, cols, dtype, 0, pad, lead, seed=rows)
    exact(gq, rows, out, cols, dtype, 32, pad, lead, beta=1.0, seed=cols)


@pytest.mark.parametrize("group", [32, 64, 128, 512, 1024, 32768])
@pytest.mark.parametrize("cols", [100, 520, 2050])
def test_groups(gq, group, cols):
    exact(gq, 200, 150, cols, "bf16", group)
    exact(gq, 77, 72, cols, "f16", group, beta=0.5)


@pytest.mark.parametrize("rows", [2000, 5000, 8255])
def test_long_sums(gq, rows):
    """Split over tokens and joined."""
    exact(gq, rows, 96, 130, "bf16", 64)
    exact(gq, rows, 64, 64, "f16", 0, beta=1.0)
    exact(gq, rows, 20, 40, "f32", 32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,group", [(50, 60, 70, 0), (300, 200, 130, 32),
                                                 (1500, 100, 260, 64), (4000, 48, 64, 0)])
def test_real_values(gq, dtype, rows, out, cols, group):
    x, dy = values(rows, rows, cols, dtype), values(out, rows, out, dtype) * 2.0 ** -8
    dy = torch.as_tensor(dy).to(TYPES[dtype]).double().numpy()
    codes, steps = A.pack(x, group, dtype)
    dw, db, _, _ = run(gq, dy, codes, steps, cols, dtype, group)
    xr = A.unpack(codes, steps, cols, group)
    ww, wb = A.wgrad(dy, xr)
    k = 2 * (TERMS[dtype] * rows + 64) * U32
    within(dw, ww, k * (np.abs(dy).T @ np.abs(xr)))
    within(db, wb, k * np.abs(dy).sum(axis=0))
    # and as a whole far nearer than that bound: errors of n roundings add
    # up like a random walk, sqrt(n) 2^-24 of a sum's own size or less
    got = dw.double().cpu().numpy()
    rel = np.linalg.norm(got - ww) / np.linalg.norm(ww)
    assert rel <= 4 * np.sqrt(TERMS[dtype] * rows) * U32


def test_full_range_of_fp32_gradients(gq):
    """24 significant bits and wide exponents reach the sum: one token."""
    rng = np.random.default_rng(9)
    dy = (rng.standard_normal((1, 300)) * np.exp(rng.uniform(-40, 40, 300))).astype(np.float32)
    codes = np.zeros((1, 16), np.int8)
    codes[0, :3] = 1, -64, 127
    steps = np.ones((1, 1), np.float32)
    dw, db, _, _ = run(gq, dy.astype(np.float64), codes, steps, 3, "f32", 0)
    want = np.outer(dy[0].astype(np.float64), [1, -64, 127])
    assert np.array_equal(db.cpu().numpy(), dy[0])
    within(dw, want, 3 * U32 * np.abs(want))
    assert np.array_equal(dw.cpu().numpy()[:, :2], want[:, :2].astype(np.float32))


def test_the_ends_of_fp16(gq):
    """Subnormal and largest values of both operands: one product per sum, so
    each is off by the accumulation's one rounding at most."""
    tiny = 2.0 ** -24
    x = np.zeros((5, 40))
    x[0, :8] = np.arange(8) * tiny                 # steps below 2^-24
    x[1, :8] = 65504.0, -65504.0, 40000.0, 1.0, 0.0, 512.0, 60000.0, -33000.0
    x[2, :8] = 2.0 ** -14 * (1 + np.arange(8) / 8)
    x[3, 0] = tiny
    x[4, :8] = 127 * tiny, 128 * tiny, tiny, 0, 3 * tiny, 64 * tiny, 100 * tiny, -tiny
    codes, steps = A.pack(x, 32, "f16")
    xr = A.unpack(codes, steps, 40, 32)
    dy = np.zeros((5, 5))
    for t, v in enumerate((1.0, 0.5, 3 * tiny, -1023 * tiny, 65504.0)):
        dy[t, t] = v
    dw, db, _, _ = run(gq, dy, codes, steps, 40, "f16", 32)
    want = dy.T @ xr
    within(dw, want, 2 * U32 * np.abs(want))
    assert np.count_nonzero(dw.cpu().numpy()) == np.count_nonzero(want)
    within(db, dy.sum(axis=0), np.zeros(5))


def test_values_that_are_not_finite_stay_in_their_sums(gq):
    rng = np.random.default_rng(10)
    dy = rng.integers(-4, 5, (90, 200)).astype(np.float64)
    dy[50, 7] = np.nan
    codes, steps = A.pack(rng.standard_normal((90, 160)), 32)
    steps[20, 3] = np.nan                          # columns 96..127
    codes[20, 96:128] = 0
    for dtype in ("bf16", "f16", "f32"):
        dw, db, _, _ = run(gq, dy, codes, steps, 160, dtype, 32)
        bad = torch.isnan(dw).cpu().numpy()
        want = np.zeros((200, 160), bool)
        want[7] = True
        want[:, 96:128] = True
        assert np.array_equal(bad, want)
        assert np.array_equal(torch.isnan(db).cpu().numpy(), np.arange(200) == 7)


def test_no_rows_and_no_bias(gq):
    exact(gq, 40, 30, 50, "bf16", bias=False, beta=2.0)
    exact(gq, 4000, 30, 50, "bf16", bias=False)
    for dtype in TYPES:
        dw, db, ow, ob = run(gq, np.zeros((0, 30)), np.zeros((0, 64), np.int8),
                             np.zeros((0, 1), np.float32), 50, dtype, 0, beta=0.5)
        assert np.array_equal(dw.double().cpu().numpy(), 0.5 * ow)
        assert np.array_equal(db.double().cpu().numpy(), 0.5 * ob)


def test_repeats_bit_for_bit(gq):
    dy, x = values(1, 5000, 100, "bf16"), values(2, 5000, 90, "bf16")
    codes, steps = A.pack(x[:, :90], 32)
    p = run(gq, dy, codes, steps, 90, "bf16", 32)
    q = run(gq, dy, codes, steps, 90, "bf16", 32)
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])

"""GPU weight and bias gradients from 8-bit floating point forms, alone and by
expert, against the 64-bit sums.  Products are exact; where sums are whole
numbers below 2^24 the results are equal, otherwise a sum of n products is off by
at most 2 n 2^-24 times the sum of their magnitudes (n counts the three terms of
an fp32 value; an accumulation may round towards zero, hence the 2)."""
import numpy as np
import pytest
import torch

from oracle import step as S
from tests.act_util import TYPES, U32, matrix, values, within
from tests.test_gpu_block_linear import d8, dev, table

pytestmark = pytest.mark.gpu
TERMS = {"bf16": 1, "f16": 1, "f32": 3}


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def run(gq, dy, x, cols, dtype, off=None, pad=0, lead=0, beta=0.0, bias=True):
    rows, out = dy.shape
    k = 1 if off is None else len(off) - 1
    a = gq.act(rows, cols, TYPES[dtype], 128)
    dyt, _, _ = matrix(dy, TYPES[dtype], pad, lead)
    n, m = k * out * cols, k * out
    flat = torch.full((n + m + 9,), 77.0, device="cuda")      # odd places of a flat gradient
    dw, db = flat[3:3 + n], flat[6 + n:6 + n + m]
    old = np.random.default_rng([7, out]).integers(-8, 9, n + m).astype(np.float32)
    dw.copy_(torch.as_tensor(old[:n]))
    db.copy_(torch.as_tensor(old[n:]))
    work = gq.alloc_workspace(gq.gq_block_wgrad_workspace(a, out, k))
    if work is not None:
        work.fill_(0xFF)                                     # NaN
    gq.gq_block_wgrad(a, dyt, d8(x[0]), dev(x[1]), dw, db if bias else None,
                    offsets=None if off is None else dev(off), beta=beta, workspace=work)
    edge = torch.cat([flat[:3], flat[3 + n:6 + n], flat[6 + n + m:]])
    assert bool((edge == 77.0).all())
    return (dw.view(k, out, cols).double().cpu().numpy(), db.view(k, out).double().cpu().numpy(),
            old[:n].reshape(k, out, cols).astype(np.float64),
            old[n:].reshape(k, out).astype(np.float64))


def exact(gq, rows, out, cols, dtype, experts=1, pad=0, lead=0, beta=0.0, bias=True, before=0,
          behind=0, seed=0, off=None):
    rng = np.random.default_rng([11, seed])
    dy = rng.integers(-4, 5, (rows, out)).astype(np.float64)
    codes = np.zeros((rows, S.pitch(cols)), np.uint8)
    codes[:, :cols] = rng.choice(np.array([0, 0x38, 0x40, 0x48, 0xb8, 0xc4, 0x50], np.uint8),
                                 (rows, cols))            # -3, -1, 0 .. 8
    steps = np.exp2(rng.integers(0, 4, (rows, S.blocks(cols)))).astype(np.float32)
    assert rows * 4 * 8 * 8 < 2 ** 24
    if off is None and (experts > 1 or before or behind):
        off = table(rng, rows, experts, before, behind)
    dw, db, ow, ob = run(gq, dy, (codes, steps), cols, dtype, off, pad, lead, beta, bias)
    ww, wb = S.wgrad(dy, S.unpack(codes, steps, cols), [0, rows] if off is None else off)
    assert np.array_equal(dw, ww + beta * ow)
    assert np.array_equal(db, wb + beta * ob if bias else ob)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,pad,lead", [
    (1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (31, 7, 5, 1, 1), (32, 128, 128, 0, 0),
    (33, 129, 131, 3, 2), (64, 256, 256, 0, 0), (65, 260, 272, 4, 0), (100, 1, 300, 0, 0),
    (257, 40, 1001, 0, 3), (1000, 300, 70, 0, 0), (513, 512, 512, 8, 8), (700, 1030, 1040, 2, 0)])
def test_whole_numbers(gq, dtype, rows, out, cols, pad, lead):
    exact(gq, rows, out, cols, dtype, 1, pad, lead, seed=rows)
    exact(gq, rows, out, cols, dtype, 1, pad, lead, beta=1.0, before=rows // 5,
          behind=rows // 7, seed=cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,experts,before,behind,pad", [
    (1, 9, 40, 4, 0, 0, 0), (7, 64, 128, 16, 0, 0, 0), (32, 100, 260, 5, 3, 4, 0),
    (64, 129, 300, 64, 0, 1, 0), (200, 272, 500, 3, 1, 0, 8), (513, 136, 129, 9, 0, 30, 0),
    (1500, 72, 200, 30, 0, 0, 1), (300, 600, 512, 2, 17, 5, 0), (60, 2, 3, 1024, 0, 2, 0)])
def test_experts(gq, dtype, rows, out, cols, experts, before, behind, pad):
    exact(gq, rows, out, cols, dtype, experts, pad, 0, before=before, behind=behind, seed=rows)
    exact(gq, rows, out, cols, dtype, experts, pad, 0, beta=0.5, before=before, behind=behind,
          bias=False, seed=cols)


@pytest.mark.parametrize("experts", [1, 3])
@pytest.mark.parametrize("rows", [2000, 5000, 8255])
def test_long_sums(gq, rows, experts):
    """Split over tokens and joined."""
    a = gq.act(rows, 130, torch.bfloat16, 128)
    assert gq.gq_block_wgrad_workspace(a, 96, experts) > 0
    exact(gq, rows, 96, 130, "bf16", experts)
    exact(gq, rows, 64, 64, "f16", experts, beta=1.0, before=3, behind=100)
    exact(gq, rows, 20, 40, "f32", experts)


def test_one_expert_has_all_rows_or_none(gq):
    for rows in (40, 3000):
        for e in range(3):
            off = np.array([0] * (e + 1) + [rows] * (3 - e), np.int64)
            exact(gq, rows, 136, 200, "bf16", 3, off=off, beta=1.0)
        exact(gq, rows, 136, 200, "f32", 3, off=np.array([9, 9, 9, 9], np.int64))


def test_no_rows(gq):
    a = gq.act(0, 50, torch.bfloat16, 128)
    c, s = gq.alloc_block(a)
    for beta, want in ((0.0, 0.0), (0.5, 1.0)):
        dw, db = torch.full((2, 7, 50), 2.0, device="cuda"), torch.full((14,), 2.0, device="cuda")
        gq.gq_block_wgrad(a, torch.empty(0, 7, dtype=torch.bfloat16, device="cuda"), c, s, dw, db,
                        offsets=torch.zeros(3, dtype=torch.int64, device="cuda"), beta=beta,
                        workspace=gq.alloc_workspace(gq.gq_block_wgrad_workspace(a, 7, 2)))
        assert bool((dw == want).all()) and bool((db == want).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,experts", [(50, 60, 70, 1), (300, 200, 130, 4),
                                                   (2100, 128, 384, 2)])
def test_values(gq, dtype, rows, out, cols, experts):
    x = values(1, rows, cols, dtype)
    form = S.pack(x, dtype)
    dy = values(2, rows, out, dtype)
    off = table(np.random.default_rng(3), rows, experts)
    dw, db, _, _ = run(gq, dy, form, cols, dtype, off)
    xh = S.unpack(*form, cols)
    ww, wb = S.wgrad(dy, xh, off)
    mw, mb = S.wgrad(np.abs(dy), np.abs(xh), off)
    n = TERMS[dtype] * rows + 40        # additions, and the parts' join
    within(dw, ww, 2 * n * U32 * mw)
    within(db, wb, 2 * n * U32 * mb)


def test_gradient_against_differences(gq):
    """The gradient of sum(dy * (x^ w^T + b)) by differences of that sum, which
    is linear in w and b: exact but for rounding."""
    rng = np.random.default_rng(12)
    rows, out, cols, off = 90, 20, 150, np.array([0, 40, 40, 90])
    x = values(5, rows, cols, "bf16")
    form = S.pack(x, "bf16")
    dy = rng.integers(-4, 5, (rows, out)).astype(np.float64)
    dw, db, _, _ = run(gq, dy, form, cols, "bf16", off.astype(np.int64))
    w, b = rng.standard_normal((3, out, cols)), rng.standard_normal((3, out))
    xh = S.unpack(*form, cols)

    def loss(w, b):
        return (S.linear(xh, w, b, off)[0] * dy).sum()

    for _ in range(20):
        e, o, c = rng.integers(3), rng.integers(out), rng.integers(cols)
        d = np.zeros_like(w)
        d[e, o, c] = 1.0
        got = (loss(w + d, b) - loss(w - d, b)) / 2
        assert abs(got - dw[e, o, c]) < 1e-3 * max(1.0, abs(got))
        d = np.zeros_like(b)
        d[e, o] = 1.0
        assert abs((loss(w, b + d) - loss(w, b - d)) / 2 - db[e, o]) < 1e-6


def test_rows_of_others_do_not_leak(gq):
    """NaN and infinities in rows of no expert and of another expert."""
    rng = np.random.default_rng(13)
    rows, out, cols = 200, 136, 160
    for dtype, o in (("bf16", out), ("f16", 131), ("f32", out)):
        dy = rng.integers(-4, 5, (rows, o)).astype(np.float64)
        codes = np.full((rows, cols), 0x38, np.uint8)
        steps = np.ones((rows, 2), np.float32)
        off = np.array([10, 90, 150], np.int64)
        for bad in (slice(0, 10), slice(150, 200)):
            dy[bad] = np.nan
            steps[bad] = np.nan
        dy[100, 5] = np.inf
        dw, db, _, _ = run(gq, dy, (codes, steps), cols, dtype, off)
        fine = np.ones((2, o), bool)
        fine[1, 5] = False
        assert np.isfinite(dw[fine]).all() and np.isfinite(db[fine]).all()
        assert not np.isfinite(dw[1, 5]).any() and not np.isfinite(db[1, 5])
        assert np.array_equal(db[0], dy[10:90].sum(0))


def test_tables_out_of_range_stay_in_bounds(gq):
    rows, out, cols = 90, 40, 140
    codes = np.full((rows, S.pitch(cols)), 0x38, np.uint8)
    steps = np.ones((rows, 2), np.float32)
    for off in ([-5, 20, 10, 400, 91], [0, 1 << 40, -1 << 40, 50, 90], [90, 60, 30, 10, 0]):
        run(gq, np.ones((rows, out)), (codes, steps), cols, "bf16", np.array(off, np.int64))
    torch.cuda.synchronize()

"""GPU layer norm forward and backward against the CPU form in 64 bits.

Tolerances: a sum of n values in fp32 is off by at most depth * 2^-24 times the
sum of their magnitudes, depth the longest chain of additions: 64 covers a
thread's columns, the lanes and the waves for rows kept in registers, longer
rows add one per 512 columns; column sums add one per row.  Each further fp32
operation adds one 2^-24, the result's type half a step."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES, U32, matrix, rounding, untouched, values, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def vectors(seed, cols):
    rng = np.random.default_rng([5, seed])
    f = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    return f(1 + 0.3 * rng.standard_normal(cols)), f(0.3 * rng.standard_normal(cols))


def dev(v):
    return None if v is None else torch.as_tensor(v, dtype=torch.float32).cuda()


def depth(cols):
    return (64 + cols / 512) * U32


def check_forward(gq, x, dtype, w, b, group=0, pad=0, lead=0, x_form=False, y_form=False,
                  keep_y=True, in_place=False, eps=EPS):
    rows, cols = x.shape
    a = gq.act(rows, cols, TYPES[dtype], group)
    xt, xbuf, xmask = matrix(x, TYPES[dtype], pad, lead)
    if in_place:
        y, buf, mask = xt, xbuf, xmask
    else:
        y, buf, mask = matrix(np.zeros_like(x), TYPES[dtype], pad, lead)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    xf = gq.alloc_act(a) if x_form else None
    yf = gq.alloc_act(a) if y_form else None
    gq.gq_layer_norm(a, xt, dev(w), dev(b), eps, y if keep_y else None, mean=mean,
                     rstd=rstd, x_form=xf, y_form=yf)
    wy, wm, wr = A.layer_norm(x, w, b, eps)
    k = depth(cols)
    am = np.abs(x).mean(axis=1)
    within(mean, wm, k * am)
    # the variance: centred squares, each off by the mean's error too
    d = np.abs(x - wm[:, None])
    var = (d * d).mean(axis=1)
    dvar = k * var + 2 * k * am * d.mean(axis=1) + (k * am) ** 2
    within(rstd, wr, wr * (0.5 * dvar / (var + eps) + 4 * U32) * 1.01)
    if keep_y:
        s = np.ones(cols) if w is None else np.abs(w)
        t = np.zeros(cols) if b is None else np.abs(b)
        rel = (0.5 * dvar / (var + eps) + 8 * U32)[:, None] * 1.01
        tol = s * wr[:, None] * ((k * am)[:, None] * (1 + rel) + d * rel) + 2 * U32 * (t + np.abs(wy))
        within(y, wy, tol + rounding(np.abs(wy) + tol, dtype))
        assert untouched(buf, mask)
    if x_form:
        wc, ws = A.pack(x, group, dtype)
        assert np.array_equal(xf[0].cpu().numpy(), wc)
        assert np.array_equal(xf[1].cpu().numpy(), ws, equal_nan=True)
    if y_form and keep_y:
        wc, ws = A.pack(y.double().cpu().numpy(), group, dtype)
        assert np.array_equal(yf[0].cpu().numpy(), wc)
        assert np.array_equal(yf[1].cpu().numpy(), ws, equal_nan=True)
    return y, yf


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pad,lead", [
    (1, 1, 0, 0), (3, 7, 1, 1), (2, 64, 0, 0), (5, 100, 4, 3), (9, 512, 0, 0),
    (4, 1001, 0, 1), (3, 1024, 8, 0), (7, 2047, 1, 0), (5, 4096, 0, 0),
    (2, 5003, 0, 7), (2, 8192, 0, 0), (3, 9001, 1, 1), (2, 16384, 0, 0),
    (2, 20001, 1, 3)])
def test_forward(gq, dtype, rows, cols, pad, lead):
    w, b = vectors(cols, cols)
    check_forward(gq, values(cols, rows, cols, dtype), dtype, w, b, 0, pad, lead)


@pytest.mark.parametrize("rows", [1, 4, 1023, 2049, 8200])
def test_forward_many_rows(gq, rows):
    w, b = vectors(rows, 130)
    check_forward(gq, values(rows, rows, 130, "bf16"), "bf16", w, b)
    check_forward(gq, values(rows, rows, 2052, "f16"), "f16", w=None, b=None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [0, 32, 512, 1024])
@pytest.mark.parametrize("rows,cols", [(3, 40), (9, 777), (3, 1536), (2, 4096), (2, 8200),
                                       (2, 16390)])
def test_forward_with_forms(gq, dtype, group, rows, cols):
    w, b = vectors(cols, cols)
    x = values(cols, rows, cols, dtype)
    check_forward(gq, x, dtype, w, b, group, 1, 1, x_form=True, y_form=True)
    if cols <= 16384 and group <= 512:
        y, yf = check_forward(gq, x, dtype, w, b, group, y_form=True)
        _, only = check_forward(gq, x, dtype, w, b, group, y_form=True, keep_y=False)
        assert torch.equal(yf[0], only[0]) and torch.equal(yf[1], only[1])


@pytest.mark.parametrize("cols", [100, 3000, 9000, 20000])
def test_forward_in_place(gq, cols):
    w, b = vectors(cols, cols)
    check_forward(gq, values(cols, 600, cols, "bf16"), "bf16", w, b, in_place=True,
                  x_form=True)


def test_forward_hard_rows(gq):
    """Constant rows, rows far from zero, large and small magnitudes; weight
    or bias missing."""
    x = values(1, 8, 1000, "f32", spread=False)
    x[0] = 0.0
    x[1] = 3.0
    x[2] += 1e4
    x[3] *= 1e15
    x[4] *= 1e-12
    x[5] = 1e-3 * x[5] - 77.0
    x = x.astype(np.float32).astype(np.float64)
    w, b = vectors(1, 1000)
    for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
        check_forward(gq, x, "f32", ww, bb)
    check_forward(gq, x[5:], "f32", w, b, eps=0.0)


def test_rows_that_are_not_finite_stay_alone(gq):
    x = values(2, 6, 700, "bf16")
    x[1, 5], x[4, 699] = np.nan, np.inf
    a = gq.act(6, 700, torch.bfloat16)
    y = torch.zeros(6, 700, dtype=torch.bfloat16, device="cuda")
    yf = gq.alloc_act(a)
    gq.gq_layer_norm(a, torch.as_tensor(x).to(torch.bfloat16).cuda(), None, None, EPS, y,
                     y_form=yf)
    bad = torch.tensor([False, True, False, False, True, False])
    assert (torch.isnan(y).all(dim=1).cpu() == bad).all()
    assert (torch.isnan(yf[1][:, 0]).cpu() == bad).all()
    assert torch.isfinite(y[~bad.cuda()]).all()


def check_backward(gq, rows, cols, dtype, group=None, pad=0, lead=0, beta=0.0,
                   weight=True, grads=True, in_place=False, seed=0):
    x, dy = values(seed + 1, rows, cols, dtype), values(seed + 2, rows, cols, dtype, False)
    w = vectors(cols, cols)[0] if weight else None
    a = gq.act(rows, cols, TYPES[dtype], group or 0)
    form = group is not None
    if form:
        codes, steps = A.pack(x, group, dtype)
        x = A.unpack(codes, steps, cols, group)
        xin = (torch.as_tensor(codes).cuda(), torch.as_tensor(steps).cuda())
    else:
        xin = matrix(x, TYPES[dtype], pad, lead)[0]
    _, mean, rstd = A.layer_norm(x, w, None, EPS)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    dyt, dbuf, dmask = matrix(dy, TYPES[dtype], pad, lead)
    dx, buf, mask = (dyt, dbuf, dmask) if in_place else matrix(np.zeros_like(x), TYPES[dtype],
                                                               pad, lead)
    old = vectors(cols + 1, cols)
    flat = torch.full((2 * cols + 9,), 77.0, device="cuda")  # odd places of a flat gradient
    dw, db = flat[3:3 + cols], flat[5 + cols:5 + 2 * cols]
    dw.copy_(dev(old[0]))
    db.copy_(dev(old[1]))
    ws = gq.alloc_workspace(gq.gq_layer_norm_workspace(a)) if grads else None
    gq.gq_layer_norm_backward(a, dyt, xin, dev(mean), dev(rstd), dev(w), dx,
                              dw if grads else None, db if grads else None, beta=beta,
                              workspace=ws)
    m64, r64 = mean.astype(np.float64), rstd.astype(np.float64)
    wx, ww, wb = A.layer_norm_backward(dy, x, m64, r64, w)
    k = depth(cols)
    xh = np.abs((x - m64[:, None]) * r64[:, None])
    ad = np.abs(dy) * (1.0 if w is None else np.abs(w))
    tol = (k + 8 * U32) * r64[:, None] * (ad + ad.mean(axis=1)[:, None] +
                                          xh * (ad * xh).mean(axis=1)[:, None])
    within(dx, wx, tol + rounding(np.abs(wx) + tol, dtype))
    assert untouched(buf, mask)
    if grads:
        kr = (rows + 64 + 4) * U32
        within(dw, ww + beta * old[0],
               kr * (np.abs(dy) * xh).sum(axis=0) + 2 * U32 * np.abs(beta * old[0]) + 1e-30)
        within(db, wb + beta * old[1],
               kr * np.abs(dy).sum(axis=0) + 2 * U32 * np.abs(beta * old[1]) + 1e-30)
        edge = torch.cat([flat[:3], flat[3 + cols:5 + cols], flat[5 + 2 * cols:]])
        assert (edge == 77.0).all()
    return dw, db, dx


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [None, 0, 32, 1024])
@pytest.mark.parametrize("rows,cols,pad,lead", [
    (1, 1, 0, 0), (3, 7, 1, 1), (70, 64, 0, 0), (33, 512, 0, 0), (40, 1001, 1, 3),
    (19, 2048, 0, 0), (9, 4099, 2, 1), (6, 8192, 0, 0), (5, 9001, 1, 1), (3, 16384, 0, 0),
    (4, 20001, 0, 1)])
def test_backward(gq, dtype, group, rows, cols, pad, lead):
    check_backward(gq, rows, cols, dtype, group, pad, lead)


@pytest.mark.parametrize("rows", [1, 5, 64, 257, 2100, 4500])
@pytest.mark.parametrize("group", [None, 64])
def test_backward_many_rows(gq, rows, group):
    check_backward(gq, rows, 200, "bf16", group, beta=1.0)
    check_backward(gq, rows, 1300, "f16", group, beta=-0.5)


@pytest.mark.parametrize("cols", [300, 5000, 17000])
def test_backward_options(gq, cols):
    check_backward(gq, 600, cols, "bf16", weight=False)
    check_backward(gq, 600, cols, "bf16", grads=False)
    check_backward(gq, 600, cols, "bf16", in_place=True, pad=2)
    check_backward(gq, 600, cols, "f32", 128, in_place=True)


def test_backward_of_no_rows_scales_the_gradients(gq):
    a = gq.act(0, 50, torch.bfloat16)
    e = torch.empty(0, 50, dtype=torch.bfloat16, device="cuda")
    n = torch.empty(0, device="cuda")
    dw, db = torch.full((50,), 3.0, device="cuda"), torch.full((50,), 5.0, device="cuda")
    ws = gq.alloc_workspace(gq.gq_layer_norm_workspace(a))
    gq.gq_layer_norm(a, e, None, None, EPS, e)
    gq.gq_layer_norm_backward(a, e, e, n, n, None, torch.empty_like(e), dw, db, beta=0.5,
                              workspace=ws)
    assert (dw == 1.5).all() and (db == 2.5).all()
    gq.gq_layer_norm_backward(a, e, e, n, n, None, torch.empty_like(e), dw, None,
                              workspace=ws)
    assert (dw == 0).all() and (db == 2.5).all()


def test_backward_repeats_bit_for_bit(gq):
    first = check_backward(gq, 3000, 500, "bf16", None, seed=3)
    again = check_backward(gq, 3000, 500, "bf16", None, seed=3)
    assert all(torch.equal(p, q) for p, q in zip(first, again))

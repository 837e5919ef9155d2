"""GPU calls that read an 8-bit form, on every code an int8 holds: -128 comes
in forms from elsewhere and has to decode like its neighbours."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES, U32, rounding, values, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def form(seed, rows, cols, group, lo=-6, hi=7):
    """Every code, -128 as often as all others together, and its neighbours."""
    rng = np.random.default_rng([14, seed])
    codes = np.zeros((rows, A.pitch(cols)), np.int8)
    q = rng.integers(-128, 128, (rows, cols))
    codes[:, :cols] = np.where(rng.random((rows, cols)) < 0.5, -128, q)
    steps = 2.0 ** rng.integers(lo, hi, (rows, A.groups(cols, group))).astype(np.float32)
    return codes, steps


def test_every_byte_decodes(gq):
    """All pairs of neighbouring codes, in each of a word's places."""
    q = np.stack(np.meshgrid(np.arange(-128, 128), np.arange(-128, 128)), -1)
    for lead in range(4):
        codes = np.zeros((256, 528), np.int8)
        codes[:, lead:lead + 512] = q.reshape(256, 512)
        steps = np.full((256, 1), 0.25, np.float32)
        a = gq.act(256, 520, torch.float32)
        out = torch.empty(256, 520, device="cuda")
        gq.gq_act_unpack(a, torch.as_tensor(codes).cuda(), torch.as_tensor(steps).cuda(), out)
        assert np.array_equal(out.cpu().numpy(), codes[:, :520] * np.float32(0.25))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [0, 32, 1024])
@pytest.mark.parametrize("rows,cols", [(1, 5), (3, 100), (9, 1001), (4, 4096)])
def test_unpack(gq, dtype, group, rows, cols):
    codes, steps = form(cols, rows, cols, group)
    a = gq.act(rows, cols, TYPES[dtype], group)
    out = torch.empty(rows, cols, dtype=TYPES[dtype], device="cuda")
    gq.gq_act_unpack(a, torch.as_tensor(codes).cuda(), torch.as_tensor(steps).cuda(), out)
    assert np.array_equal(out.double().cpu().numpy(), A.unpack(codes, steps, cols, group))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_unpack_at_the_largest_steps(gq, dtype):
    """127 steps stay finite there; so does -128 one step below."""
    top = A.STEP_CAP[dtype]
    codes = np.zeros((2, 16), np.int8)
    codes[0, :4] = 127, -127, 0, 1
    codes[1, :4] = 127, -128, 0, -128
    steps = np.array([[2.0 ** top], [2.0 ** (top - 1)]], np.float32)
    out = torch.empty(2, 4, dtype=TYPES[dtype], device="cuda")
    gq.gq_act_unpack(gq.act(2, 4, TYPES[dtype]), torch.as_tensor(codes).cuda(),
                     torch.as_tensor(steps).cuda(), out)
    assert np.array_equal(out.double().cpu().numpy(), A.unpack(codes, steps, 4))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,group", [(1, 8, 16, 0), (70, 24, 100, 32),
                                                 (513, 264, 260, 64)])
def test_weight_gradient(gq, dtype, rows, out, cols, group):
    codes, steps = form(rows, rows, cols, group, 0, 3)
    dy = np.random.default_rng([15, rows]).integers(-4, 5, (rows, out)).astype(np.float64)
    assert rows * 4 * 128 * 4 < 2 ** 24      # whole numbers: exact sums
    a = gq.act(rows, cols, TYPES[dtype], group)
    dw = torch.empty(out, cols, device="cuda")
    gq.gq_act_wgrad(a, torch.as_tensor(dy).to(TYPES[dtype]).cuda(), torch.as_tensor(codes).cuda(),
                    torch.as_tensor(steps).cuda(), dw,
                    workspace=gq.alloc_workspace(gq.gq_act_wgrad_workspace(a, out)))
    want = A.wgrad(dy, A.unpack(codes, steps, cols, group))[0]
    assert np.array_equal(dw.double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 7), (5, 1001), (20, 2048), (2, 20001)])
def test_layer_norm_backward(gq, dtype, rows, cols):
    codes, steps = form(cols, rows, cols, 0, -3, 3)
    x, dy = A.unpack(codes, steps, cols), values(cols, rows, cols, dtype, False)
    _, mean, rstd = A.layer_norm(x, None, None, 1e-5)
    mean, rstd = mean.astype(np.float32), rstd.astype(np.float32)
    a = gq.act(rows, cols, TYPES[dtype])
    dx = torch.empty(rows, cols, dtype=TYPES[dtype], device="cuda")
    gq.gq_layer_norm_backward(
        a, torch.as_tensor(dy).to(TYPES[dtype]).cuda(),
        (torch.as_tensor(codes).cuda(), torch.as_tensor(steps).cuda()),
        torch.as_tensor(mean).cuda(), torch.as_tensor(rstd).cuda(), None, dx)
    m, r = mean.astype(np.float64), rstd.astype(np.float64)
    want, _, _ = A.layer_norm_backward(dy, x, m, r, None)
    # a thread's columns, lanes and waves: 64 additions, one more per 512
    # columns of a long row; eight further operations
    xh, ad = np.abs((x - m[:, None]) * r[:, None]), np.abs(dy)
    tol = (72 + cols / 512) * U32 * r[:, None] * (
        ad + ad.mean(axis=1)[:, None] + xh * (ad * xh).mean(axis=1)[:, None])
    within(dx, want, tol + rounding(np.abs(want) + tol, dtype))

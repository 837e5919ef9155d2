"""GPU pack and unpack of the 8-bit activation form against the CPU form:
codes, padding and steps bit for bit, x^ exactly as the type rounds it."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from tests.act_util import TYPES, matrix, untouched, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def check(gq, x, dtype, group, pad=0, lead=0):
    rows, cols = x.shape
    a = gq.act(rows, cols, TYPES[dtype], group)
    xt, _, _ = matrix(x, TYPES[dtype], pad, lead)
    codes, steps = gq.alloc_act(a)
    guard = torch.full((codes.numel() + 64,), 99, dtype=torch.int8, device="cuda")
    codes = guard[:codes.numel()].view(codes.shape)
    codes.fill_(55)
    steps.fill_(5.0)
    gq.gq_act_pack(a, xt, codes, steps)
    want_c, want_s = A.pack(x, group, dtype)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(steps.cpu().numpy(), want_s, equal_nan=True)
    assert (guard[codes.numel():] == 99).all()
    out, buf, mask = matrix(np.zeros_like(x), TYPES[dtype], pad, lead)
    gq.gq_act_unpack(a, codes, steps, out)
    want = torch.as_tensor(A.unpack(want_c, want_s, cols, group)).to(TYPES[dtype])
    assert torch.equal(out.cpu().nan_to_num(nan=1e4), want.nan_to_num(nan=1e4))
    assert untouched(buf, mask)
    return codes, steps


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256, 512, 1024, 32768])
@pytest.mark.parametrize("rows,cols,pad,lead", [
    (1, 1, 0, 0), (3, 7, 2, 1), (5, 32, 0, 0), (2, 100, 0, 3), (17, 129, 6, 1),
    (6, 511, 0, 0), (4, 1001, 1, 5), (3, 2048, 8, 0), (2, 4100, 0, 0)])
def test_sizes_and_groups(gq, dtype, group, rows, cols, pad, lead):
    check(gq, values(rows * cols, rows, cols, dtype), dtype, group, pad, lead)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 512, 2048, 16384])
@pytest.mark.parametrize("cols", [5000, 8200, 16400, 40001])
def test_long_rows(gq, dtype, group, cols):
    check(gq, values(cols, 3, cols, dtype), dtype, group, 1, 1)


def test_many_rows(gq):
    check(gq, values(1, 3001, 40, "bf16"), "bf16", 32)
    check(gq, values(2, 2050, 130, "f16"), "f16", 0, 2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [0, 32, 1024])
def test_edge_values(gq, dtype, group):
    big = float(torch.finfo(TYPES[dtype]).max)
    tiny = float(torch.finfo(TYPES[dtype]).tiny)
    x = values(3, 12, 1500, dtype)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 40] = np.nan                      # one group; its neighbours stay
    x[3, 1400] = np.inf
    x[4, 0], x[4, 1] = -np.inf, np.nan
    x[5] = big
    x[6, ::3] = -big
    x[7] = tiny
    x[8] *= tiny
    x[9] = 127.0                           # 127 step = max exactly
    x[10] = 127.5                          # just past it
    x[11] = np.tile([0.5, 1.5, 2.5, -0.5, 127.0], 300)   # ties
    check(gq, torch.as_tensor(x).to(TYPES[dtype]).double().numpy(), dtype, group)


@pytest.mark.parametrize("exp", range(-149, 128, 23))
def test_every_scale(gq, exp):
    m = np.ldexp(1.0 + np.arange(128) / 128, exp)        # 128 rows, one peak each
    x = m[:, None] * np.linspace(-1, 1, 48)[None, :]
    x = x.astype(np.float32).astype(np.float64)
    check(gq, x, "f32", 0)


def test_no_rows(gq):
    a = gq.act(0, 10, torch.bfloat16)
    x = torch.empty(0, 10, dtype=torch.bfloat16, device="cuda")
    codes, steps = gq.alloc_act(a)
    gq.gq_act_pack(a, x, codes, steps)
    gq.gq_act_unpack(a, codes, steps, x)


def test_a_stream_of_its_own(gq):
    x = values(9, 64, 512, "bf16")
    want_c, want_s = A.pack(x, 128)
    a = gq.act(64, 512, torch.bfloat16, 128)
    side = torch.cuda.Stream()
    xt = torch.as_tensor(x).to(torch.bfloat16).cuda()
    codes, steps = gq.alloc_act(a)
    side.wait_stream(torch.cuda.current_stream())
    gq.gq_act_pack(a, xt, codes, steps, stream=side)
    side.synchronize()
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(steps.cpu().numpy(), want_s)


def test_binding_refuses_on_the_device(gq):
    a = gq.act(4, 64, torch.bfloat16)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    codes, steps = gq.alloc_act(a)
    for bad in (x.float(), ):
        with pytest.raises(TypeError):
            gq.gq_act_pack(a, bad, codes, steps)
    for bad in (x[:3], x.view(8, 32), torch.zeros(64, 4, dtype=x.dtype, device="cuda").t(),
                x[:1].expand(4, 64)):
        with pytest.raises(ValueError):
            gq.gq_act_pack(a, bad, codes, steps)
    with pytest.raises(ValueError):
        gq.gq_act_pack(a, x, codes[:3], steps)
    with pytest.raises(ValueError):
        gq.gq_act_pack(a, x, codes, steps[:3])
    with pytest.raises(TypeError):
        gq.gq_act_pack(a, x, codes.view(torch.uint8), steps)

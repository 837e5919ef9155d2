"""Forms that did not come from packing: every code with every step from 2^-126 to
2^127.  A weight gradient of one token with dy = 1 is x^ itself, as unpacking
gives it in the activations' type; in fp32 to a multiple of 2^-133 (bf16's last
place), and NaN where x^ is past the largest number.  The fp32 product takes x^ in
the same way, with infinities; 16-bit products take a step's exponent alone."""
import numpy as np
import pytest
import torch

from oracle import activations as A
from oracle import step as S
from tests.act_util import TYPES
from tests.test_gpu_block_linear import d8, dev

pytestmark = pytest.mark.gpu
EXPONENTS = np.arange(-126, 128)
N = len(EXPONENTS)


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def same(got, want):
    got, want = got.double().cpu(), want.double()
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


def in_type(x, dtype):
    """fp32 values that float64 values are, rounded to the type by torch."""
    with np.errstate(over="ignore"):
        return torch.as_tensor(np.asarray(x, np.float64).astype(np.float32)).to(TYPES[dtype])


def every_form():
    """[exponents, 256 codes] with its steps, and x^ in 64 bits."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (N, 1))
    steps = np.exp2(EXPONENTS.astype(np.float64))
    return codes, np.repeat(steps.astype(np.float32)[:, None], 2, 1), S.values(codes) * steps[:, None]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", [1, 8, 130])
def test_gradients_take_what_unpack_gives(gq, dtype, out):
    codes, steps, x = every_form()
    a = gq.act(N, 256, TYPES[dtype], 128)
    c, s = d8(codes), dev(steps)
    back = torch.empty(N, 256, dtype=TYPES[dtype], device="cuda")
    gq.gq_block_unpack(a, c, s, back)
    assert same(back, in_type(x, dtype))
    # a token to an expert: no x^ meets another
    dw, db = torch.empty(N, out, 256, device="cuda"), torch.empty(N, out, device="cuda")
    gq.gq_block_wgrad(a, torch.ones(N, out, dtype=TYPES[dtype], device="cuda"), c, s, dw, db,
                      offsets=torch.arange(N + 1, device="cuda"),
                      workspace=gq.alloc_workspace(gq.gq_block_wgrad_workspace(a, out, N)))
    if dtype == "f32":
        want = in_type(x, "bf16").double()
        want[want.isinf()] = float("nan")       # infinity times the zeros that dy has below
    else:
        want = back.double().cpu()
    assert same(dw, want[:, None, :].expand(N, out, 256))
    assert bool((db == 1).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_of_the_integer_form_too(gq, dtype):
    codes = np.arange(-128, 128).astype(np.int8)[None]
    for k in range(-40, 41):
        step = np.full((1, 1), 2.0 ** k, np.float32)
        a = gq.act(1, 256, TYPES[dtype], 0)
        dw = torch.empty(256, device="cuda")
        gq.gq_act_wgrad(a, torch.ones(1, 1, dtype=TYPES[dtype], device="cuda"), dev(codes),
                        dev(step), dw)
        back = torch.empty(1, 256, dtype=TYPES[dtype], device="cuda")
        gq.gq_act_unpack(a, dev(codes), dev(step), back)
        assert same(back[0], in_type(A.unpack(codes, step, 256, 0)[0], dtype))
        assert same(dw, back[0].cpu()), k


@pytest.mark.parametrize("each", [16, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_products(gq, dtype, each):
    """One code of a row with one of 1 in the weight, at the ends of the range; by
    the kernel for few tokens and by tiles."""
    x = np.zeros((256, 128), np.uint8)
    x[:, 3] = np.arange(256)
    w = np.zeros((1, 1, 128), np.uint8)
    w[0, 0, 3] = 0x38
    a = gq.act(each, 128, TYPES[dtype], 128)
    y = torch.empty(256, 1, dtype=TYPES[dtype], device="cuda")
    for e in (-126, -125, -124, 0, 119, 120, 127):
        for k in (0, -20, 20, 100):
            for lo in range(0, 256, each):
                gq.gq_block_linear(a, d8(x[lo:lo + each]), torch.full((each, 1), 2.0 ** e, device="cuda"),
                                   d8(w), torch.full((1, 1, 1), 2.0 ** k, device="cuda"), None,
                                   y[lo:lo + each])
            v = S.values(x[:, 3]) * 2.0 ** e
            if dtype == "f32":
                v = in_type(v, "bf16").double().numpy()
            assert same(y[:, 0], in_type(v * 2.0 ** k, dtype)), (e, k)

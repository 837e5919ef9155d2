"""GPU integer product of up to 64 tokens, on both sides of the sizes at which
the kernel for few tokens gives way to the tiled one."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 32, 33, 63, 64])
@pytest.mark.parametrize("out", [4095, 4096, 4097, 8192, 8193, 12001])
def test_both_kernels(gq, dtype, rows, out):
    cols = 130
    rng = np.random.default_rng([18, rows, out])
    c, w = (np.zeros((n, A.pitch(cols)), np.int8) for n in (rows, out))
    c[:, :cols] = rng.integers(-128, 128, (rows, cols))
    w[:, :cols] = rng.integers(-128, 128, (out, cols))
    s, v = (np.exp(rng.standard_normal(k)).astype(np.float32) / 100 for k in ((rows, 1), out))
    b = rng.standard_normal(out).astype(np.float32)
    a = gq.act(rows, cols, TYPES[dtype])
    y, buf, mask = matrix(np.zeros((rows, out)), TYPES[dtype], 1, 1)
    d = lambda t: torch.as_tensor(t).cuda()  # noqa: E731
    gq.gq_act_linear(a, d(c), d(s), d(w), d(v), d(b), y)
    # the integer sum is exact; four fp32 roundings and the type's
    want, prod = A.linear(c, s, w, v, b, cols), A.linear(c, s, w, v, None, cols)
    tol = 4 * U32 * (np.abs(prod) + np.abs(want))
    within(y, want, tol + rounding(np.abs(want) + tol, dtype))
    assert untouched(buf, mask)


def test_the_kernels_agree_bit_for_bit(gq):
    out, cols = 4608, 2064
    g = torch.Generator(device="cuda").manual_seed(5)
    w = gq.alloc_act(gq.act(out, cols, torch.float32))
    gq.gq_act_pack(gq.act(out, cols, torch.float32),
                   torch.randn(out, cols, generator=g, device="cuda"), *w)
    a = gq.act(64, cols, torch.float32)
    x = gq.alloc_act(a)
    gq.gq_act_pack(a, torch.randn(64, cols, generator=g, device="cuda"), *x)
    full = torch.empty(64, out, device="cuda")
    gq.gq_act_linear(a, *x, w[0], w[1].view(-1), None, full)
    for lo, n in ((0, 1), (3, 8), (11, 9), (20, 17), (30, 34)):
        part = torch.empty(n, out, device="cuda")
        gq.gq_act_linear(gq.act(n, cols, torch.float32), x[0][lo:lo + n], x[1][lo:lo + n], w[0],
                         w[1].view(-1), None, part)
        assert torch.equal(part, full[lo:lo + n])

"""GPU product from 8-bit floating point forms through every kernel and way of
splitting the sum, in all types (tolerances: test_gpu_block_linear.py).  Which
shapes reach which is checked on the host (test_fp8_plan.py)."""
import pytest
import torch

from tests.test_gpu_block_linear import check

# (tile, teams of waves, whole or in parts, k-tiles of a part): rows, out, cols, experts
SHAPES = {
    (0, 1, "whole", "odd"): [(60, 300, 600, 3), (33, 400, 2100, 5)],
    (0, 1, "whole", "even"): [(64, 700, 1000, 2), (12, 1400, 256, 1)],
    (64, 2, "parts", "odd"): [(1111, 100, 16000, 3), (300, 90, 7600, 3), (100, 500, 12900, 2)],
    (64, 2, "parts", "even"): [(1111, 100, 15001, 3), (80, 64, 5100, 20), (200, 130, 16100, 1)],
    (64, 2, "whole", "odd"): [(90, 100, 4200, 3), (90, 300, 2100, 2), (64, 3000, 300, 3)],
    (64, 2, "whole", "even"): [(130, 70, 3800, 2)],
    (64, 1, "whole", "odd"): [(1500, 700, 600, 12)],
    (64, 1, "whole", "even"): [(33, 6000, 1500, 20)],
    (64, 1, "parts", "even"): [(400, 1001, 15100, 3)],
    (128, 1, "whole", "even"): [(5000, 512, 500, 9)],
    (128, 1, "parts", "even"): [(1100, 1001, 15001, 1)],
    (256, 1, "whole", "odd"): [(4100, 2048, 300, 4)],
}


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,experts", sum(SHAPES.values(), []))
def test_products(gq, dtype, rows, out, cols, experts):
    check(gq, rows, out, cols, dtype, experts, whole=True, pad=1, lead=1, before=3, behind=2,
          seed=rows)
    check(gq, rows, out, cols, dtype, experts, bias=False, seed=cols)

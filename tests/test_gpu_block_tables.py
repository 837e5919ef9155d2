"""Device tables that hold anything: outputs are unspecified then, but nothing is
written outside of them.  Every buffer that a call writes lies between two bands
that have to stay as they were; every kernel that reads a table is reached
(test_fp8_plan.py pins which shape reaches which kernel of the product)."""
import numpy as np
import pytest
import torch

from oracle import step as S
from tests.act_util import TYPES
from tests.test_gpu_block_linear import d8, dev, forms

BAND = 4096


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


class Banded:
    """A 16-byte aligned buffer of `n` values with bands on both sides."""

    def __init__(self, n, dtype, fill=None):
        size = torch.empty(0, dtype=dtype).element_size()
        self.bytes = n * size
        self.raw = torch.full((BAND + -(-self.bytes // 16) * 16 + BAND,), 0x5a, dtype=torch.uint8,
                              device="cuda")
        self.t = self.raw[BAND:BAND + self.bytes].view(dtype)
        if fill is not None:
            self.t.view(torch.uint8).fill_(fill)

    def kept(self):
        return bool((self.raw[:BAND] == 0x5a).all()) and bool(
            (self.raw[BAND + self.bytes:] == 0x5a).all())


def tables(entries, n):
    """Tables of `entries` numbers over n rows or values that no program should make:
    below, past the end, descending, all of it, the largest numbers."""
    rng = np.random.default_rng([21, entries])
    wild = rng.integers(-(1 << 62), 1 << 62, entries)
    near = rng.integers(-n, 2 * n + 1, entries)
    yield [-5, n // 4, n // 9, 4 * n, n + 1] + [n] * (entries - 5) if entries > 4 else near.tolist()
    yield np.linspace(n, 0, entries).astype(np.int64).tolist()
    yield np.where(np.arange(entries) % 2, n, 0).tolist()
    yield [1 << 62] * entries
    yield [-(1 << 62)] + [1 << 62] * (entries - 1)
    yield wild.tolist()
    yield near.tolist()
    yield rng.integers(0, n + 1, entries).tolist()


# (tile, teams, whole or in parts): rows, out, cols, experts
PRODUCTS = {
    (0, 1, "whole"): [(3, 70, 400, 4), (40, 130, 140, 6)],
    (64, 2, "whole"): [(90, 130, 140, 4), (100, 90, 200, 1024)],
    (64, 2, "parts"): [(300, 90, 7600, 4)],
    (64, 1, "whole"): [(1500, 700, 300, 12), (100, 300, 200, 1024)],
    (64, 1, "parts"): [(400, 1001, 15100, 3)],
    (128, 1, "whole"): [(5000, 512, 300, 9)],
    (256, 1, "whole"): [(4100, 2048, 200, 4)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,out,cols,experts", sum(PRODUCTS.values(), []))
def test_products(gq, dtype, rows, out, cols, experts):
    x, w, b = forms(3, rows, out, cols, experts, True)
    args = [d8(x[0]), dev(x[1]), d8(w[0]), dev(w[1]), dev(b)]
    a = gq.act(rows, cols, TYPES[dtype], 128)
    y = Banded(rows * out, TYPES[dtype])
    need = gq.gq_block_linear_workspace(a, out, experts)
    ws = Banded(need, torch.uint8, 0)
    for off in tables(experts + 1, rows):
        gq.gq_block_linear(a, *args, y.t.view(rows, out), offsets=dev(np.array(off, np.int64)),
                           workspace=ws.t)
        assert y.kept() and ws.kept(), off


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,experts,parts", [
    (90, 40, 140, 4, False), (60, 3, 5, 1024, False), (2100, 136, 130, 3, True),
    (9000, 64, 300, 6, True), (9000, 131, 300, 17, True)])
def test_weight_gradients(gq, dtype, rows, out, cols, experts, parts):
    codes = np.full((rows, S.pitch(cols)), 0x38, np.uint8)
    codes[:, cols:] = 0
    a = gq.act(rows, cols, TYPES[dtype], 128)
    form = d8(codes), torch.ones(rows, a.groups, device="cuda")
    dy = torch.ones(rows, out, dtype=TYPES[dtype], device="cuda")
    need = gq.gq_block_wgrad_workspace(a, out, experts)
    assert (need > 0) == parts
    dw, db = Banded(experts * out * cols, torch.float32, 0), Banded(experts * out, torch.float32, 0)
    ws = Banded(need, torch.uint8, 0)
    for off in tables(experts + 1, rows):
        gq.gq_block_wgrad(a, dy, *form, dw.t, db.t, offsets=dev(np.array(off, np.int64)), beta=0.5,
                          workspace=ws.t)
        assert dw.kept() and db.kept() and ws.kept(), off


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("n", [5, 3000, 70001])
@pytest.mark.parametrize("layers", [1, 4, 300])
def test_updates(gq, bits, n, layers):
    d = gq.adamw(1e-3, bits=bits)
    rng = np.random.default_rng(22)
    p = Banded(n, torch.float32)
    p.t.copy_(dev(rng.standard_normal(n).astype(np.float32)))
    g = dev(rng.standard_normal(n).astype(np.float32))
    half = Banded(n, torch.bfloat16)
    kinds = (torch.float32,) * 2 if bits == 32 else (gq.E4M3, gq.E5M2)
    codes = [Banded(n, k, 0) for k in kinds]
    steps = [Banded(-(-n // 256), torch.float32, 0) for _ in kinds]
    m, v = (c.t if bits == 32 else (c.t, s.t) for c, s in zip(codes, steps))
    for t, off in enumerate(tables(layers + 1, n), 1):
        gq.gq_adamw(d, g, p.t, m, v, t, layer_offsets=dev(np.array(off, np.int64)),
                    lr_scale=torch.ones(layers, device="cuda"),
                    decay=torch.zeros(layers, device="cuda"), p16=half.t)
        assert all(b.kept() for b in (p, half, *codes, *steps)), off
        assert bool(torch.isfinite(p.t).all())

"""Helpers of the GPU tests of the 8-bit activation operators."""
import numpy as np
import torch

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8 / 2, "f16": 2.0 ** -11}  # half a step
HALF["bf16"] = torch.finfo(torch.bfloat16).eps / 2
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}     # smallest steps
U32 = 2.0 ** -24


def matrix(values, dtype, pad=0, lead=0):
    """A device matrix of those values in a wider buffer: `pad` more columns
    per row, `lead` elements before the first (any alignment).  Returns
    (matrix, buffer, mask of the buffer's elements that are the matrix's)."""
    rows, cols = values.shape
    buf = torch.full((lead + rows * (cols + pad) + 8,), 77.0, dtype=dtype, device="cuda")
    mask = torch.zeros(buf.shape, dtype=torch.bool, device="cuda")
    view = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    mview = mask[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.as_tensor(values))
    mview.fill_(True)
    return view, buf, mask


def untouched(buf, mask):
    return bool((buf[~mask] == 77.0).all())


def values(seed, rows, cols, dtype, spread=True):
    """float64 values that the type holds."""
    rng = np.random.default_rng([4, seed])
    x = rng.standard_normal((rows, cols))
    if spread:
        x *= np.exp(rng.standard_normal(cols))
    return torch.as_tensor(x).to(TYPES[dtype]).double().numpy()


def within(got, want, tol):
    """|got - want| <= tol elementwise; not-finite values have to be equal."""
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    over = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
    assert over.size == 0 or over.max() <= 0, f"off by {over.max()} more than allowed"


def rounding(want, dtype):
    """One rounding of a result to its type (the smallest step below it)."""
    return HALF[dtype] * np.abs(want) + TINY[dtype]

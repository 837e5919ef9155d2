"""GPU product from 8-bit floating point forms, alone and by expert, against the
64-bit product of the same forms.  fp32 results: products are exact and each of
the sum's additions may round or cut to 24 bits, so a result is off by at most
cols + 2 steps of 2^-23 of the terms' magnitudes.  16-bit results: eight products
at a time are cut at 2^-13 of the largest before, eight times 2^-13 of what is at
most the sum of the eight magnitudes, so 2^-10 of the magnitudes in all; and the
type's rounding.  Whole numbers whose products lie within 2^13 of each other and
whose sums stay below 2^24 do not round."""
import numpy as np
import pytest
import torch

from oracle import step as S
from tests.act_util import TYPES, matrix, rounding, untouched, within

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def table(rng, rows, experts, before=0, behind=0):
    """Ragged loads, some of them none."""
    cut = np.sort(rng.integers(before, rows - behind + 1, experts - 1))
    off = np.concatenate([[before], cut, [rows - behind]]).astype(np.int64)
    if experts > 2:
        off[2] = off[1]
    return off


def forms(seed, rows, out, cols, experts, whole):
    """Codes and powers of two: whole small numbers, or all finite codes."""
    rng = np.random.default_rng([9, seed])

    def codes(*shape):
        c = np.zeros(shape[:-1] + (S.pitch(cols),), np.uint8)
        if whole:       # -2 .. 2
            v = rng.choice(np.array([0, 0x38, 0x40, 0xb8, 0xc0], np.uint8), shape)
        else:
            v = rng.integers(0, 0x7f, shape) | (rng.integers(0, 2, shape) << 7)
        c[..., :cols] = v
        return c

    def steps(*shape):
        e = rng.integers(0, 2, shape) if whole else rng.integers(-20, -7, shape)
        return np.exp2(e).astype(np.float32)

    x = codes(rows, cols), steps(rows, S.blocks(cols))
    w = codes(experts, out, cols), steps(experts, S.blocks(out), S.blocks(cols))
    bias = rng.integers(-9, 10, (experts, out)).astype(np.float32)
    return x, w, bias


def d8(c):
    return torch.as_tensor(c).cuda().view(E4M3)


def dev(a):
    return torch.as_tensor(a).cuda()


def run(gq, x, w, bias, off, rows, out, cols, dtype, pad=0, lead=0):
    a = gq.act(rows, cols, TYPES[dtype], 128)
    experts = w[0].shape[0]
    y, buf, mask = matrix(np.zeros((rows, out)), TYPES[dtype], pad, lead)
    buf.fill_(77.0)
    work = gq.alloc_workspace(gq.gq_block_linear_workspace(a, out, experts))
    if work is not None:
        work.fill_(0x55)
    gq.gq_block_linear(a, d8(x[0]), dev(x[1]), d8(w[0]), dev(w[1]),
                     None if bias is None else dev(bias), y,
                     offsets=None if off is None else dev(off), workspace=work)
    assert untouched(buf, mask)
    if off is not None:         # rows of no expert
        assert bool((y[:off[0]] == 77.0).all()) and bool((y[off[-1]:] == 77.0).all())
    return y


def check(gq, rows, out, cols, dtype, experts=1, whole=False, bias=True, pad=0, lead=0,
          before=0, behind=0, seed=0, off=None):
    x, w, b = forms(seed, rows, out, cols, experts, whole)
    if not bias:
        b = None
    if off is None and (experts > 1 or before or behind):
        off = table(np.random.default_rng([10, seed]), rows, experts, before, behind)
    y = run(gq, x, w, b, off, rows, out, cols, dtype, pad, lead)
    o = [0, rows] if off is None else off
    want, mag = S.linear(S.unpack(*x, cols), S.unpack_weight(*w, cols), b, o)
    mine = slice(o[0], o[-1])
    if whole:
        assert np.abs(mag[mine]).max(initial=0) < 2 ** 24
        exact = torch.as_tensor(want[mine]).float().to(TYPES[dtype])
        assert torch.equal(y[mine].cpu(), exact)
    else:
        tol = ((cols + 2) * 2.0 ** -23 + (0.0 if dtype == "f32" else 2.0 ** -10)) * mag[mine]
        within(y[mine], want[mine], tol + rounding(np.abs(want[mine]) + tol, dtype))
    return y


SIZES = [(1, 1, 1, 0, 0), (1, 64, 64, 0, 0), (1, 1001, 777, 0, 1), (2, 130, 16, 1, 3),
         (3, 33, 1030, 0, 0), (16, 512, 2048, 0, 0), (17, 511, 100, 1, 1), (31, 65, 129, 0, 0),
         (33, 257, 513, 3, 2), (64, 128, 128, 0, 0), (65, 200, 260, 0, 0),
         (129, 131, 4100, 1, 1), (200, 520, 1000, 0, 0), (300, 300, 64, 0, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,pad,lead", SIZES)
def test_sizes(gq, dtype, rows, out, cols, pad, lead):
    check(gq, rows, out, cols, dtype, whole=True, pad=pad, lead=lead, seed=rows)
    check(gq, rows, out, cols, dtype, bias=False, seed=cols)


@pytest.mark.parametrize("rows", [1, 5, 16, 32, 48, 64, 80, 128, 256, 257])
@pytest.mark.parametrize("cols", [48, 1024, 6000])
def test_row_counts(gq, rows, cols):
    check(gq, rows, 272, cols, "bf16", seed=rows)
    check(gq, rows, 272, cols, "f32", whole=True, seed=rows)


def test_large_tiles(gq):
    check(gq, 2049, 4100, 300, "bf16")
    check(gq, 4096, 2048, 256, "f32", whole=True)
    check(gq, 2500, 2500, 129, "f16", whole=True)


def test_long_sums_are_split(gq):
    a = gq.act(1111, 16000, torch.bfloat16, 128)
    assert gq.gq_block_linear_workspace(a, 1000) > 0
    check(gq, 1111, 1000, 16000, "bf16", pad=3, lead=1)
    check(gq, 1100, 1001, 15001, "f32", whole=True, before=7, behind=11)
    check(gq, 1111, 500, 16000, "f32", experts=3, whole=True, before=5, behind=2)
    # parts of tiles that two teams take, of odd and even numbers of k-tiles
    for dtype, cols in (("f32", 16000), ("bf16", 15001), ("f16", 8192), ("bf16", 9600)):
        a = gq.act(1111, cols, {"f32": torch.float32, "f16": torch.float16}.get(
            dtype, torch.bfloat16), 128)
        assert gq.gq_block_linear_workspace(a, 100, 3) > 0
        check(gq, 1111, 100, cols, dtype, experts=3, whole=True, before=5, behind=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1, 128, 129, 256, 300, 640, 1000, 1152])
def test_tiles_of_two_teams(gq, dtype, cols):
    """One to nine k-tiles, the second team's last one past the end or not."""
    check(gq, 100, 150, cols, dtype, whole=True, pad=1, lead=1, seed=cols)
    check(gq, 300, 64, cols, dtype, experts=5, before=2, behind=3, seed=cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,out,cols,experts,before,behind", [
    (1, 70, 40, 4, 0, 0), (7, 64, 128, 16, 0, 0), (32, 100, 260, 5, 3, 4), (64, 129, 300, 64, 0, 1),
    (200, 270, 500, 3, 1, 0), (513, 130, 129, 9, 0, 30), (1500, 400, 200, 100, 0, 0),
    (40, 20, 30, 1024, 2, 3), (2300, 600, 256, 2, 17, 5)])
def test_experts(gq, dtype, rows, out, cols, experts, before, behind):
    check(gq, rows, out, cols, dtype, experts, whole=True, before=before, behind=behind,
          seed=rows)
    check(gq, rows, out, cols, dtype, experts, bias=False, pad=1, lead=1, before=before,
          behind=behind, seed=cols)


@pytest.mark.parametrize("rows", [40, 700])
def test_one_expert_has_all_rows_or_none(gq, rows):
    for e in range(3):
        off = np.array([0] * (e + 1) + [rows] * (3 - e), np.int64)
        check(gq, rows, 150, 200, "f32", 3, whole=True, off=off)
    check(gq, rows, 150, 200, "f32", 3, whole=True, off=np.array([9, 9, 9, 9], np.int64))


def test_tables_out_of_range_stay_in_bounds(gq):
    """What the table holds may be wrong: every row of y is then written or not,
    and nothing else is."""
    rows, out, cols = 90, 130, 140
    x, w, b = forms(3, rows, out, cols, 4, True)
    for off in ([-5, 20, 10, 400, 91], [0, 1 << 40, -1 << 40, 50, 90], [90, 60, 30, 10, 0]):
        y = torch.zeros(rows, out, device="cuda")
        a = gq.act(rows, cols, torch.float32, 128)
        gq.gq_block_linear(a, d8(x[0]), dev(x[1]), d8(w[0]), dev(w[1]), dev(b), y,
                         offsets=dev(np.array(off, np.int64)))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,split", [(150, 70), (30, 9)])
def test_steps_that_are_not_finite_stay_alone(gq, dtype, rows, split):
    out, cols = 300, 400
    x, w, b = forms(4, rows, out, cols, 2, True)
    x[1][3, 1] = np.nan
    x[0][3, 128:256] = 0
    w[1][1, 1, 2] = np.nan
    w[0][1, 128:256, 256:384] = 0
    off = np.array([0, split, rows], np.int64)
    y = run(gq, x, w, b, off, rows, out, cols, dtype).double().cpu().numpy()
    want, _ = S.linear(S.unpack(*x, cols), S.unpack_weight(*w, cols), b, off)
    bad = np.isnan(want)
    assert bad[3].all() and bad[split:, 128:256].all()
    assert bad.sum() == out + (rows - split) * 128
    assert np.array_equal(np.isnan(y), bad)
    exact = torch.as_tensor(want).float().to(TYPES[dtype]).double().numpy()
    assert np.array_equal(y[~bad], exact[~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [20, 200])
def test_codes_that_are_nan(gq, dtype, rows):
    """e4m3's NaN is a code like any other: its row and its outputs."""
    out, cols = 140, 200
    x, w, b = forms(5, rows, out, cols, 1, True)
    x[0][7, 150] = 0x7f
    w[0][0, 9, 3] = 0xff
    y = run(gq, x, w, b, None, rows, out, cols, dtype).float().cpu().numpy()
    bad = np.zeros((rows, out), bool)
    bad[7], bad[:, 9] = True, True
    assert np.array_equal(np.isnan(y), bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("each", [50, 300])
def test_extreme_steps(gq, dtype, each):
    """Every exponent that a form can have, with the other side's opposite."""
    for lo in range(-126, 120, each):
        e = np.arange(lo, min(lo + each, 120))
        rows, cols = len(e), 128
        x = np.zeros((rows, 128), np.uint8)
        x[:, 5] = 0x38
        w = np.zeros((1, 1, 128), np.uint8)
        w[0, 0, 5] = 0xb9           # -1.125
        for k in (-3, 0, 6):
            y = run(gq, (x, np.exp2(e)[:, None].astype(np.float32)),
                    (w, np.full((1, 1, 1), 2.0 ** k, np.float32)), None, None, rows, 1, cols,
                    dtype)
            want = (-1.125 * np.exp2(e.astype(np.float64) + k)).astype(np.float32)
            fine = np.abs(want) >= 2.0 ** -126      # below: may be flushed
            assert np.array_equal(y.float().cpu().numpy()[fine, 0], want[fine])


def behind(values, dtype, poison, rows=200):
    """A contiguous device array with `rows` more of poison behind it."""
    buf = torch.full((values.shape[0] + rows,) + values.shape[1:], poison, device="cuda",
                     dtype=dtype)
    buf[:values.shape[0]] = torch.as_tensor(values)
    return buf[:values.shape[0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 17, 33, 50, 65, 130, 300])
@pytest.mark.parametrize("out,cols", [(1, 16), (17, 100), (40, 64), (63, 1000), (131, 272)])
def test_reads_zeros_behind_the_last_rows(gq, dtype, rows, out, cols):
    """Codes, steps, weights and biases of other things behind the matrices."""
    x, w, b = forms(rows, rows, out, cols, 2, True)
    off = np.array([0, rows // 2, rows], np.int64)
    a = gq.act(rows, cols, TYPES[dtype], 128)
    y = torch.full((rows + 9, out), 77.0, device="cuda", dtype=TYPES[dtype])
    nan = float("nan")
    gq.gq_block_linear(
        a, behind(x[0], torch.uint8, 0x7f).view(E4M3), behind(x[1], torch.float32, nan),
        behind(w[0], torch.uint8, 0x7f).view(E4M3), behind(w[1], torch.float32, nan),
        behind(b, torch.float32, nan), y[:rows], offsets=dev(off),
        workspace=gq.alloc_workspace(gq.gq_block_linear_workspace(a, out, 2)))
    want, _ = S.linear(S.unpack(*x, cols), S.unpack_weight(*w, cols), b, off)
    assert torch.equal(y[:rows].cpu(), torch.as_tensor(want).float().to(TYPES[dtype]))
    assert bool((y[rows:] == 77.0).all())


def test_no_rows(gq):
    a = gq.act(0, 64, torch.bfloat16, 128)
    c, s = gq.alloc_block(a)
    wa = gq.act(8, 64, torch.float32, 128)
    w = gq.alloc_block_weight(wa)
    gq.gq_block_linear(a, c, s, *w, None, torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"))

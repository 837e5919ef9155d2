"""The 8-bit floating point form on the GPU: codes and steps equal the CPU form's
bit for bit, activations and weights, both directions of a weight."""
import numpy as np
import pytest
import torch

from oracle import step as S
from tests.act_util import TYPES, matrix, untouched, values

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def same_steps(got, want):
    got, want = got.cpu().numpy(), np.asarray(want, np.float32)
    assert np.array_equal(got.view(np.uint32)[~np.isnan(want)],
                          want.view(np.uint32)[~np.isnan(want)])
    assert np.isnan(got[np.isnan(want)]).all()


def check(gq, x, dtype, pad=0, lead=0):
    rows, cols = x.shape
    a = gq.act(rows, cols, TYPES[dtype], 128)
    view, _, _ = matrix(x, TYPES[dtype], pad, lead)
    codes, steps = gq.alloc_block(a)
    codes.view(torch.uint8).fill_(0x55)
    gq.gq_block_pack(a, view, codes, steps)
    wc, ws = S.pack(x, dtype)
    same_steps(steps, ws)
    assert np.array_equal(raw(codes), wc)
    back, buf, mask = matrix(np.zeros_like(x), TYPES[dtype], pad, lead)
    gq.gq_block_unpack(a, codes, steps, back)
    want = torch.as_tensor(S.unpack(wc, ws, cols)).to(TYPES[dtype])
    assert torch.equal(torch.nan_to_num(back.cpu().double(), 7e77),
                       torch.nan_to_num(want.double(), 7e77))
    assert untouched(buf, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols,pad,lead", [
    (1, 1, 0, 0), (3, 5, 0, 1), (2, 7, 1, 0), (5, 8, 0, 0), (1, 16, 0, 0), (4, 127, 1, 1),
    (3, 128, 0, 0), (2, 129, 0, 3), (7, 255, 2, 0), (33, 1000, 0, 0), (9, 2049, 1, 1),
    (2, 5000, 0, 0)])
def test_sizes(gq, dtype, rows, cols, pad, lead):
    check(gq, values(rows * cols, rows, cols, dtype), dtype, pad, lead)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_edges(gq, dtype):
    """Each row a case: zeros, signs of zero, all places between codes (ties
    among them), step boundaries, the largest and smallest of the type, and
    values that are not finite."""
    top = float(torch.finfo(TYPES[dtype]).max)
    tiny = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[dtype]
    rows = [[0.0] * 130, [-0.0] * 130, [top, 1.0, -top, 0.5] * 33, [tiny, -tiny, 0, 2 * tiny] * 33]
    mids = (S.E4M3[:0x7e] + S.E4M3[1:0x7f]) / 2
    for grid in (mids, S.E4M3[:0x7f], np.nextafter(mids, 1e9).astype(np.float32)):
        for scale in (1.0, 2.0 ** -7):
            rows.append([448.0 * scale] + list(grid[-127:] * scale) + [-448.0 * scale, 0.0])
    for b in (448.0, 449.0, 447.0, 450.0, 1.75, 1.7578125, 224.0):
        rows.append([b] * 64 + [-b / 3] * 64 + [b, 1.0])
    for bad in (np.nan, np.inf, -np.inf):
        rows.append([1.0] * 77 + [bad] + [2.0] * 60)
        rows.append([1.0] * 128 + [bad])
    n = max(len(r) for r in rows)
    x = np.array([list(r) + [0.25] * (n - len(r)) for r in rows])
    x = torch.as_tensor(x).to(TYPES[dtype]).double().numpy()
    check(gq, x, dtype)


def test_every_code_is_decoded(gq):
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    steps = np.array([[2.0 ** -3], [2.0 ** 5]], np.float32)
    a = gq.act(2, 128, torch.float32, 128)
    out = torch.empty(2, 128, device="cuda")
    gq.gq_block_unpack(a, torch.as_tensor(codes).cuda().view(E4M3), torch.as_tensor(steps).cuda(),
                     out)
    want = S.unpack(codes, steps, 128)
    assert np.array_equal(np.isnan(out.cpu().numpy()), np.isnan(want))
    fine = ~np.isnan(want)
    assert np.array_equal(out.cpu().numpy()[fine], want[fine].astype(np.float32))


def test_no_rows(gq):
    a = gq.act(0, 64, torch.bfloat16, 128)
    c, s = gq.alloc_block(a)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gq.gq_block_pack(a, x, c, s)
    gq.gq_block_unpack(a, c, s, x)


def check_weight(gq, w, dtype, lead=0):
    k, o, c = w.shape
    a = gq.act(o, c, TYPES[dtype], 128)
    flat = torch.zeros(lead + w.size, dtype=TYPES[dtype], device="cuda")
    flat[lead:] = torch.as_tensor(w).flatten()
    dev = flat[lead:].view(k, o, c)
    want, turned = S.pack_weight(w, dtype), S.pack_weight(w.transpose(0, 2, 1), dtype)
    for which in ((True, True), (True, False), (False, True)):
        forms = [gq.alloc_block_weight(a, k, transposed=t) if on else None
                 for t, on in zip((False, True), which)]
        for f in forms:
            if f:
                f[0].view(torch.uint8).fill_(0x55)
        gq.gq_block_pack_weight(a, dev, *forms)
        for f, (wc, ws) in zip(forms, (want, turned)):
            if f:
                same_steps(f[1], ws)
                assert np.array_equal(raw(f[0]), wc)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k,o,c,lead", [
    (1, 1, 1, 0), (2, 3, 5, 1), (1, 7, 300, 0), (3, 130, 17, 1), (1, 128, 128, 0),
    (2, 127, 129, 3), (2, 257, 200, 0), (1, 16, 1000, 0), (1, 1000, 8, 0)])
def test_weights(gq, dtype, k, o, c, lead):
    rng = np.random.default_rng([8, o, c])
    w = rng.standard_normal((k, o, c)) * np.exp(rng.standard_normal((k, o, 1)))
    check_weight(gq, torch.as_tensor(w).to(TYPES[dtype]).double().numpy(), dtype, lead)


def test_weights_that_are_not_finite(gq):
    w = np.ones((2, 200, 260))
    w[0, 130, 5], w[1, 3, 259] = np.nan, np.inf
    w[0, :128, 128:256] = 0
    check_weight(gq, w, "f32")


def test_weight_of_a_matrix(gq):
    """A matrix is one expert's weight."""
    a = gq.act(40, 50, torch.float32, 128)
    w = torch.randn(40, 50, device="cuda")
    one, two = gq.alloc_block_weight(a), gq.alloc_block_weight(a)
    gq.gq_block_pack_weight(a, w, one)
    gq.gq_block_pack_weight(a, w[None], two)
    assert np.array_equal(raw(one[0]), raw(two[0])) and torch.equal(one[1], two[1])

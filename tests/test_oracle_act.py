"""Pins of the CPU forms of the 8-bit activation operators: hand-computed
steps and codes, the step's definition, and every gradient against central
differences of the forward formula."""
import numpy as np
import pytest

from oracle import activations as A


def test_steps_by_hand():
    # 127 = 127 * 1; 127.5 needs the next power; 63.5 = 127 / 2
    for m, s in [(127.0, 1.0), (127.5, 2.0), (128.0, 2.0), (63.5, 0.5),
                 (63.51, 1.0), (1.0, 2.0 ** -6), (0.9921875, 2.0 ** -7),
                 (0.0, 0.0), (2.0 ** -149, 2.0 ** -126),
                 (127 * 2.0 ** -126, 2.0 ** -126), (3.4e38, 2.0 ** 121)]:
        assert A.step(m) == s, m
    assert A.step(65504.0, "f16") == 512.0 and A.step(65024.0, "f16") == 512.0
    assert np.isnan(A.step(np.inf)) and np.isnan(A.step(np.nan))


def test_codes_by_hand():
    x = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -127.0, 0.49999]])
    c, s = A.pack(x)
    assert s[0, 0] == 1.0 and c.shape == (1, 16)
    assert c[0].tolist() == [127, 0, 2, 2, 0, -2, -127, 0] + [0] * 8
    # groups are independent; a group with a NaN is all NaN, the next one is not
    x = np.zeros((1, 70))
    x[0, 3], x[0, 40], x[0, 69] = np.nan, 254.0, -1e-3
    c, s = A.pack(x, 32)
    assert np.isnan(s[0, 0]) and s[0, 1] == 2.0 and s[0, 2] == 2.0 ** -16
    back = A.unpack(c, s, 70, 32)
    assert np.isnan(back[0, :32]).all() and back[0, 40] == 254.0
    assert np.count_nonzero(back[0, 32:]) == 2
    assert not c[0, 70:].any()


@pytest.mark.parametrize("group", [0, 32, 64])
def test_error_is_half_a_step_and_exact_in_bf16(group):
    x = np.random.default_rng(5).standard_normal((7, 150)) * np.exp(
        np.random.default_rng(6).uniform(-8, 8, (7, 150)))
    c, s = A.pack(x, group)
    back = A.unpack(c, s, 150, group)
    half = np.repeat(s.astype(np.float64), group or 150, axis=1)[:, :150] / 2
    assert (np.abs(back - x) <= half).all()
    # seven significant bits: the low 16 bits of the fp32 pattern are 0
    assert not (back.astype(np.float32).view(np.uint32) & 0xFFFF).any()


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(7)
    x, w, b, dy = (rng.standard_normal(s) for s in ((5, 9), 9, 9, (5, 9)))
    eps = 1e-3

    def loss(x, w, b):
        return (A.layer_norm(x, w, b, eps)[0] * dy).sum()

    _, mean, rstd = A.layer_norm(x, w, b, eps)
    grads = A.layer_norm_backward(dy, x, mean, rstd, w)
    h = 1e-5
    for k, (v, g) in enumerate(zip((x, w, b), grads)):
        for i in np.ndindex(v.shape):
            up, dn = [x.copy(), w.copy(), b.copy()], [x.copy(), w.copy(), b.copy()]
            up[k][i] += h
            dn[k][i] -= h
            diff = (loss(*up) - loss(*dn)) / (2 * h)
            # the difference is off by h^2 f''' / 6 and by rounding / h
            assert abs(diff - g[i]) < 1e-7 * max(1.0, abs(g[i]))


def test_wgrad_against_differences():
    rng = np.random.default_rng(8)
    x, w, b, dy = (rng.standard_normal(s) for s in ((6, 4), (3, 4), 3, (6, 3)))
    dw, db = A.wgrad(dy, x)

    def loss(w, b):
        return ((x @ w.T + b) * dy).sum()

    h = 1e-4                     # linear: no error but rounding
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((loss(w + d, b) - loss(w - d, b)) / (2 * h) - dw[i]) < 1e-9
    for i in range(3):
        d = np.eye(3)[i] * h
        assert abs((loss(w, b + d) - loss(w, b - d)) / (2 * h) - db[i]) < 1e-9


def test_linear_is_the_product_of_the_decoded_operands():
    rng = np.random.default_rng(9)
    x, w, b = rng.standard_normal((4, 21)), rng.standard_normal((5, 21)), rng.standard_normal(5)
    c, s = A.pack(x)
    wc, ws = A.pack(w)
    want = A.unpack(c, s, 21) @ A.unpack(wc, ws, 21).T + b.astype(np.float32)
    got = A.linear(c, s, wc, ws.ravel(), b.astype(np.float32), 21)
    np.testing.assert_allclose(got, want, rtol=1e-13, atol=1e-13)

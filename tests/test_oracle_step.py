"""Pins of the CPU forms of the 8-bit floating point products and the optimizer's
step (no GPU needed)."""
import numpy as np
import pytest
import torch

from oracle import step as S


def test_codes_are_the_types_values():
    bits = torch.arange(256, dtype=torch.uint8)
    want = bits.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(S.values(bits.numpy()), want, equal_nan=True)
    want = bits[:128].view(torch.float8_e5m2).double().numpy()
    assert np.array_equal(S.E5M2[:0x7c], want[:0x7c])


def test_nearest_is_the_types_rounding():
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.standard_normal(20000) * 100, rng.standard_normal(20000) * 2.0 ** -7,
                        (S.E4M3[:0x7e] + S.E4M3[1:0x7f]) / 2, S.E4M3[:0x7f], [0.0, -0.0]])
    y = np.clip(y, -448, 448).astype(np.float32)
    want = torch.as_tensor(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.nearest(y.astype(np.float64)), want)
    assert S.values(S.nearest(np.array([1e9, -460.0]))).tolist() == [448.0, -448.0]


@pytest.mark.parametrize("m,want", [
    (448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (0.0, 0.0), (1e-45, 2.0 ** -126),
    (3.4e38, 2.0 ** 119), (57344.0, 128.0), (1.0, 2.0 ** -8)])
def test_step(m, want):
    assert S.step(m) == want


def test_pack_and_transpose():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 300)) * np.exp(rng.standard_normal((5, 1)))
    c, s = S.pack(x)
    assert c.shape == (5, 304) and s.shape == (5, 3) and not c[:, 300:].any()
    back = S.unpack(c, s, 300)
    # half a step of e4m3, or of its smallest values
    grain = np.repeat(s.astype(np.float64), 128, axis=1)[:, :300] * 2.0 ** -10
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, grain)).all()
    w = rng.standard_normal((2, 130, 200))
    a = S.unpack_weight(*S.pack_weight(w), 200)
    b = S.unpack_weight(*S.pack_weight(w.transpose(0, 2, 1)), 130)
    assert np.array_equal(a, b.transpose(0, 2, 1))


def test_products_by_expert():
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((9, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((3, 5))
    y, _ = S.linear(x, w, b, [1, 4, 4, 8])
    for t in range(9):
        e = {1: 0, 2: 0, 3: 0, 4: 2, 5: 2, 6: 2, 7: 2}.get(t)
        assert np.isnan(y[t]).all() if e is None else np.allclose(y[t], w[e] @ x[t] + b[e])
    dy = rng.standard_normal((9, 5))
    dw, db = S.wgrad(dy, x, [1, 4, 4, 8])
    assert not dw[1].any() and not db[1].any()
    # against differences of sum(dy * y), linear in w
    for _ in range(10):
        e, o, c = rng.integers(3), rng.integers(5), rng.integers(4)
        d = np.zeros_like(w)
        d[e, o, c] = 1.0
        up, dn = (np.nansum(S.linear(x, w + k * d, b, [1, 4, 4, 8])[0] * dy) for k in (1, -1))
        assert abs((up - dn) / 2 - dw[e, o, c]) < 1e-12 * (1 + abs(up))


def test_adamw_is_torchs():
    rng = np.random.default_rng(4)
    p = rng.standard_normal(50)
    q = torch.nn.Parameter(torch.as_tensor(p.copy()))
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m = v = np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        q.grad = torch.as_tensor(g)
        opt.step()
        p, m, v = S.adamw(p, m, v, g, t, 1e-2, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(p, q.detach().numpy(), rtol=1e-12, atol=1e-13)


def test_adamw_in_32_bits():
    """Against 64 bits: m is off by three roundings of its terms, v by five,
    the update by those, fifteen of its own and what its terms' errors make, and
    p by its last rounding."""
    rng, u = np.random.default_rng(5), 2.0 ** -24
    n = 20000
    f = np.float32
    p, m, v = rng.standard_normal(n).astype(f), rng.standard_normal(n).astype(f), \
        (rng.standard_normal(n) ** 2).astype(f)
    g = (rng.standard_normal(n) * np.exp(rng.standard_normal(n))).astype(f)
    a = S.adamw(p, m, v, g, 7, f(1e-2), 0.9, 0.999, 1e-8, f(0.1), kind=f)
    b = S.adamw(*(x.astype(np.float64) for x in (p, m, v, g)), 7, float(f(1e-2)), 0.9, 0.999,
                1e-8, float(f(0.1)))
    tm = 3 * u * (0.9 * np.abs(m) + 0.1 * np.abs(g)) * 1.01
    tv = 5 * u * b[2] * 1.01
    assert (np.abs(a[1] - b[1]) <= tm).all()
    assert (np.abs(a[2] - b[2]) <= tv).all()
    root = np.sqrt(b[2] / (1 - 0.999 ** 7)) + 1e-8
    size = 1e-2 / (1 - 0.9 ** 7)
    upd = size * np.abs(b[1]) / root
    tp = (u * (np.abs(p) + np.abs(b[0])) + 20 * u * upd + size * tm / root
          + 4 * u * 1e-3 * np.abs(p)) * 1.01
    assert (np.abs(a[0] - b[0]) <= tp).all()


def test_philox_is_the_quantizers():
    import oracle
    oracle.lib()
    w = S.philox(0x1234567890abcdef, 77, 64)
    for c in range(16):
        want = oracle.philox(0x1234567890abcdef, c, 77)
        assert [int(x) for x in w[4 * c:4 * c + 4]] == [int(x) for x in want]
    # a vector of the published generator: key and counter zero
    assert [int(x) for x in S.philox(0, 0, 4)] == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]


def test_state_codes_round_at_random():
    rng = np.random.default_rng(6)
    x = np.concatenate([[448.0], np.full(255, 17.0)])       # between 16 and 18
    ups = 0
    for k in range(64):
        r = rng.integers(0, 65536, 256).astype(np.uint64)
        c, s = S.state_codes(x, r, S.E4M3, 448.0)
        assert s[0] == 1.0 and c[0] == 0x7e
        got = S.state_values(c, s, S.E4M3)[1:]
        assert set(got) <= {16.0, 18.0}
        ups += (got == 18.0).sum()
    n = 64 * 255
    assert abs(ups - n / 2) < 5 * np.sqrt(n) / 2
    # v over 0 stays over 0, zeros stay zeros
    x = np.concatenate([[57344.0, 1e-30, 0.0], np.zeros(253)])
    c, s = S.state_codes(x, np.zeros(256, np.uint64), S.E5M2, 57344.0)
    assert c[:3].tolist() == [0x7b, 1, 0]


def test_states_near_the_largest_number_stay_finite():
    for table, top in ((S.E4M3, 448.0), (S.E5M2, 57344.0)):
        x = np.full(256, np.float64(np.float32(3.2e38)))
        c, s = S.state_codes(x, np.full(256, 65535, np.uint64), table, top)
        assert np.isfinite(S.state_values(c, s, table).astype(np.float32)).all()

"""Plain CPU forms of the 8-bit floating point products and the optimizer's step
(numpy, 64 bits), written from their definitions in include/gq.h: test
infrastructure only."""
from __future__ import annotations

import numpy as np

BLOCK, STATES = 128, 256
CAP = {"f32": 119, "bf16": 119, "f16": 7}


def _table(exp_bits: int, man_bits: int, top: int):
    """Value of each of the 128 codes without sign; NaN past `top`."""
    bias = 2 ** (exp_bits - 1) - 1
    v = np.empty(128)
    for c in range(128):
        e, m = c >> man_bits, c & ((1 << man_bits) - 1)
        v[c] = (m * 2.0 ** (1 - bias - man_bits) if e == 0 else
                (1 + m * 2.0 ** -man_bits) * 2.0 ** (e - bias))
        if c > top:
            v[c] = np.nan
    return v


E4M3 = _table(4, 3, 0x7e)           # largest 448
E5M2 = _table(5, 2, 0x7b)           # largest 57344


def pitch(cols: int) -> int:
    return -(-cols // 16) * 16


def blocks(n: int, size: int = BLOCK) -> int:
    return -(-n // size)


def step(m: float, top: float = 448.0, cap: int = 119) -> float:
    """The smallest power of two with top * step >= m, within the limits."""
    if not np.isfinite(m):
        return float("nan")
    if m == 0:
        return 0.0
    k = max(-126, int(np.floor(np.log2(m / top))) - 2)
    while k < cap and top * 2.0 ** k < m:
        k += 1
    return 2.0 ** k


def nearest(y: np.ndarray) -> np.ndarray:
    """e4m3 codes nearest to y (|y| <= 448 or saturating), ties to even."""
    a = np.minimum(np.abs(y), 448.0)
    hi = np.minimum(np.searchsorted(E4M3[:0x7f], a), 0x7e)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (c | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def values(codes: np.ndarray) -> np.ndarray:
    """What e4m3 codes stand for."""
    c = np.asarray(codes, np.uint8)
    return np.where(c & 128, -1.0, 1.0) * E4M3[c & 127]


def _part(part, cap):
    s = step(np.abs(part).max() if np.isfinite(part).all() else np.nan, 448.0, cap)
    if not s > 0:
        return np.zeros(part.shape, np.uint8), s
    return nearest(part / s), s


def pack(x: np.ndarray, dtype: str = "f32"):
    """(codes uint8 [rows, pitch], steps float32 [rows, groups])."""
    rows, cols = x.shape
    codes = np.zeros((rows, pitch(cols)), np.uint8)
    steps = np.zeros((rows, blocks(cols)), np.float32)
    for k, lo in enumerate(range(0, cols, BLOCK)):
        for r in range(rows):
            part = x[r, lo:lo + BLOCK]
            codes[r, lo:lo + part.size], steps[r, k] = _part(part, CAP[dtype])
    return codes, steps


def unpack(codes, steps, cols: int) -> np.ndarray:
    s = np.repeat(steps.astype(np.float64), BLOCK, axis=-1)[..., :cols]
    return values(codes[..., :cols]) * s


def pack_weight(w: np.ndarray, dtype: str = "f32"):
    """(codes [experts, out, pitch], steps [experts, blocks, blocks])."""
    k, o, c = w.shape
    codes = np.zeros((k, o, pitch(c)), np.uint8)
    steps = np.zeros((k, blocks(o), blocks(c)), np.float32)
    for e in range(k):
        for i, a in enumerate(range(0, o, BLOCK)):
            for j, b in enumerate(range(0, c, BLOCK)):
                part = w[e, a:a + BLOCK, b:b + BLOCK]
                q, steps[e, i, j] = _part(part, CAP[dtype])
                codes[e, a:a + BLOCK, b:b + part.shape[1]] = q
    return codes, steps


def unpack_weight(codes, steps, cols: int) -> np.ndarray:
    s = np.repeat(steps, BLOCK, axis=-2)[..., :codes.shape[-2], :]
    return unpack(codes, s, cols)


def linear(x, w, bias, offsets):
    """(y, sum of the terms' magnitudes); rows of no expert are NaN, 0."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        r = slice(offsets[e], offsets[e + 1])
        y[r] = x[r] @ w[e].T
        mag[r] = np.abs(x[r]) @ np.abs(w[e]).T
        if bias is not None:
            y[r] += bias[e]
            mag[r] += np.abs(bias[e])
    return y, mag


def wgrad(dy, x, offsets):
    """(dweight [experts, out, cols], dbias [experts, out])."""
    k = len(offsets) - 1
    dw = np.zeros((k, dy.shape[1], x.shape[1]))
    db = np.zeros((k, dy.shape[1]))
    for e in range(k):
        r = slice(offsets[e], offsets[e + 1])
        dw[e], db[e] = dy[r].T @ x[r], dy[r].sum(0)
    return dw, db


# ------------------------------------------------------------- the step ----
def philox(seed: int, step: int, n: int, first: int = 0) -> np.ndarray:
    """Word i mod 4 of Philox4x32-10 at the counter (i / 4, step), for n values i
    from `first` on."""
    low, skip = np.uint64(0xffffffff), first % 4
    i = np.arange(-(-(n + skip) // 4), dtype=np.uint64) + np.uint64(first // 4)
    c = [i & low, i >> np.uint64(32), np.full_like(i, step), np.zeros_like(i)]
    k = [seed & 0xffffffff, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return np.stack(c, 1).reshape(-1)[skip:skip + n]


def state_codes(x, r16, table, top: float):
    """Codes and steps of a state (float64 [n], uint64 r16 [n]); up where the
    place between two codes, cut to 16 bits, and r16 reach one."""
    n = x.size
    cap = 112 if table is E5M2 else 119     # top * 2^cap is finite in 32 bits
    steps = np.array([step(np.abs(x[a:a + STATES]).max() if np.isfinite(x[a:a + STATES]).all()
                           else np.nan, top, cap) for a in range(0, n, STATES)], np.float32)
    s = np.repeat(steps.astype(np.float64), STATES)[:n]
    fine = s > 0
    y = np.where(fine, np.abs(x) / np.where(fine, s, 1.0), 0.0)
    good = table[~np.isnan(table)]
    lo = np.searchsorted(good, y, side="right") - 1
    hi = np.minimum(lo + 1, good.size - 1)
    gap = np.where(hi > lo, good[hi] - good[lo], 1.0)
    f = np.floor((y - good[lo]) / gap * 65536.0)
    c = np.where(f + r16.astype(np.float64) >= 65536.0, hi, lo)
    if table is E5M2:
        c = np.where(fine & (x > 0), np.maximum(c, 1), c)
    c = np.where(fine, c | np.where(x < 0, 128, 0), c * 0)
    return c.astype(np.uint8), steps


def state_values(codes, steps, table):
    v = np.where(codes & 128, -1.0, 1.0) * table[codes & 127]
    return v * np.repeat(steps.astype(np.float64), STATES)[:codes.size]


def adamw(p, m, v, g, t, lr, beta1, beta2, eps, decay, grad_scale=1.0, kind=np.float64):
    """(p, m, v) after a step; lr, decay: numbers or one per value.  kind =
    np.float32: every operation rounded to 32 bits, in the order that the
    library's arithmetic has."""
    if kind is np.float64:
        g = g * grad_scale
        m = beta1 * m + (1 - beta1) * g
        v = beta2 * v + (1 - beta2) * g * g
        mh, vh = m / (1 - beta1 ** t), v / (1 - beta2 ** t)
        return p - lr * (mh / (np.sqrt(vh) + eps)) - lr * decay * p, m, v
    f = np.float32
    p, m, v, g, lr, decay = (np.asarray(a, f) for a in (p, m, v, g, lr, decay))
    d = g * f(grad_scale)
    m = m * f(beta1) + d * f(1 - beta1)
    v = v * f(beta2) + d * f(1 - beta2) * d
    size, wd = lr * f(1 / (1 - beta1 ** t)), lr * decay
    root = np.sqrt(v) * f(1 / np.sqrt(1 - beta2 ** t)) + f(eps)
    return p - (size * m / root + wd * p), m, v

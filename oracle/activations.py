"""Plain CPU forms of the 8-bit activation operators (numpy, 64 bits), written
from their definitions in include/gq.h: test infrastructure only.

Matrices are float64 arrays that hold values of the activations' type."""
from __future__ import annotations

import numpy as np

STEP_CAP = {"f32": 121, "bf16": 121, "f16": 9}


def pitch(cols: int) -> int:
    return -(-cols // 16) * 16


def groups(cols: int, group: int) -> int:
    return -(-cols // group) if group else 1


def step(m: float, dtype: str = "f32") -> float:
    """The smallest power of two with 127 * step >= m, within the limits."""
    if not np.isfinite(m):
        return float("nan")
    if m == 0:
        return 0.0
    k = -126
    while k < STEP_CAP[dtype] and 127.0 * 2.0 ** k < m:
        k += 1
    return 2.0 ** k


def pack(x: np.ndarray, group: int = 0, dtype: str = "f32"):
    """(codes int8 [rows, pitch], steps float32 [rows, groups])."""
    rows, cols = x.shape
    codes = np.zeros((rows, pitch(cols)), np.int8)
    steps = np.zeros((rows, groups(cols, group)), np.float32)
    for k, lo in enumerate(range(0, cols, group or cols)):
        part = x[:, lo:lo + (group or cols)]
        mags = np.abs(part).max(axis=1)       # NaN where a NaN is
        tabled = {m: step(m, dtype) for m in set(mags[np.isfinite(mags)].tolist())}
        for r in range(rows):
            s = tabled[mags[r]] if np.isfinite(mags[r]) else float("nan")
            steps[r, k] = s
            if s > 0:
                q = np.rint(part[r] / s)      # ties to even
                codes[r, lo:lo + part.shape[1]] = np.clip(q, -127, 127)
    return codes, steps


def unpack(codes: np.ndarray, steps: np.ndarray, cols: int, group: int = 0) -> np.ndarray:
    s = np.repeat(steps.astype(np.float64), group or cols, axis=1)[:, :cols]
    return codes[:, :cols].astype(np.float64) * s


def linear(codes, steps, w_codes, w_steps, bias, cols: int) -> np.ndarray:
    # whole numbers below 2^53: exact in 64-bit floats
    acc = codes[:, :cols].astype(np.float64) @ w_codes[:, :cols].astype(np.float64).T
    y = acc * steps.reshape(-1, 1).astype(np.float64) * w_steps.astype(np.float64)[None, :]
    return y if bias is None else y + bias.astype(np.float64)


def wgrad(dy: np.ndarray, x: np.ndarray):
    """(dweight [out, cols], dbias [out]) of y = x w^T + b."""
    return dy.T @ x, dy.sum(axis=0)


def layer_norm(x, weight, bias, eps: float):
    """(y, mean, rstd); weight and bias may be None."""
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias) with mean and rstd as they were kept."""
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy if weight is None else dy * weight
    m1 = a.mean(axis=1)[:, None]
    m2 = (a * xh).mean(axis=1)[:, None]
    return rstd[:, None] * (a - m1 - xh * m2), (dy * xh).sum(axis=0), dy.sum(axis=0)

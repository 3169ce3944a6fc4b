"""Oracle of the 8-bit rows, the norm that writes them and the 8-bit integer linears.

Test infrastructure only (see the package docstring). Codes and scales of given fp32 rows are defined bit for bit and
restated in numpy fp32; the norm and the gated product are plain fp64, the integer product is exact.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


def quantize_rows(v: np.ndarray):
    """Rows of fp32 values [M][K] -> (codes int8 [M][K], scales fp32 [M]):
    a = max |v|, scale = fl(a / 127), code = clamp(rint(v * fl(127 / a)), -127, 127); a < 2^-100: zeros; not finite: NaN."""
    v = np.ascontiguousarray(v, dtype=F32)
    codes, scales = np.zeros(v.shape, np.int8), np.zeros(v.shape[0], F32)
    for i, row in enumerate(v):
        if not np.all(np.isfinite(row)):
            scales[i] = np.nan
            continue
        a = F32(np.abs(row).max())
        if a >= F32(2.0 ** -100):
            scales[i] = a / F32(127)
            codes[i] = np.clip(np.rint(row * (F32(127) / a)), -127, 127).astype(np.int8)
    return codes, scales


def rms_norm(x, weight, eps, residual=None):
    """(h, v) in fp64 of x, residual [M][K] and weight [K]: h = x + residual, v = h / sqrt(mean h^2 + eps) * weight."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def sums(q_x: np.ndarray, q_w: np.ndarray) -> np.ndarray:
    """Exact integer products [M][N] of codes [M][K] and [N][K]. Codes are at most 128 in size, so that fp64 holds the
    products and sums of any K below 2^38 exactly."""
    return np.asarray(q_x, np.float64) @ np.asarray(q_w, np.float64).T


def linear(q_x, s_x, q_w, s_w) -> np.ndarray:
    """fp32 [M][N]: fl(fl(sum * s_x) * s_w), for sums below 2^24."""
    p = sums(q_x, q_w)
    assert np.abs(p).max(initial=0) < 2 ** 24
    return p.astype(F32) * np.asarray(s_x, F32)[:, None] * np.asarray(s_w, F32)


def act(g: np.ndarray, kind: str) -> np.ndarray:
    g = np.asarray(g, np.float64)
    z = g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-z))


def gated(q_x, s_x, q_w, s_w, q_u, s_u, kind="silu") -> np.ndarray:
    """fp64 [M][N]: act(x W^T) * (x U^T)."""
    s_x = np.asarray(s_x, np.float64)[:, None]
    return act(sums(q_x, q_w) * s_x * np.asarray(s_w, np.float64), kind) * (sums(q_x, q_u) * s_x * np.asarray(s_u, np.float64))

"""Plain numpy restatement of the 4-bit key/value cache and its attention.

Quantisation and rotation follow the definition operation by operation in fp32
(their results are defined bit for bit); attention is fp64 and returns, beside
the result, what its error bounds are made of.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bit patterns, round to nearest even (NaN -> 0x7FC0)."""
    u = np.ascontiguousarray(x, dtype=F32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FC0), r)


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(F32)


def rotate(x: np.ndarray, table_rows: np.ndarray, interleaved: bool) -> np.ndarray:
    """x fp32 [T][H][D], table_rows fp32 [T][R] (cosines, sines): rotated fp32."""
    R = table_rows.shape[1]
    y = x.astype(F32).copy()
    if R == 0:
        return y
    c, s = table_rows[:, None, :R // 2].astype(F32), table_rows[:, None, R // 2:].astype(F32)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    x1, x2 = y[..., a].copy(), y[..., b].copy()
    with np.errstate(all="ignore"):
        y[..., a] = x1 * c - x2 * s
        y[..., b] = x2 * c + x1 * s
    return y


def quantise(x: np.ndarray):
    """Rows x fp32 [..., D]: codes uint8 [..., D] and bf16 bits (scale, offset) uint16 [..., 2]."""
    x = np.asarray(x, F32)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        rng = hi - lo
        sb, ob = bf16_bits(rng * F32(1.0 / 15.0)), bf16_bits(lo)
        s = bf16_value(sb)
        sb = np.where(s < F32(2.0 ** -126), np.uint16(0), sb)
        s, o = bf16_value(sb), bf16_value(ob)
        inv = np.where(s > 0, F32(1) / np.where(s > 0, s, F32(1)), F32(0)).astype(F32)
        code = np.rint((x - o) * inv)
        code = np.where(np.isnan(code), 0, np.clip(code, 0, 15)).astype(np.uint8)
        bad = ~np.isfinite(x).all(-1, keepdims=True) | ~(rng <= F32(2.0 ** 120))
    par = np.concatenate([sb, ob], -1)
    return code, np.where(bad, np.uint16(0x7FC0), par)


def pack_rows(pool: np.ndarray, page_size: int, D: int, slots, k_codes, k_par, v_codes, v_par) -> None:
    """Write tokens' rows into a pool uint8 [pages][heads][page bytes] (in place)."""
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        page, at = divmod(int(slot), page_size)
        blk, r = divmod(at, 16)
        base = blk * 16 * (D + 8)
        for is_v, (codes, par) in enumerate(((k_codes[t], k_par[t]), (v_codes[t], v_par[t]))):
            packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
            o = base + is_v * 8 * D + r * (D // 2)
            pool[page, :, o:o + D // 2] = packed
            o = base + 16 * D + is_v * 64 + r * 4
            pool[page, :, o:o + 4] = np.ascontiguousarray(par.astype("<u2")).view(np.uint8).reshape(par.shape[0], 4)


def unpack_rows(pool: np.ndarray, page_size: int, D: int, slots):
    """(K, V) fp64 values [len(slots)][heads][D] that the slots stand for."""
    out = []
    slots = np.asarray(slots, np.int64)
    page, at = slots // page_size, slots % page_size
    base, r = at // 16 * 16 * (D + 8), at % 16
    heads = np.arange(pool.shape[1])[None, :, None]
    for is_v in (0, 1):
        o = (base + is_v * 8 * D + r * (D // 2))[:, None, None] + np.arange(D // 2)
        b = pool[page[:, None, None], heads, o]
        codes = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:2], D).astype(np.float64)
        o = (base + 16 * D + is_v * 64 + r * 4)[:, None, None] + np.arange(4)
        par = np.ascontiguousarray(pool[page[:, None, None], heads, o]).view("<u2")
        v = bf16_value(par).astype(np.float64)
        out.append(codes * v[..., :1] + v[..., 1:])
    return out


def attention(q: np.ndarray, K: np.ndarray, V: np.ndarray, scale: float, window: int = 0):
    """q fp64 [n][Hq][D], K and V fp64 [L][Hk][D]. Returns out [n][Hq][D] and, for error bounds, [n][Hq] each:
    the weighted mean of the values' largest elements and the largest sum of |q k| scale."""
    n, Hq, D = q.shape
    L, Hk = K.shape[:2]
    g = Hq // Hk
    out, mag, ref = np.zeros((n, Hq, D)), np.zeros((n, Hq)), np.zeros((n, Hq))
    for i in range(n):
        p = L - n + i
        lo = max(0, p - window + 1) if window else 0
        if p < lo:
            continue
        for h in range(Hq):
            k, v = K[lo:p + 1, h // g], V[lo:p + 1, h // g]
            s = (k @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ v, w @ np.abs(v).max(-1)
            ref[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
    return out, mag, ref


def tolerance(out: np.ndarray, mag: np.ndarray, ref: np.ndarray, keys: float = 2.0 ** -9) -> np.ndarray:
    """Largest error of an implementation that rounds the result to bf16 once, weights and cached values to f16 once, and
    keeps everything else in fp32. Keys off by `keys` move a score by d = keys ref at most and a weight by a factor
    within exp(+-2 d) (numerator and denominator). The result's rounding is 2^-8 of it at most, which is no larger than
    mag; those of weights and values are 2^-11 each, of a value or of its distance from the middle of its row's range,
    which is at most 16/15 of the row's largest element (mag). That leaves 2^-8 of mag for fp32 sums and for keys whose
    weights and values go through bf16, 2^-8 each: where such a key alone makes the result and all three roundings are
    at their worst together, they pass the bound by a quarter. The bound scales with the values and is zero for a row
    that sees none but zeros: such a row has no error."""
    d = keys * ref[..., None]
    return 2.0 ** -9 * np.abs(out) + (np.expm1(2 * d) + 3.5 * 2.0 ** -9) * mag[..., None] * 16 / 15

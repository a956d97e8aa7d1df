"""The cache in 4 or 8 bits, modelled on the host in 64 bits (test helper; numpy and torch's number formats only).

Every rule is evaluated by looking through all values that a scale or a code can have, exactly: scales have
4 bits, codes 2 or 7, inputs at most 24, so the products compared here are exact in 64 bits.
"""
import numpy as np
import torch

MAGS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
FMT = {"e2m1": 0, "int8": 1}


def scale_values() -> np.ndarray:
    """The 248 finite scales by their byte: fp16 numbers whose bits are byte << 7."""
    return (np.arange(248, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)


def row_bytes(fmt, hd):
    return (hd // 2 if fmt == "e2m1" else hd) + hd // 16


def scale_byte(amax: np.ndarray, fmt: str) -> np.ndarray:
    s = scale_values()
    if fmt == "int8":
        return np.minimum(np.searchsorted(127 * s, amax), 192)      # the first that is large enough
    b = np.arange(227)
    six = 6 * s[b]
    hi = np.minimum(np.searchsorted(six, amax), 226)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(six[hi] - amax), np.abs(amax - six[lo])
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """[..., head_dim] values (float64 holding fp32 / fp16 / bf16 numbers) as bytes [..., row_bytes]."""
    hd = x.shape[-1]
    g = x.reshape(*x.shape[:-1], hd // 16, 16)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    byte = scale_byte(np.abs(g).max(-1), fmt)
    s = scale_values()[byte][..., None]
    if fmt == "e2m1":
        a = np.abs(g)
        code = np.zeros(g.shape, dtype=np.int64)
        for k in range(1, 8):     # past the middle of k - 1 and k, or on it and k even
            mid = (MAGS[k - 1] + MAGS[k]) / 2 * s
            code = np.where((a > mid) | ((a == mid) & (k % 2 == 0)), k, code)
        code = np.where(np.signbit(g), code + 8, code)
        code = np.where((byte == 0)[..., None], 0, code).reshape(*x.shape)
        codes = code[..., 0::2] + 16 * code[..., 1::2]
    else:
        lim = np.clip(g, -127 * s, 127 * s)
        n = np.rint(lim / np.where(s == 0, 1, s))
        r = lim - n * s             # exact
        n = n + ((2 * r > s) | ((2 * r == s) & (n % 2 != 0))) - ((2 * r < -s) | ((2 * r == -s) & (n % 2 != 0)))
        codes = np.where((byte == 0)[..., None], 0, n).reshape(*x.shape).astype(np.int8).view(np.uint8)
    byte = np.where(bad, 255, byte)
    codes = np.where(np.repeat(bad, codes.shape[-1] // (hd // 16), -1), 0, codes)
    return np.concatenate([codes, byte], -1).astype(np.uint8)


def decode(rows: np.ndarray, fmt: str, hd: int) -> np.ndarray:
    """Bytes [..., row_bytes] as float64 values [..., head_dim]."""
    n = row_bytes(fmt, hd) - hd // 16
    s = (rows[..., n:].astype(np.uint16) << 7).view(np.float16).astype(np.float64).repeat(16, -1)
    if fmt == "int8":
        return rows[..., :n].view(np.int8).astype(np.float64) * s
    c = np.stack([rows[..., :n] & 15, rows[..., :n] >> 4], -1).reshape(*rows.shape[:-1], hd)
    return np.where(c & 8, -MAGS[c & 7], MAGS[c & 7]) * s


def rounded(x: np.ndarray, dtype: torch.dtype) -> np.ndarray:
    """float64 rounded once, to nearest even, to the dtype (normal range), as float64."""
    if dtype == torch.float32:
        return x.astype(np.float32).astype(np.float64)
    bits, low = (8, -126) if dtype == torch.bfloat16 else (11, -14)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - 1, low) - (bits - 1.0))
    with np.errstate(invalid="ignore"):
        y = np.rint(x / step) * step
    top = float(torch.finfo(dtype).max)
    return np.where(np.abs(y) > top, np.copysign(np.inf, y), y)


def rotated(x: np.ndarray, c: np.ndarray, s: np.ndarray, style: str) -> np.ndarray:
    """x [T, heads, hd] rotated by c, s [T, hd / 2] (float64, one rounding at 2^-53)."""
    c, s = c[:, None], s[:, None]
    y = np.empty_like(x)
    h = x.shape[-1] // 2
    a, b = (slice(0, h), slice(h, None)) if style == "neox" else (slice(0, None, 2), slice(1, None, 2))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def held_k(x, c, s, style, dtype):
    """The rotated K that is quantised: rounded to fp32, and from there to the dtype."""
    return rounded(rounded(rotated(x, c, s, style), torch.float32), dtype)

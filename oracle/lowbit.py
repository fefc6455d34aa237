"""Plain numpy definitions of the norm with quantized output and of MXFP4 (test infrastructure only).

Written from the formats' definitions, without the library's code: sums and statistics in 64 bits, and
every fp32 operation that decides a code as one IEEE operation, so that codes can be compared exactly.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(v: np.ndarray):
    """MXFP4 of fp32 v [rows, cols]: codes uint8 [rows, cols] (0..15) and scale bytes uint8 [rows, cols/32]."""
    v = np.ascontiguousarray(v, np.float32)
    rows, cols = v.shape
    b = v.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], np.float32(0), b)
    top = np.abs(b).max(-1).astype(np.float64)
    _, e = np.frexp(top)  # top = m * 2^e, m in [0.5, 1)
    E = np.where(top > 0, np.clip(e - 3, -127, 127), -127)
    a = np.ldexp(np.abs(b).astype(np.float64), -E[..., None])
    # nearest magnitude; a tie goes to the one with an even code
    dist = np.abs(a[..., None] - MAGNITUDES)
    best = dist.min(-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(a > 6.0, 7, code).astype(np.uint8)
    code |= (np.signbit(b).astype(np.uint8) << 3)
    code[bad] = 0
    return code.reshape(rows, cols), np.where(bad, 255, E + 127).astype(np.uint8)


def mx4_values(code: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The values (float64 [rows, cols]) of codes and scale bytes."""
    rows, cols = code.shape
    m = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
    s = np.ldexp(1.0, scale.astype(np.int64) - 127)
    s = np.where(scale == 255, np.nan, s)
    return (m.reshape(rows, cols // 32, 32) * s[..., None]).reshape(rows, cols)


def pack_codes(code: np.ndarray) -> np.ndarray:
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def scale_offsets(rows: int, cols: int) -> np.ndarray:
    """Byte offset [rows, cols/32] of each block's scale in the tiled layout."""
    r = np.arange(rows, dtype=np.int64)[:, None]
    b = np.arange(cols // 32, dtype=np.int64)[None, :]
    tile = (r // 128) * (-(-cols // 128)) + b // 4
    return tile * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def tile_scales(scale: np.ndarray, fill: int = 127) -> np.ndarray:
    rows, blocks = scale.shape
    out = np.full((-(-rows // 128)) * (-(-blocks // 4)) * 512, fill, np.uint8)
    out[scale_offsets(rows, blocks * 32)] = scale
    return out


def rmsnorm(x: np.ndarray, r, gamma: np.ndarray, eps: float):
    """h = fl32(x + r), rstd [rows] and y = fl32(fl32(h*rstd)*gamma), all fp32, with the row statistic in 64 bits.

    Also returns, per row, whether the 64-bit statistic lies so near a border between two fp32 values
    that the order of its sum (n terms, each addition off by 2^-53) decides rstd's rounding.
    """
    h = x.astype(np.float32)
    if r is not None:
        h = (h + r.astype(np.float32)).astype(np.float32)
    n = h.shape[1]
    with np.errstate(all="ignore"):
        ms = (h.astype(np.float64) ** 2).sum(-1) / n + eps
        rstd64 = 1.0 / np.sqrt(ms)
        slack = (n + 4) * 2.0 ** -53
        rstd = rstd64.astype(np.float32)
        near = (rstd64 * (1 - slack)).astype(np.float32) != (rstd64 * (1 + slack)).astype(np.float32)
        y = ((h * rstd[:, None]).astype(np.float32) * gamma.astype(np.float32)).astype(np.float32)
    return h, rstd, y, near


def act_codes(v: np.ndarray, bits: int):
    """Per-row symmetric integer codes int8 and scales fl32(max|v| / qmax) of fp32 v; a row that is not
    finite: NaN and 0."""
    qmax = np.float32(2 ** (bits - 1) - 1)
    ok = np.isfinite(v).all(-1)
    w = np.where(ok[:, None], v, np.float32(0)).astype(np.float32)
    sa = (np.abs(w).max(-1) / qmax).astype(np.float32)
    with np.errstate(all="ignore"):
        q = np.rint((w / sa[:, None]).astype(np.float32))
    q = np.where(sa[:, None] > 0, np.clip(q, -qmax, qmax), 0).astype(np.int8)
    return q, np.where(ok, sa, np.float32("nan"))

"""MXFP4 in numpy, 64 bits: the conversion, its inverse and the layout in bytes.

OCP Microscaling Formats 1.0, sections 5.3 (E2M1 elements, E8M0 scales, blocks of 32) and 6.3
(conversion). Written from the format's definition: the element is found among the eight
magnitudes, not computed from bit fields.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def code_pitch(K: int) -> int:
    return -(-K // 128) * 64


def scale_pitch(K: int) -> int:
    return -(-K // 512) * 16


def _nearest(a: np.ndarray) -> np.ndarray:
    """Index of the nearest magnitude, ties to the even index, saturating at the last."""
    a = np.minimum(a, 6.0)
    lo = np.searchsorted(MAGNITUDES, a, side="right") - 1
    hi = np.minimum(lo + 1, 7)
    below, above = a - MAGNITUDES[lo], MAGNITUDES[hi] - a
    take_hi = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def encode(v: np.ndarray):
    """(codes uint8 [rows, code_pitch], scales uint8 [rows, scale_pitch]) of [rows, K] values."""
    v = np.asarray(v, dtype=np.float64)
    rows, K = v.shape
    codes = np.zeros((rows, code_pitch(K)), np.uint8)
    scales = np.zeros((rows, scale_pitch(K)), np.uint8)
    for b in range(-(-K // 32)):
        x = np.zeros((rows, 32))
        part = v[:, 32 * b:32 * b + 32]
        x[:, :part.shape[1]] = part
        bad = ~np.isfinite(x).all(1)
        amax = np.abs(np.where(bad[:, None], 0.0, x)).max(1)
        e = np.frexp(np.where(amax > 0, amax, 1.0))[1] - 1          # floor(log2 amax)
        s = np.where(amax > 0, np.maximum(e - 2, -127), -127)
        c = _nearest(np.abs(np.ldexp(np.where(bad[:, None], 0.0, x), -s[:, None])))
        c = np.where(np.signbit(x) & ~bad[:, None], c + 8, c).astype(np.uint8)
        codes[:, 16 * b:16 * b + 16] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[:, b] = np.where(bad, 255, s + 127)
    return codes, scales


def decode(codes: np.ndarray, scales: np.ndarray, K: int) -> np.ndarray:
    """The values [rows, K] that the bytes stand for."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)[:, :K]
    v = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = scales[:, np.arange(K) // 32].astype(np.int64)
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127))

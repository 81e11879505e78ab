"""Rows in 8 bits in float64 (oracle; test infrastructure only): e4m3 numbers and an
exponent byte, which stand for number * 2^(byte - 127).

A byte of e4m3: sign, four bits of exponent e, three of significand m; (1 + m / 8) 2^(e - 7),
or m / 8 * 2^-6 where e is 0; e = 15, m = 7 is NaN.
"""
import numpy as np


def _magnitude(code):
    e, m = code >> 3, code & 7
    return (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6


MAGNITUDES = np.array([_magnitude(c) for c in range(127)] + [np.nan])
NUMBERS = np.concatenate((MAGNITUDES, -MAGNITUDES))  # by code
BORDERS = (MAGNITUDES[1:127] + MAGNITUDES[:126]) / 2  # between code i and i + 1


def exponent(top):
    """The byte of rows whose largest finite magnitude is `top`: 0 for none, else the smallest from 1
    on with top <= 448 * 2^(byte - 127)."""
    top = np.asarray(top, dtype=np.float64)
    part, up = np.frexp(top)  # top = part * 2^up, part in [1/2, 1); 448 = 7/8 * 2^9
    return np.where(top > 0, np.maximum(up - 9 + (part > 0.875) + 127, 1), 0).astype(np.uint8)


def quantise(x):
    """(codes uint8, bytes uint8 [..]) of rows x [.., width]."""
    x = np.asarray(x, dtype=np.float64)
    finite = np.isfinite(x)
    top = np.where(finite, np.abs(x), 0.0).max(-1)
    byte = exponent(top)
    z = np.abs(np.where(finite, x, 0.0)) * 2.0 ** (127.0 - np.maximum(byte, 1))[..., None]
    below, upto = np.searchsorted(BORDERS, z, "left"), np.searchsorted(BORDERS, z, "right")
    code = np.where(below % 2 == 0, below, upto)  # they differ on a border alone: the even one
    return np.where(finite, code | np.where(np.signbit(x), 0x80, 0), 0x7F).astype(np.uint8), byte


def values(codes, byte):
    """Rows in float64; a byte of 0 is a row of zeros."""
    scale = np.where(byte == 0, 0.0, 2.0 ** (np.asarray(byte, dtype=np.float64) - 127))
    with np.errstate(invalid="ignore"):
        return NUMBERS[codes] * scale[..., None]

"""Append into 8-bit pages at the farthest positions and the highest frequencies: an angle of 2^37
radians does not fit 53 bits, and its codes are those of the exact one."""
import math

import numpy as np
import pytest
import torch

from e4m3_inputs import Batch8
from oracle import e4m3

# 2 pi in units of 2^-160, by Machin's formula in integers with 32 bits to spare.
_BITS = 160


def _arctan_inverse(n, unit):
    term, total, k = unit // n, 0, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= n * n
        k += 2
    return total


def _two_pi():
    unit = 1 << (_BITS + 32)
    return 2 * (16 * _arctan_inverse(5, unit) - 4 * _arctan_inverse(239, unit)) >> 32


def _turn(pos, freq):
    """(cos, sin) of pos * freq, freq a float: the product exact, its whole turns taken out exactly."""
    num, den = float(freq).as_integer_ratio()
    angle = (pos * num << _BITS) // den  # off by 2^-160
    rest = angle % _two_pi()
    x = rest / (1 << _BITS)
    return math.cos(x), math.sin(x)


def test_the_reduction():
    assert abs(_two_pi() / (1 << _BITS) - 2 * math.pi) < 1e-15
    for pos, freq in ((3, 0.25), (1000, 1.0), (12345, 0.123)):
        c, s = _turn(pos, np.float32(freq))
        assert abs(c - math.cos(pos * float(np.float32(freq)))) < 1e-11 and abs(s - math.sin(pos * float(np.float32(freq)))) < 1e-11


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs,inter", [(64, False), (64, True), (60, False)])
def test_codes_of_far_positions(pairs, inter, dtype):
    import exact_tiled_softmax_gb300 as ex
    n, d, kv, offset = 1500, 128, 8, 2 ** 31 - 1 - 1700
    b = Batch8([n], [n], 1, kv, d, 16, dtype, 64, seed=pairs + inter)
    inv = (64.0 * 10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    k, v, table, lens, starts, ks, vs = b.cache()
    kn, vn = b.dev("k_new", "v_new")
    ex.append_paged(kn, vn, k, v, table, lens, q_starts=starts, inv_freq=torch.from_numpy(inv).cuda(),
                    interleaved=inter, pos_offset=offset, k_scales=ks, v_scales=vs)
    cs = np.array([[_turn(offset + i, f) for f in inv] for i in range(n)])[:, None]  # [n][1][pairs][2]
    x = b.np(b.k_new)
    first, second = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if inter else (slice(0, pairs), slice(pairs, 2 * pairs))
    y = x.copy()
    y[..., first] = x[..., first] * cs[..., 0] - x[..., second] * cs[..., 1]
    y[..., second] = x[..., second] * cs[..., 0] + x[..., first] * cs[..., 1]
    codes, byte = e4m3.quantise(y)
    at, off = b.table[0][np.arange(n) // 64], np.arange(n) % 64
    got, gb = k.view(torch.uint8).cpu().numpy()[at, :, off], ks.cpu().numpy()[at, :, off]
    got, codes = (np.where(z == 0x80, 0, z) for z in (got, codes))
    assert np.array_equal(gb, byte)
    assert np.array_equal(got, codes), int((got != codes).sum())

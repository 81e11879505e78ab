"""Attention over 8-bit pages whose rows are very large or very small, against the oracle, with Y's
bound taken at the size of the values (tests that compare Y itself have an absolute term of 1e-30)."""
import math

import numpy as np
import pytest
import torch

from e4m3_inputs import Batch8, small_weights, weight_bits
from oracle import e4m3
from oracle import paged as oracle
from paged_inputs import check_attention
from test_gpu_paged_e4m3 import _attend, _behind, ex, path  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def _check_at(path, b, y, L, scale, mask, up, prefix=None):
    """The results against the oracle's, Y and its bound times 2^up."""
    with np.errstate(invalid="ignore"):
        Y, Lr, A, D = oracle.attend(b.np(b.q), b.k64, b.v64, b.table, b.lens, b.starts, scale, mask, 0, prefix)
    W = b.largest_weight((Y, Lr, A, D), scale, mask, 0, prefix)
    d, v = b.k64.shape[3], b.v64.shape[3]
    n = int(b.lens.max()) + (prefix[1] if prefix else 0)
    rows = (b.T if prefix else -(-b.T // len(b.lens))) * (b.H // b.kv)
    bits = weight_bits(path, b.dtype, d, v, b.page, rows, scale)
    A = A + small_weights(W, n) * 2.0 ** bits
    own = np.isfinite(Lr)
    assert np.median(A[own]) * 2.0 ** up > 2.0 ** -20  # the term of 1e-30 is far below the bound
    check_attention(b.dtype, y.double() * 2.0 ** up, L, (Y * 2.0 ** up, Lr, A * 2.0 ** up, D), d, n, bits,
                    extra=2.0 ** -20 if prefix else 0.0)


def _shift(b, name, up, least, most):
    s = getattr(b, name + "_scales")
    used = s != 255
    s[used] = np.clip(s[used].astype(int) + up, least, most).astype(np.uint8)
    b.requantised()


@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 6), ("bf16", 40), ("f32", 2)])
@pytest.mark.parametrize("v_up", [-110, -100, -60])
def test_small_values(ex, path, dtype, nq, v_up, prefix):  # noqa: F811
    b = Batch8([200, 43], [nq, nq], 4, 2, 64, 64, dtype, 16, seed=13, prefix=prefix)
    _shift(b, "v", v_up, 3, 246)
    if prefix:
        y, L, status = _behind(ex, b, prefix, "causal", 0.06)
    else:
        y, L, status = _attend(ex, b, "causal", 0, 0.06)
    assert status == 0
    _check_at(path, b, y, L, 0.06, "causal", -v_up, (b.prefix_table, prefix) if prefix else None)


def _coded(rng, shape, size, least, most):
    """Codes and bytes of rows of about `size`, bytes anywhere from `least` to `most`."""
    byte = rng.integers(least, most + 1, shape[:3]).astype(np.uint8)
    z = rng.standard_normal(shape) * (size / 2.0 ** (byte.astype(np.float64) - 127))[..., None]
    return e4m3.quantise(np.concatenate((np.clip(z, -448, 448), np.full(shape[:3] + (1,), 448.0)), -1))[0][..., :-1], byte


# The kernels whose operands are codes without their rows' powers of two: all but the 256-row one.
@pytest.mark.parametrize("dtype,nq,d", [("bf16", 1, 64), ("bf16", 6, 16), ("f32", 2, 64), ("f32", 9, 16), ("bf16", 20, 256)])
@pytest.mark.parametrize("k_bytes,k_size,v_bytes,v_size,q_size,gain", [
    ((247, 254), 2.0 ** 121, (247, 254), 2.0 ** 117, 2.0 ** -120, 1),
    ((247, 254), 2.0 ** 126, (1, 2), 2.0 ** -118, 2.0 ** -110, 1),
    ((252, 254), 2.0 ** 134, (1, 1), 2.0 ** -118, 2.0 ** -123, 1),  # scale times q below fp32's normal numbers
    ((1, 2), 2.0 ** -118, (1, 254), 2.0 ** -50, 2.0 ** 122, 1),
    ((1, 1), 2.0 ** -120, (120, 130), 1.0, 2.0 ** 124, 8)])  # scale times q times a code above its largest
def test_bytes_of_either_end(ex, path, dtype, nq, d, k_bytes, k_size, v_bytes, v_size, q_size, gain):  # noqa: F811
    b = Batch8([150, 35], [nq, nq], 4, 2, d, d, dtype, 16, seed=21 + d, q_gain=q_size)
    rng = np.random.default_rng(33)
    for name, (least, most), size in (("k", k_bytes, k_size), ("v", v_bytes, v_size)):
        codes, byte = getattr(b, name + "_pages"), getattr(b, name + "_scales")
        new, new_byte = _coded(rng, codes.shape, size, least, most)
        used = byte != 255
        codes[used], byte[used] = new[used], new_byte[used]
    b.requantised()
    scale = gain / (k_size * q_size * math.sqrt(d))
    y, L, status = _attend(ex, b, "causal", 0, scale)
    assert status == 0
    _check_at(path, b, y, L, scale, "causal", -round(math.log2(v_size)))


# The 256-row kernel's operands are the rows themselves, as bf16 numbers.
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("k_bytes,k_size,v_bytes,v_size,q_size", [
    ((240, 246), 2.0 ** 118, (240, 246), 2.0 ** 116, 2.0 ** -116),
    ((3, 6), 2.0 ** -122, (3, 6), 2.0 ** -118, 2.0 ** 118),
    ((3, 5), 2.0 ** -128, (3, 5), 2.0 ** -122, 2.0 ** 122)])  # keys below 2^-126
def test_bytes_of_the_tall_tiles(ex, d, page, k_bytes, k_size, v_bytes, v_size, q_size):  # noqa: F811
    b = Batch8([150, 45], [40, 40], 4, 2, d, d, "bf16", page, seed=27 + d, q_gain=q_size)
    rng = np.random.default_rng(35)
    for name, (least, most), size in (("k", k_bytes, k_size), ("v", v_bytes, v_size)):
        codes, byte = getattr(b, name + "_pages"), getattr(b, name + "_scales")
        new, new_byte = _coded(rng, codes.shape, size, least, most)
        used = byte != 255
        codes[used], byte[used] = new[used], new_byte[used]
    b.requantised()
    scale = 1.0 / (k_size * q_size * math.sqrt(d))
    y, L, status = _attend(ex, b, "causal", 0, scale)
    assert status == 0
    _check_at("auto", b, y, L, scale, "causal", -round(math.log2(v_size)))

"""Append into 8-bit pages of pairs that do not stay finite: an infinity, a NaN, or a rotation beyond
fp32 in either entry makes both NaN, whatever form the pairs have, and neither counts for the row's
exponent."""
import numpy as np
import pytest
import torch

from e4m3_inputs import Batch8
from oracle import e4m3
from oracle import paged as oracle
from paged_inputs import DT

pytestmark = pytest.mark.gpu

MOST = float(np.finfo(np.float32).max)
# (d, pairs, interleaved): halves, neighbours, halves that eight columns do not reach; 16 lanes a row.
FORMS = [(64, 32, False), (64, 32, True), (128, 48, False), (64, 13, False), (80, 20, False), (80, 21, True),
         (16, 3, False), (256, 100, False), (256, 64, False), (256, 90, True)]


def _rows(rng, n, kv, d, pairs, inter, turns, dt):
    """Keys [n][kv][d] of moderate size, with a few pairs of each row as the docstring says: they turn to
    1.1 to 1.3 times the largest fp32 number and to something smaller, or hold an infinity or a NaN.  A fifth of the
    rows has a pair of that size that stays finite."""
    x = rng.standard_normal((n, kv, d)) * 2.0 ** rng.integers(-30, 31, (n, kv, 1))
    for i in range(n):
        for h in range(kv):
            for f in rng.choice(pairs, min(3, pairs), replace=False):
                a, b = (2 * f, 2 * f + 1) if inter else (f, f + pairs)
                if rng.integers(2):
                    a, b = b, a
                kind = (i + int(f)) % 6
                if kind < 4:  # x' = c x - s y, y' = c y + s x
                    c, s = np.cos(turns[f]), np.sin(turns[f])
                    big, other = rng.uniform(1.1, 1.3) * MOST * rng.choice([-1, 1]), (0.0, 1.0, 1e33, 1e38)[kind]
                    big *= 0.7 if i % 5 == 0 and kind < 3 else 1
                    big, other = (big, other) if rng.integers(2) else (other, big)
                    first, second = (2 * f, 2 * f + 1) if inter else (f, f + pairs)
                    x[i, h, first], x[i, h, second] = c * big + s * other, c * other - s * big
                else:
                    x[i, h, a] = (np.inf, np.nan)[kind - 4] * rng.choice([-1, 1])
    return torch.from_numpy(x).to(dt)


def _rotated(row, pos, inv, inter):
    """In float64, pairs that are not finite in fp32 NaN."""
    with np.errstate(invalid="ignore"):
        y = oracle.rotate(row, pos, inv, inter)
        r = len(inv)
        for f in range(r):
            a, b = (2 * f, 2 * f + 1) if inter else (f, f + r)
            pair = np.abs(y[..., [a, b]])
            assert not ((pair > MOST * 0.99) & (pair < MOST * 1.01)).any()  # no case on the edge
            bad = ~(pair <= MOST).all(-1)
            y[bad, a] = y[bad, b] = np.nan
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,pairs,inter", FORMS)
def test_pairs_that_are_not_finite(d, pairs, inter, dtype):
    import exact_tiled_softmax_gb300 as ex
    n, kv, pos = 24, 3, 10
    b = Batch8([pos + 1] * n, [1] * n, 3, kv, d, d, dtype, 16, seed=d + pairs)
    rng = np.random.default_rng(d + pairs + inter)
    # A tenth of a radian a token and more, so that at position 10 no factor is above 0.75.
    inv = rng.uniform(0.0740, 0.0830, pairs).astype(np.float32)
    b.k_new = _rows(rng, n, kv, d, pairs, inter, pos * inv.astype(np.float64), DT[dtype])
    assert torch.isfinite(b.k_new.float()).float().mean() > 0.9
    b.v_new[0, 0, d - 1], b.v_new[1, 1, 0], b.v_new[2, 2, :] = np.inf, np.nan, -np.inf
    k, v, table, lens, starts, ks, vs = b.cache()
    kn, vn = b.dev("k_new", "v_new")
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    ex.append_paged(kn, vn, k, v, table, lens, q_starts=starts, inv_freq=torch.from_numpy(inv).cuda(),
                    interleaved=inter, ws=ws, k_scales=ks, v_scales=vs)
    assert ex.device_status(ws) == 0
    got = [t.view(torch.uint8).cpu().numpy() for t in (k, ks, v, vs)]
    hurt = 0
    for t in range(n):
        at, off = int(b.table[t, pos // 16]), pos % 16
        want = e4m3.quantise(_rotated(b.np(b.k_new[t]), pos, inv, inter)) + e4m3.quantise(b.np(b.v_new[t]))
        for name, x, y in zip(("k_pages", "k_scales", "v_pages", "v_scales"), got, want):
            x = x[at, :, off]
            if name.endswith("pages"):  # zeros of either sign, NaN of either sign
                x, y = (np.where(z & 0x7F == 0x7F, 0x7F, np.where(z == 0x80, 0, z)) for z in (x, y))
                hurt += int((y == 0x7F).sum())
            assert np.array_equal(x, y), (name, t, int((x != y).sum()))
    assert hurt > n * kv  # the pairs were there


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,pairs,inter", [(64, 5, True), (80, 21, True), (256, 90, True), (128, 48, True), (64, 13, False),
                                           (16, 3, False), (128, 48, False), (64, 0, False)])
def test_columns_that_pass_do_not_hurt_one_another(d, pairs, inter, dtype):
    """Behind the last pair each entry is by itself: infinities and NaN there become NaN, their neighbours stay."""
    import exact_tiled_softmax_gb300 as ex
    n, kv, pos = 40, 3, 10
    b = Batch8([pos + 1] * n, [1] * n, 3, kv, d, 16, dtype, 16, seed=d + pairs)
    rng = np.random.default_rng(d + pairs + inter)
    inv = rng.uniform(0.0740, 0.0830, pairs).astype(np.float32)
    x = b.np(b.k_new).copy()
    for i in range(n):
        for h in range(kv):
            x[i, h, rng.integers(2 * pairs, d, 3)] = (np.inf, np.nan, -np.inf)[i % 3]
    b.k_new = torch.from_numpy(x).to(DT[dtype])
    k, v, table, lens, starts, ks, vs = b.cache()
    kn, vn = b.dev("k_new", "v_new")
    ex.append_paged(kn, vn, k, v, table, lens, q_starts=starts, inv_freq=torch.from_numpy(inv).cuda() if pairs else None,
                    interleaved=inter, k_scales=ks, v_scales=vs)
    got, byte = k.view(torch.uint8).cpu().numpy(), ks.cpu().numpy()
    for t in range(n):
        at, off = int(b.table[t, pos // 16]), pos % 16
        codes, want = e4m3.quantise(_rotated(b.np(b.k_new[t]), pos, inv, inter))
        z, codes = (np.where(y & 0x7F == 0x7F, 0x7F, np.where(y == 0x80, 0, y)) for y in (got[at, :, off], codes))
        assert np.array_equal(byte[at, :, off], want) and np.array_equal(z, codes), (t, int((z != codes).sum()))

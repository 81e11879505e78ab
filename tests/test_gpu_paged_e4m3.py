"""GPU parity of the paged cache in 8 bits against the float64 oracle: append that quantises,
attention over pages, attention behind a shared prefix, and a run of the three together."""
import math

import numpy as np
import pytest
import torch

from e4m3_inputs import Batch8, small_weights, weight_bits
from oracle import e4m3
from oracle import paged as oracle
from paged_inputs import DT, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import exact_tiled_softmax_gb300 as mod
    mod.load_library()
    assert torch.cuda.is_available()
    return mod


@pytest.fixture(params=["auto", "simt"])
def path(ex, request):
    prev = ex.set_path(request.param)
    yield request.param
    ex.set_path(prev)


# ----------------------------------------------------------------------------- append
# (lens, nqs, H, kv, d, v, dtype, page, pairs, interleaved, offset, pad, with q, strided)
APPEND = [
    ([1], [1], 1, 1, 64, 64, "bf16", 16, 32, False, 0, 0, True, False),
    ([40, 7, 300], [1, 1, 1], 8, 2, 128, 128, "bf16", 16, 64, False, 0, 0, True, True),
    ([40, 7, 300, 9], [5, 7, 30, 0], 6, 2, 80, 96, "f32", 32, 20, True, 1000, 3, True, True),
    ([33, 34], [3, 4], 4, 4, 80, 64, "bf16", 8, 20, False, 0, 0, True, False),   # halves of 20 columns
    ([33, 34], [3, 4], 4, 4, 64, 64, "bf16", 4, 3, False, 5, 0, True, False),    # of 3
    ([33, 34], [3, 4], 4, 4, 64, 16, "f32", 1, 5, True, 0, 0, False, True),
    ([100], [100], 2, 1, 256, 256, "bf16", 64, 128, True, 0, 0, True, False),
    ([100, 60], [20, 1], 3, 1, 16, 208, "f32", 2, 0, False, 0, 1, True, False),  # not rotated
    ([100, 60], [50, 1], 3, 3, 112, 112, "bf16", 16, 16, False, 7, 1, True, False),  # columns that pass
    ([700], [500], 4, 2, 128, 96, "f32", 64, 64, False, 0, 0, True, False),
    ([900000], [2], 4, 2, 128, 128, "f32", 1024, 64, False, 100000, 0, True, False),
]


def _append(ex, b, pairs, inter, offset, q=None, k_new=None, v_new=None):
    """Device tensors after an append of the batch's new tokens, and the status."""
    inv = (10000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    k, v, table, lens, starts, ks, vs = b.cache()
    kn, vn = b.dev("k_new", "v_new")
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    out = None if q is None else torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    ex.append_paged(kn if k_new is None else k_new, vn if v_new is None else v_new, k, v, table, lens, q_starts=starts,
                    q=q, q_out=out, inv_freq=torch.from_numpy(inv).cuda() if pairs else None, interleaved=inter,
                    pos_offset=offset, ws=ws, k_scales=ks, v_scales=vs)
    status = ex.device_status(ws)
    return [t.view(torch.uint8).cpu().numpy() for t in (k, v, ks, vs)] + [out, status]


def _appended(b, inv, inter, offset):
    """The oracle's codes and bytes, and its rotated queries.  Pages hold their tokens' float64 values
    first, 7 anywhere else, and are then quantised row by row where a token was written."""
    mark = np.full(b.k_pages.shape, 7.0), np.full(b.v_pages.shape, 7.0)
    qo, kr, vr = oracle.append(b.np(b.k_new), b.np(b.v_new), *mark, b.table, b.lens, b.starts, b.np(b.q), inv, inter,
                               offset)
    out = []
    for x, codes, byte in ((kr, b.k_pages, b.k_scales), (vr, b.v_pages, b.v_scales)):
        written = ~(x == 7.0).all(-1)
        c, e = e4m3.quantise(x)
        out += [np.where(written[..., None], c, codes), np.where(written, e, byte)]
    return qo, out[0], out[2], out[1], out[3]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_append(ex, case):
    """Codes and bytes are those of 64-bit arithmetic, all of them; rows without a token stay."""
    lens, nqs, H, kv, d, v, dtype, page, pairs, inter, offset, pad, with_q, strided = case
    b = Batch8([min(n, 2000) for n in lens], nqs, H, kv, d, v, dtype, page, seed=APPEND.index(case) + 300, pad=pad)
    if max(lens) > 2000:  # a far position: its page alone is in the table
        b.lens = np.array(lens, dtype=np.int32)
        far = np.full((len(lens), -(-max(lens) // page)), -1, dtype=np.int32)
        far[:, -1] = 0
        b.table = far
    inv = (10000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    q, kn, vn = b.dev("q", "k_new", "v_new")
    if strided:
        wide = torch.zeros(b.T, H * d + kv * (d + v) + 8, dtype=q.dtype, device="cuda")
        wide[:, :H * d], wide[:, H * d:H * d + kv * d] = q.reshape(b.T, -1), kn.reshape(b.T, -1)
        wide[:, H * d + kv * d:H * d + kv * (d + v)] = vn.reshape(b.T, -1)
        q = wide[:, :H * d].view(b.T, H, d)
        kn = wide[:, H * d:H * d + kv * d].view(b.T, kv, d)
        vn = wide[:, H * d + kv * d:H * d + kv * (d + v)].view(b.T, kv, v)
    *got, out, status = _append(ex, b, pairs, inter, offset, q if with_q else None, kn, vn)
    assert status == 0
    qo, *want = _appended(b, inv, inter, offset)
    for name, x, y in zip(("k_pages", "v_pages", "k_scales", "v_scales"), got, want):
        x, y = (np.where(t == 0x80, 0, t) if name.endswith("pages") else t for t in (x, y))  # zeros of either sign
        assert np.array_equal(x, y), (name, int((x != y).sum()))
    if with_q:
        n = int(b.starts[-1])
        # As for a cache of the inputs' type: 2^-20 of the pair's size, then one rounding.
        size = 2 * float(b.q.double().abs().max())
        eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        tol = 2.0 ** -20 * size + eps * (np.abs(qo[:n]) + 2.0 ** -20 * size)
        assert (np.abs(out[:n].double().cpu().numpy() - qo[:n]) <= tol).all()
        assert (out[n:] == 7).all()


@pytest.mark.parametrize("pairs,inter", [(0, False), (32, False), (32, True), (5, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_on_the_borders(ex, dtype, pairs, inter):
    """Entries that lie on a border of the rounding exactly (ties to even), rows whose largest entry
    is 448 times a power of two and one step above, of any size, zeros, a single entry; at position 0
    a rotation leaves them as they are."""
    n, d = 24, 64
    b = Batch8([1] * n, [1] * n, 1, 1, d, d, dtype, 16, seed=7)
    rng = np.random.default_rng(3)
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    x = np.zeros((n, d))
    for i in range(n):
        x[i] = rng.choice(e4m3.BORDERS, d) * rng.choice([-1, 1], d)
        x[i, rng.integers(d)] = [448, 448 * (1 + step), 447, 256][i % 4]
        big = {0: 0, 1: 100, 2: -100, 3: 7}[i // 4 % 4]
        x[i] *= 2.0 ** big
    x[5], x[6, 1:], x[7] = 0, 0, -x[4]
    x[8] = 2.0 ** -130 if dtype == "f32" else 2.0 ** -126  # nothing but the smallest
    b.k_new = torch.from_numpy(x).to(DT[dtype])[:, None]
    b.v_new = torch.from_numpy(x[::-1].copy()).to(DT[dtype])[:, None]
    inv = (10000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    *got, _, status = _append(ex, b, pairs, inter, 0)
    assert status == 0
    _, *want = _appended(b, inv, inter, 0)
    for x, y in zip(got[:2], want[:2]):
        assert np.array_equal(np.where(x == 0x80, 0, x), np.where(y == 0x80, 0, y))
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])


@pytest.mark.parametrize("offset", [0, 11])
@pytest.mark.parametrize("pairs,inter", [(32, False), (32, True), (13, False), (21, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_rows_whose_largest_lies_on_the_border(ex, dtype, pairs, inter, offset):
    """Of columns that pass, of a pair that its rotation brings to 448 times a power of two within a
    rounding, and of both, at the first position and behind it."""
    n, d = 48, 128
    b = Batch8([n], [n], 1, 3, d, d, dtype, 16, seed=23)
    rng = np.random.default_rng(29)
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    inv = (10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    x = rng.uniform(-300, 300, (n, 3, d))
    for i in range(n):
        for h in range(3):
            f = int(rng.integers(pairs))
            turn = float(i + offset) * float(inv[f])
            at = (2 * f, 2 * f + 1) if inter else (f, f + pairs)
            if h != 1:  # x cos - y sin = 448
                x[i, h, at[0]], x[i, h, at[1]] = 448 * math.cos(turn), -448 * math.sin(turn)
            if h != 0:
                x[i, h, rng.integers(2 * pairs, d)] = [448, -448 * (1 + step), 448 * (1 - step / 2)][i % 3]
            x[i, h] *= 2.0 ** int(rng.integers(-20, 20))
    b.k_new = torch.from_numpy(x).to(DT[dtype])
    *got, _, status = _append(ex, b, pairs, inter, offset)
    assert status == 0
    _, *want = _appended(b, inv, inter, offset)
    for x, y in zip(got[:2], want[:2]):
        assert np.array_equal(np.where(x == 0x80, 0, x), np.where(y == 0x80, 0, y))
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])


@pytest.mark.parametrize("form", [(64, False), (64, True), (20, False)])
def test_append_keeps_its_side_of_every_border(ex, form):
    """Many rotated rows: an entry in some 2^16 lies nearer to a border than fp32 can tell."""
    pairs, inter = form
    n = 4000
    b = Batch8([n], [n], 1, 4, 128, 128, "f32", 64, seed=pairs + inter)
    inv = (10000.0 ** (-np.arange(pairs) / pairs)).astype(np.float32)
    *got, _, status = _append(ex, b, pairs, inter, 0)
    assert status == 0
    _, *want = _appended(b, inv, inter, 0)
    for x, y in zip(got, want):
        assert np.array_equal(x, y), int((x != y).sum())


@pytest.mark.parametrize("pairs", [0, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_of_entries_that_are_not_finite(ex, dtype, pairs):
    """They become NaN (and so does their pair's other entry where it is rotated), the row's exponent
    is that of its finite entries; other rows are what they are."""
    b = Batch8([40, 9], [3, 2], 2, 2, 64, 64, dtype, 16, seed=9)
    want = _append(ex, b, pairs, False, 5)
    b.k_new[1, 0, 3], b.k_new[2, 1, 40], b.v_new[1, 1, 63] = math.inf, math.nan, -math.inf
    b.v_new[3, 0, :] = math.nan
    got = _append(ex, b, pairs, False, 5)
    hurt = {(1, 0): {3, 35} if pairs else {3}, (2, 1): {8, 40} if pairs else {40}}
    for t in range(b.T):
        s = 0 if t < 3 else 1
        pos = int(b.lens[s]) - (3, 2)[s] + t - int(b.starts[s])
        at = int(b.table[s, pos // 16]), pos % 16
        for h in range(2):
            k, ke = got[0][at[0], h, at[1]], got[2][at[0], h, at[1]]
            bad = hurt.get((t, h), set())
            assert set(np.flatnonzero(k & 0x7F == 0x7F)) == bad
            keep = [c for c in range(64) if c not in bad]
            if ke == want[2][at[0], h, at[1]]:
                assert np.array_equal(k[keep], want[0][at[0], h, at[1]][keep])
            else:
                assert bad
            ve, v = got[3][at[0], h, at[1]], got[1][at[0], h, at[1]]
            nan = np.flatnonzero(v & 0x7F == 0x7F)
            assert list(nan) == (list(range(64)) if (t, h) == (3, 0) else [63] if (t, h) == (1, 1) else [])
            assert ve == 0 if (t, h) == (3, 0) else ve > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs,inter", [(32, False), (32, True), (20, False), (13, False)])
def test_append_rotates_q_in_place(ex, dtype, pairs, inter):
    b = Batch8([400, 9], [300, 2], 6, 2, 64, 64, dtype, 16, seed=1)
    k, v, table, lens, starts, ks, vs = b.cache()
    q, kn, vn = b.dev("q", "k_new", "v_new")
    inv = torch.pow(10000.0, -torch.arange(pairs, device="cuda") / pairs).float()
    kw = dict(q_starts=starts, inv_freq=inv, interleaved=inter, k_scales=ks, v_scales=vs)
    want = ex.append_paged(kn, vn, k, v, table, lens, q=q, **kw)
    got = ex.append_paged(kn, vn, k, v, table, lens, q=q, q_out=q, **kw)
    assert got is q and torch.equal(got, want)


def test_append_without_a_place(ex):
    """Tokens before position 0, behind the table, or on a page outside the pool: nothing of
    theirs is written, the others' are, and the status word says so."""
    for lens, edit in (([1, 20], None), ([20, 20], (0, 1, -7)), ([20, 20], (0, 1, 99)), ([900, 20], None)):
        b = Batch8([20, 20], [3, 2], 2, 1, 64, 64, "bf16", 16, seed=6)
        b.lens = np.array(lens, dtype=np.int32)
        if edit:
            b.table[edit[0], edit[1]] = edit[2]
        *got, _, status = _append(ex, b, 0, False, 0)
        assert status == 8
        _, *want = _appended(b, (), False, 0)
        for x, y in zip(got, want):
            assert np.array_equal(x, y)


# ------------------------------------------------------------------------- attention
# (lens, nqs, H, kv, d, v, dtype, page, mask, window, pad)
ATTEND = [
    ([1], [1], 1, 1, 64, 64, "bf16", 16, "causal", 0, 0),
    ([33], [1], 8, 2, 128, 128, "bf16", 16, "causal", 0, 0),
    ([1000, 1, 17, 640], [1, 1, 1, 1], 8, 8, 128, 128, "bf16", 64, "none", 0, 0),
    ([129, 777, 2], [3, 5, 2], 6, 2, 64, 64, "bf16", 32, "causal", 0, 2),       # a group of 3
    ([300, 40, 512], [4, 1, 7], 7, 1, 128, 96, "bf16", 8, "window", 100, 3),    # a group of 7, d != v
    ([2047], [4], 32, 8, 128, 128, "bf16", 16, "causal", 0, 0),
    ([5, 0, 90, 64], [1, 0, 2, 0], 4, 4, 80, 96, "f32", 16, "causal", 0, 0),    # sequences without tokens
    ([700, 1300], [2, 1], 16, 2, 128, 128, "f32", 32, "window", 333, 0),
    ([61, 200], [3, 1], 4, 1, 64, 128, "f32", 4, "none", 0, 1),
    ([1, 2, 3, 4, 5], [1, 1, 1, 1, 1], 2, 1, 16, 16, "bf16", 1, "causal", 0, 0),  # pages of one key
    ([400], [1], 4, 4, 256, 256, "bf16", 16, "causal", 0, 0),
    ([150, 90], [3, 6], 4, 2, 192, 128, "f32", 16, "window", 64, 0),
    ([300], [70], 8, 2, 128, 128, "bf16", 64, "causal", 0, 0),                  # a chunk of a prompt
    ([257, 130], [257, 130], 4, 2, 64, 64, "bf16", 16, "causal", 0, 0),         # whole prompts
    ([90, 200], [33, 50], 3, 3, 112, 64, "f32", 128, "window", 20, 0),
    ([640, 5], [20, 5], 8, 1, 96, 96, "bf16", 1024, "none", 0, 5),
    ([500, 31, 32, 33, 63, 64, 65], [1] * 7, 2, 2, 128, 128, "bf16", 8, "causal", 0, 0),
    ([500, 31, 32, 33, 63, 64, 65], [2] * 7, 6, 2, 96, 112, "f32", 8, "causal", 0, 0),
]


def _attend(ex, b, mask, window, scale, **kw):
    k, v, table, lens, starts, ks, vs = b.cache()
    q, = b.dev("q")
    y = torch.full((b.T, b.H, v.shape[3]), 7.0, dtype=q.dtype, device="cuda")
    L = torch.full((b.T, b.H), 7.0, dtype=torch.float32, device="cuda")
    ws = torch.full((ex.paged_workspace_size(ex.paged_shape(q, k, v, table)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    y, L = ex.fwd_paged(q, k, v, table, lens, scale, mask, window, q_starts=starts, y=y, L=L, ws=ws, k_scales=ks,
                        v_scales=vs, **kw)
    return y, L, ex.device_status(ws)


def _check(path, b, y, L, scale, mask, window=0, n=None, prefix=None, extra=0.0, rows=None):
    n = int(b.lens.max()) if n is None else n
    with np.errstate(invalid="ignore"):
        ref = oracle.attend(b.np(b.q), b.k64, b.v64, b.table, np.clip(b.lens, 0, None), b.starts, scale, mask, window,
                            prefix)
    W = b.largest_weight(ref, scale, mask, window, prefix)
    d, v = b.k64.shape[3], b.v64.shape[3]
    if rows is None:  # a prefix's pass takes every token as one sequence's
        rows = (b.T if prefix else -(-b.T // len(b.lens))) * (b.H // b.kv)
    keys = n + (prefix[1] if prefix else 0)
    # The smallest weights' own term, as a part of A (which it may exceed in a column of small numbers).
    Y, Lr, A, D = ref
    bits = weight_bits(path, b.dtype, d, v, b.page, rows, scale)
    A = A + small_weights(W, keys) * 2.0 ** bits
    check_attention(b.dtype, y, L, (Y, Lr, A, D), d, keys, bits, extra=extra)


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention_over_pages(ex, path, case):
    lens, nqs, H, kv, d, v, dtype, page, mask, window, pad = case
    b = Batch8(lens, nqs, H, kv, d, v, dtype, page, seed=ATTEND.index(case) + 100, pad=pad)
    scale = 0.25 / math.sqrt(d)  # the rows' sizes differ
    y, L, status = _attend(ex, b, mask, window, scale)
    assert status == 0
    _check(path, b, y, L, scale, mask, window)
    if pad:  # rows behind the last sequence stay as they were
        assert (y[-pad:] == 7).all() and (L[-pad:] == 7).all()


# Rows of a key head around the edges of a 128-row half and of a 256-row tile, with
# prompts before and behind 128-key blocks.
@pytest.mark.parametrize("nqs,G", [([127], 1), ([128], 1), ([129, 3], 1), ([256, 1, 200], 1), ([257], 1),
                                   ([86, 85], 3), ([37, 74, 1], 7)])
@pytest.mark.parametrize("page,d,v,mask,window", [(8, 128, 128, "causal", 0), (64, 64, 64, "window", 150),
                                                  (128, 80, 112, "causal", 0), (256, 128, 64, "none", 0)])
def test_many_rows(ex, nqs, G, page, d, v, mask, window):
    lens = [n + x for n, x in zip(nqs, (130, 0, 400))]
    b = Batch8(lens, nqs, 2 * G, 2, d, v, "bf16", page, seed=len(nqs) + G + page)
    y, L, status = _attend(ex, b, mask, window, 0.03)
    assert status == 0
    _check("auto", b, y, L, 0.03, mask, window)


@pytest.mark.parametrize("nqs", [[3, 4], [4, 1]])
def test_two_row_tiles_over_many_keys(ex, nqs):
    """17 to 32 bf16 rows to a key head stay on the 16-row tiles where the tables hold many keys."""
    b = Batch8([8200, 300], nqs, 64, 8, 64, 64, "bf16", 32, seed=15)
    y, L, status = _attend(ex, b, "causal", 0, 0.03)
    assert status == 0
    _check("auto", b, y, L, 0.03, "causal", rows=16)


@pytest.mark.parametrize("case", [([300, 40, 512], [1, 1, 1], 32, 8, "bf16"), ([2000, 9], [2, 3], 8, 1, "bf16"),
                                  ([700, 90], [60, 2], 8, 2, "bf16"), ([300, 900], [2, 1], 8, 2, "f32")], ids=str)
def test_calls_repeat_themselves(ex, path, case):
    """The same bits whatever the workspace held, also behind a prefix."""
    lens, nqs, H, kv, dtype = case
    b = Batch8(lens, nqs, H, kv, 128, 128, dtype, 16, seed=16, prefix=2500)
    k, v, table, ln, starts, ks, vs = b.cache()
    q, pt = b.dev("q", "prefix_table")
    kw = dict(q_starts=starts, k_scales=ks, v_scales=vs)
    size = ex.prefix_workspace_size(ex.paged_shape(q, k, v, table))
    want = None
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = ex.fwd_paged(q, k, v, table, ln, 0.05, "causal", ws=ws, **kw)
        got += ex.fwd_prefix(q, k, v, pt, 2500, table, ln, 0.05, "causal", ws=ws, **kw)
        want = want or got
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(ex, path, dtype, scale):
    b = Batch8([70, 300], [2, 50], 8, 2, 64, 64, dtype, 16, seed=3)
    y, L, status = _attend(ex, b, "causal", 0, scale)
    assert status == 0
    _check(path, b, y, L, scale, "causal")


@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 40), ("f32", 2)])
@pytest.mark.parametrize("k_up,v_up,q_up", [(60, 0, -60), (-60, 90, 60), (0, -110, 0), (-105, 115, 90), (110, 3, -110)])
def test_exponents_of_any_size(ex, path, dtype, nq, k_up, v_up, q_up):
    """Rows of any size: a row's exponent comes out of both products, and a query row's too."""
    b = Batch8([200, 33], [nq, nq], 4, 2, 64, 64, dtype, 16, seed=13, q_gain=2.0 ** q_up)
    for name, up in (("k", k_up), ("v", v_up)):
        s = getattr(b, name + "_scales")
        used = s != 255
        s[used] = np.clip(s[used].astype(int) + up, 1, 246).astype(np.uint8)
    b.requantised()
    scale = 0.06 * 2.0 ** (-k_up - q_up)
    y, L, status = _attend(ex, b, "causal", 0, scale)
    assert status == (5 if nq > 33 else 0)  # tokens before every key
    _check(path, b, y, L, scale, "causal")


@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 40), ("f32", 2)])
def test_values_of_very_unequal_rows(ex, path, dtype, nq):
    """One key whose value is 2^40 times the others' and whose score is far below them: the others'
    weights keep their bits.  And rows of zeros (byte 0) among them."""
    b = Batch8([300], [nq], 2, 1, 64, 64, dtype, 16, seed=14)
    at = int(b.table[0, 2]), 0, 5
    b.v_scales[at] += 40
    b.k_pages[at], b.k_scales[at] = (x[0] for x in e4m3.quantise(-b.np(b.q[-1, 0])[None] * 4))
    z = int(b.table[0, 3]), 0, 7
    b.k_pages[z], b.k_scales[z], b.v_pages[z], b.v_scales[z] = 0, 0, 0, 0
    b.requantised()
    y, L, status = _attend(ex, b, "causal", 0, 0.125)
    assert status == 0
    _check(path, b, y, L, 0.125, "causal")


@pytest.mark.parametrize("dtype,G,nq", [("bf16", 1, 1), ("bf16", 4, 1), ("bf16", 2, 40), ("f32", 4, 2)])
def test_rows_without_keys(ex, path, dtype, G, nq):
    """A sequence of no cached keys, and one with fewer keys than tokens."""
    b = Batch8([0, 2, 50, 1], [nq, nq + 2, nq, nq], 2 * G, 2, 64, 64, dtype, 16, seed=5)
    y, L, status = _attend(ex, b, "causal", 0, 0.05)
    assert status == 5
    _check(path, b, y, L, 0.05, "causal")
    assert np.isneginf(L.cpu().numpy()[:nq]).all()


@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 3), ("bf16", 40), ("f32", 2)])
def test_pages_outside_the_pool_are_left_out(ex, path, dtype, nq):
    b = Batch8([200, 90], [nq, nq], 4, 2, 64, 64, dtype, 16, seed=9)
    num = b.k_pages.shape[0]
    b.table[0, 3], b.table[0, 5], b.table[1, 0] = -1, num, 2 ** 31 - 1
    y, L, status = _attend(ex, b, "causal", 0, 0.05)
    assert status == 8
    _check(path, b, y, L, 0.05, "causal")
    b = Batch8([200, 90], [nq, nq], 4, 2, 64, 64, dtype, 16, seed=9)
    b.table[0, :4] = -5
    y, L, status = _attend(ex, b, "window", 70, 0.05)
    assert status == 0
    _check(path, b, y, L, 0.05, "window", 70)


def test_numbers_that_do_not_fit_are_clamped(ex, path):
    b = Batch8([40, 60], [2, 2], 2, 1, 64, 64, "bf16", 16, seed=2)
    b.lens[0] = -3
    y, L, status = _attend(ex, b, "none", 0, 0.05)
    assert status == 8
    _check(path, b, y, L, 0.05, "none", n=60)
    b = Batch8([40, 60], [2, 2], 2, 1, 64, 64, "bf16", 16, seed=2)
    b.starts[2] = 1000  # behind the tokens
    y, L, status = _attend(ex, b, "none", 0, 0.05)
    assert status == 8
    b.starts[2] = 4
    _check(path, b, y, L, 0.05, "none")


@pytest.mark.parametrize("dtype,nq,G", [("bf16", 1, 2), ("bf16", 3, 4), ("bf16", 40, 2), ("f32", 3, 2)])
def test_keys_before_every_window_leave_no_trace(ex, path, dtype, nq, G):
    """Keys and values that no token's window reaches hold NaN, under bytes of every kind."""
    n, w = 300, 70
    b = Batch8([n, 50], [nq, nq], 2 * G, 2, 64, 96, dtype, 32, seed=18)
    for j in range(n - nq + 1 - w):
        at = int(b.table[0, j // 32]), slice(None), j % 32
        b.k_pages[at], b.v_pages[at] = (0x7F, 0xFF, 0x7E)[j % 3], (0xFF, 0x7F, 0xFE)[j % 3]
        b.k_scales[at], b.v_scales[at] = (255, 0, 254)[j % 3], (254, 255, 0)[j % 3]
    b.requantised()
    y, L, status = _attend(ex, b, "window", w, 0.05)
    assert status == 0
    _check(path, b, y, L, 0.05, "window", w, n=w)


@pytest.mark.parametrize("dtype,nq,n", [("bf16", 1, 40), ("bf16", 2, 2500), ("bf16", 40, 300), ("f32", 2, 700)])
def test_entries_that_are_not_numbers_stay_where_they_reach(ex, path, dtype, nq, n):
    """A NaN value reaches its column of the rows that allow its key, a NaN key all of them and
    no others, a NaN query its own row."""
    b = Batch8([n, 5 + nq, n], [nq] * 3, 4, 2, 64, 96, dtype, 16, seed=19)
    y0, L0, _ = _attend(ex, b, "causal", 0, 0.05)
    at = int(b.table[0, 1]), 1, 3  # key 19 of the first sequence, key head 1
    here = torch.zeros(b.T, 4, dtype=torch.bool, device="cuda")
    here[:nq, 2:] = True
    kept = b.v_pages[at].copy()
    b.v_pages[at][95] = 0x7F
    y, L, status = _attend(ex, b, "causal", 0, 0.05)
    assert status == 0 and torch.equal(L, L0)
    assert torch.isnan(y[..., 95][here]).all()
    assert torch.equal(y[..., :95], y0[..., :95]) and torch.equal(y[~here], y0[~here])
    b.v_pages[at] = kept
    kept = b.k_pages[at].copy()
    b.k_pages[at][0] = 0xFF
    y, L, status = _attend(ex, b, "causal", 0, 0.05)
    assert torch.isnan(y[here]).all() and torch.isnan(L[here]).all()
    assert torch.equal(y[~here], y0[~here]) and torch.equal(L[~here], L0[~here])
    b.k_pages[at] = kept
    b.q[0, 1, 63] = math.nan
    here[:] = False
    here[0, 1] = True
    y, L, status = _attend(ex, b, "causal", 0, 0.05)
    assert torch.isnan(y[here]).all() and torch.isnan(L[here]).all()
    assert torch.equal(y[~here], y0[~here]) and torch.equal(L[~here], L0[~here])


@pytest.mark.parametrize("dtype,d,v,nq,page", [("bf16", 16, 16, 1, 8), ("bf16", 32, 128, 5, 16), ("bf16", 128, 16, 60, 64),
                                               ("bf16", 48, 48, 60, 8), ("f32", 16, 128, 3, 32), ("f32", 112, 112, 9, 8),
                                               ("bf16", 64, 64, 40, 4), ("f32", 64, 32, 3, 2), ("bf16", 144, 32, 2, 16),
                                               ("f32", 32, 240, 1, 16), ("bf16", 96, 96, 2, 64), ("f32", 80, 96, 2, 32),
                                               ("bf16", 96, 80, 7, 1024), ("bf16", 256, 256, 3, 32), ("f32", 208, 256, 9, 64),
                                               ("f32", 256, 256, 2, 128), ("bf16", 256, 144, 20, 8), ("bf16", 128, 128, 5, 1),
                                               ("f32", 96, 64, 1, 2), ("bf16", 256, 256, 2, 2), ("bf16", 64, 64, 1, 4)])
def test_widths_between(ex, path, dtype, d, v, nq, page):
    b = Batch8([700, nq, 90], [nq, nq, nq], 4, 2, d, v, dtype, page, seed=d + v + nq)
    y, L, status = _attend(ex, b, "causal", 0, 0.03)
    assert status == 0
    _check(path, b, y, L, 0.03, "causal")


@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("f32", 2), ("bf16", 30)])
def test_large_batches(ex, path, dtype, nq, prefix):
    """The largest batch, most sequences short, some without tokens or keys."""
    B = 1024 if nq < 30 else 60
    rng = np.random.default_rng(B)
    nqs = [0 if x == 0 else int(rng.integers(1, nq + 1)) for x in rng.integers(0, 5, B)]
    lens = [int(rng.integers(0, 40)) + q for q in nqs]
    b = Batch8(lens, nqs, 2, 1, 64, 64, dtype, 16, seed=B, prefix=prefix)
    if prefix:
        y, L, status = _behind(ex, b, prefix, "causal", 0.05)
    else:
        y, L, status = _attend(ex, b, "causal", 0, 0.05)
    assert status == 0
    _check(path, b, y, L, 0.05, "causal", prefix=(b.prefix_table, prefix) if prefix else None, extra=2.0 ** -20)


def test_equal_tokens_without_q_starts(ex, path):
    b = Batch8([70, 33, 128], [2, 2, 2], 4, 2, 128, 128, "bf16", 16, seed=21)
    k, v, table, lens, starts, ks, vs = b.cache()
    q, = b.dev("q")
    y0, L0 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal", q_starts=starts, k_scales=ks, v_scales=vs)
    y1, L1 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal", k_scales=ks.view(torch.float8_e8m0fnu), v_scales=vs)
    assert torch.equal(y0, y1) and torch.equal(L0, L1)


def test_queries_that_are_columns_of_a_projection(ex, path):
    b = Batch8([70, 33], [1, 2], 4, 2, 64, 64, "bf16", 16, seed=22)
    k, v, table, lens, starts, ks, vs = b.cache()
    q, = b.dev("q")
    wide = torch.randn(b.T, 4 * 64 + 72, device="cuda").to(q.dtype)
    wide[:, 8:8 + 256] = q.reshape(b.T, 256)
    kw = dict(q_starts=starts, k_scales=ks, v_scales=vs)
    y0, L0 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal", **kw)
    y1, L1 = ex.fwd_paged(wide[:, 8:8 + 256].view(b.T, 4, 64), k, v, table, lens, 0.1, "causal", **kw)
    assert torch.equal(y0, y1) and torch.equal(L0, L1)


@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 40), ("f32", 1)])
def test_pool_beyond_32_bit_offsets(ex, path, dtype, nq):
    """Pages at the far end of a pool of more than 2^32 bytes."""
    kv, page, d = 8, 64, 128
    num = (1 << 32) // (kv * page * d) + 40
    b = Batch8([500], [nq], 16, kv, d, d, dtype, page, seed=31)
    k, v, t0, lens, starts, ks, vs = b.cache()
    far = [torch.empty(num, *t.shape[1:], dtype=torch.uint8, device="cuda") for t in (k, v, ks, vs)]
    table = b.table.copy()
    for i, at in enumerate(b.table[0, :8]):
        for x, y in zip(far, (k, v, ks, vs)):
            x[num - 1 - i] = y.view(torch.uint8)[int(at)]
        table[0, i] = num - 1 - i
    q, kn, vn = b.dev("q", "k_new", "v_new")
    table = torch.from_numpy(table).cuda()
    pages = [x.view(torch.float8_e4m3fn) for x in far[:2]]
    kw = dict(k_scales=far[2], v_scales=far[3])
    y, L = ex.fwd_paged(q, *pages, table, lens, 0.1, "causal", **kw)
    y0, L0 = ex.fwd_paged(q, k, v, t0, lens, 0.1, "causal", k_scales=ks, v_scales=vs)
    assert torch.equal(y, y0) and torch.equal(L, L0)
    ex.append_paged(kn, vn, *pages, table, lens, **kw)
    ex.append_paged(kn, vn, k, v, t0, lens, k_scales=ks, v_scales=vs)
    for i, at in enumerate(b.table[0, :8]):
        for x, y in zip(far, (k, v, ks, vs)):
            assert torch.equal(x[num - 1 - i], y.view(torch.uint8)[int(at)])


# ------------------------------------------------------------------------ shared prefix
# (prefix, lens, nqs, H, kv, d, v, dtype, page, mask, pad)
PREFIX = [
    (1, [1], [1], 1, 1, 64, 64, "bf16", 16, "causal", 0),
    (300, [5, 1, 40], [1, 1, 1], 8, 2, 128, 128, "bf16", 16, "causal", 0),
    (1000, [3, 70, 1, 0, 9], [3, 5, 1, 0, 2], 6, 2, 64, 64, "bf16", 64, "causal", 2),
    (513, [40, 80], [2, 1], 4, 1, 80, 96, "f32", 32, "none", 0),
    (90, [12] * 40, [1] * 40, 16, 2, 128, 128, "bf16", 16, "causal", 0),
    (257, [20, 30], [20, 30], 8, 2, 64, 128, "bf16", 32, "none", 1),
    (130, [7, 9], [1, 1], 2, 2, 208, 112, "bf16", 16, "causal", 0),
    (2000, [1, 1], [1, 1], 4, 4, 128, 128, "f32", 64, "causal", 0),
    (0, [30, 5], [2, 1], 4, 2, 64, 64, "bf16", 16, "causal", 0),
    # Long enough for tall tiles in a launch of their own.
    (4001, [40, 1, 90, 17] * 4, [1, 1, 1, 0] + [1] * 12, 32, 8, 128, 128, "bf16", 64, "causal", 1),
    (8003, [40, 1, 90, 17] * 4, [1, 1, 1, 0] + [1] * 12, 32, 8, 128, 128, "bf16", 8, "causal", 0),
]


def _behind(ex, b, prefix, mask, scale):
    k, v, table, lens, starts, ks, vs = b.cache()
    q, pt = b.dev("q", "prefix_table")
    y = torch.full((b.T, b.H, v.shape[3]), 7.0, dtype=q.dtype, device="cuda")
    L = torch.full((b.T, b.H), 7.0, device="cuda")
    ws = torch.full((ex.prefix_workspace_size(ex.paged_shape(q, k, v, table)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    ex.fwd_prefix(q, k, v, pt, prefix, table, lens, scale, mask, q_starts=starts, y=y, L=L, ws=ws, k_scales=ks,
                  v_scales=vs)
    return y, L, ex.device_status(ws)


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention_behind_a_shared_prefix(ex, path, case):
    prefix, lens, nqs, H, kv, d, v, dtype, page, mask, pad = case
    b = Batch8(lens, nqs, H, kv, d, v, dtype, page, seed=PREFIX.index(case) + 200, pad=pad, prefix=prefix)
    if pad:
        b.q[-pad:] = float("nan")
    scale = 0.25 / math.sqrt(d)
    y, L, status = _behind(ex, b, prefix, mask, scale)
    assert status == 0
    _check(path, b, y, L, scale, mask, prefix=(b.prefix_table, prefix), extra=2.0 ** -20)
    if pad:
        assert (y[-pad:] == 7).all() and (L[-pad:] == 7).all()


def test_a_sequence_without_own_keys_still_has_the_prefix(ex, path):
    b = Batch8([0, 1], [2, 3], 4, 2, 64, 64, "bf16", 16, seed=8, prefix=50)
    for mask in ("none", "causal"):
        y, L, status = _behind(ex, b, 50, mask, 0.05)
        assert status == 0
        _check(path, b, y, L, 0.05, mask, prefix=(b.prefix_table, 50), extra=2.0 ** -20)
    b.prefix_table[1] = -1
    y, L, status = _behind(ex, b, 50, "none", 0.05)
    assert status == 8
    _check(path, b, y, L, 0.05, "none", prefix=(b.prefix_table, 50), extra=2.0 ** -20)


# ----------------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,G,widths", [("bf16", 4, (128, 128)), ("f32", 1, (80, 96)), ("bf16", 16, (64, 64))])
def test_a_run_of_the_three(ex, path, dtype, G, widths):
    """A server's program: a common prompt appended, each request's own tokens behind it, then
    decode steps, each an append and an attention behind the prefix, against the oracle over the rows
    that it rotates and quantises itself."""
    d, v = widths
    kv, page, P, B, steps = 2, 16, 75, 3, 4
    H, dt = kv * G, DT[dtype]
    g = torch.Generator().manual_seed(77)
    inv = (10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
    inv_d = torch.from_numpy(inv).cuda()
    num = 40
    kp, vp = (torch.full((num, kv, page, w), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
              for w in (d, v))
    kw = dict(k_scales=torch.full((num, kv, page), 255, dtype=torch.uint8, device="cuda"),
              v_scales=torch.full((num, kv, page), 255, dtype=torch.uint8, device="cuda"))
    perm = np.random.default_rng(1).permutation(num).astype(np.int32)
    pt = torch.from_numpy(perm[:5].copy()).cuda()
    table = torch.from_numpy(perm[5:5 + 4 * B].reshape(B, 4).copy()).cuda()

    def tokens(n):
        return tuple(torch.randn(n, h, w, generator=g).to(dt) for h, w in ((H, d), (kv, d), (kv, v)))

    _, k0, v0 = tokens(P)
    ex.append_paged(k0.cuda(), v0.cuda(), kp, vp, pt[None], torch.tensor([P], dtype=torch.int32).cuda(),
                    inv_freq=inv_d, **kw)
    keys, vals = [[k0] for _ in range(B)], [[v0] for _ in range(B)]
    lens, nqs = [0] * B, [17, 1, 30]
    for step in range(steps):
        starts = np.concatenate(([0], np.cumsum(nqs))).astype(np.int32)
        q, k, vv = tokens(int(starts[-1]))
        for b in range(B):
            keys[b].append(k[starts[b]:starts[b + 1]])
            vals[b].append(vv[starts[b]:starts[b + 1]])
            lens[b] += nqs[b]
        ln = torch.tensor(lens, dtype=torch.int32).cuda()
        st = torch.from_numpy(starts).cuda()
        qr = ex.append_paged(k.cuda(), vv.cuda(), kp, vp, table, ln, q_starts=st, q=q.cuda(), inv_freq=inv_d,
                             pos_offset=P, **kw)
        y, L = ex.fwd_prefix(qr, kp, vp, pt, P, table, ln, 1 / math.sqrt(d), "causal", q_starts=st, **kw)
        for b in range(B):
            kk = torch.cat(keys[b]).double().numpy()
            kk = e4m3.values(*e4m3.quantise(np.stack([oracle.rotate(x, i, inv, False) for i, x in enumerate(kk)])))
            vv64 = e4m3.values(*e4m3.quantise(torch.cat(vals[b]).double().numpy()))
            for i in range(nqs[b]):
                t, n = starts[b] + i, P + lens[b] - nqs[b] + i + 1
                qq = oracle.rotate(q[t].double().numpy(), n - 1, inv, False)
                for h in range(H):
                    s = kk[:n, h // G] @ qq[h] / math.sqrt(d)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    A = p @ np.abs(vv64[:n, h // G])
                    # Queries are rounded after their rotation: a score is off by 2^-8 (2^-20) of
                    # c sum |q k|, at most |q| |k| / sqrt(d); p by 2^-8 at most, Y by its own rounding.
                    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
                    ds = eps * np.linalg.norm(qq[h]) * np.linalg.norm(kk[:n, h // G], axis=1).max() / math.sqrt(d)
                    tol = (math.expm1(2 * ds) + 3 * eps) * A
                    err = np.abs(y[t, h].double().cpu().numpy() - p @ vv64[:n, h // G])
                    assert (err <= tol).all()
        nqs = [1] * B if step else [2, 1, 3]


def test_captured_launch_follows_lengths_and_tables(ex, path):
    """Two graphs over append and attention, each with its own workspaces, replayed as the sequences
    grow, and an uncaptured call between."""
    b = Batch8([60, 10, 33], [1, 1, 1], 8, 2, 64, 64, "bf16", 16, seed=41)
    b.table[:, -1] = b.k_pages.shape[0] - 1 - np.arange(3)  # room to grow (spare pages)
    b.table[2, -1] = int(b.table[0, -1])
    k, v, table, lens, _, ks, vs = b.cache()
    q, kn, vn = b.dev("q", "k_new", "v_new")
    kw = dict(k_scales=ks, v_scales=vs)
    shape = ex.paged_shape(q, k, v, table)
    s = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        y, L = torch.empty_like(q), torch.empty(3, 8, device="cuda")
        ws, ws2 = (ex.workspace(ex.paged_workspace_size(shape), "cuda") for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            ex.append_paged(kn, vn, k, v, table, lens, ws=ws2, **kw)
            ex.fwd_paged(q, k, v, table, lens, 0.05, "causal", y=y, L=L, ws=ws, **kw)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            ex.append_paged(kn, vn, k, v, table, lens, ws=ws2, **kw)
            ex.fwd_paged(q, k, v, table, lens, 0.05, "causal", y=y, L=L, ws=ws, **kw)
        graphs.append((graph, y, L, ws, ws2))  # a graph's buffers live as long as it
    for step in range(3):
        lens.add_(1)
        kn.normal_()
        graphs[0][0].replay()
        graphs[1][0].replay()
        y, L = ex.fwd_paged(q, k, v, table, lens, 0.05, "causal", **kw)
        torch.cuda.synchronize()
        for graph, yg, Lg, ws, ws2 in graphs:
            assert torch.equal(y, yg) and torch.equal(L, Lg)
            assert ex.device_status(ws) == 0 and ex.device_status(ws2) == 0
        b.lens = lens.cpu().numpy()
        for name, t in (("k_pages", k), ("v_pages", v), ("k_scales", ks), ("v_scales", vs)):
            setattr(b, name, t.view(torch.uint8).cpu().numpy())
        b.requantised()
        _check(path, b, y, L, 0.05, "causal")


def test_outputs_belong_to_the_call_stream(ex):
    """What a call allocates is memory of the stream it runs on."""
    b = Batch8([300, 80], [1, 1], 4, 2, 64, 64, "bf16", 16, seed=12, prefix=40)
    k, v, table, lens, _, ks, vs = b.cache()
    q, pt = b.dev("q", "prefix_table")
    kw = dict(k_scales=ks, v_scales=vs)
    new = q[:, :2].contiguous()
    kp, vp = torch.zeros_like(k), torch.zeros_like(v)
    side = torch.cuda.Stream()
    calls = [lambda s: ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", stream=s, **kw)[0],
             lambda s: ex.fwd_prefix(q, k, v, pt, 40, table, lens, 0.125, "causal", stream=s, **kw)[0],
             lambda s: ex.append_paged(new, new, kp, vp, table, lens, q=q, stream=s, k_scales=torch.zeros_like(ks),
                                       v_scales=torch.zeros_like(vs))]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        left = torch.empty_like(want)
        torch.cuda._sleep(20_000_000)  # about 10 ms
        left.fill_(9.0)
        del left  # its block is free for the current stream, its write still to come
        got = call(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_two_streams_at_once(ex, path):
    b = Batch8([3000, 10, 900], [1, 2, 1], 8, 2, 128, 128, "bf16", 16, seed=51)
    k, v, table, lens, starts, ks, vs = b.cache()
    q, = b.dev("q")
    kw = dict(q_starts=starts, k_scales=ks, v_scales=vs)
    want = ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", stream=s, **kw))
    torch.cuda.synchronize()
    for y, L in got:
        assert torch.equal(y, want[0]) and torch.equal(L, want[1])

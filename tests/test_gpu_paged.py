"""GPU parity of the paged-cache operators against the float64 oracle: append with
rotation, attention over pages, attention behind a shared prefix, and a run of
the three together."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from paged_inputs import DT, Batch, check_attention

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


def _p_bits(path, dtype, tokens, batch, group):
    """Significant bits of p in P.V: the kernel for many rows to a key head rounds it to
    bf16 (off by 2^-8 of p at most), the one for few keeps 2^-17 in bf16; in fp32 p is
    whole or two tf32 parts (2^-21), which the sums' own terms cover."""
    if dtype == "f32":
        return 21
    many = -(-tokens // batch) * group > 16
    return 8 if path == "auto" and dtype == "bf16" and many else 16


# Attention: (lens, nqs, H, kv, d, v, dtype, page, mask, window, pad)
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
    ([1, 2, 3, 4, 5], [1, 1, 1, 1, 1], 2, 1, 8, 8, "bf16", 1, "causal", 0, 0),  # pages of one key
    ([400], [1], 4, 4, 256, 256, "bf16", 16, "causal", 0, 0),
    ([150, 90], [3, 6], 4, 2, 192, 128, "f32", 16, "window", 64, 0),
    ([300], [70], 8, 2, 128, 128, "bf16", 64, "causal", 0, 0),                  # a chunk of a prompt
    ([257, 130], [257, 130], 4, 2, 64, 64, "bf16", 16, "causal", 0, 0),         # whole prompts
    ([90, 200], [33, 50], 3, 3, 112, 64, "f32", 128, "window", 20, 0),
    ([640, 5], [20, 5], 8, 1, 96, 96, "bf16", 1024, "none", 0, 5),
]


def _attend(ex, b, mask, window, scale, **kw):
    q, k, v, table, lens, starts = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts")
    y = torch.full((b.T, b.H, v.shape[3]), 7.0, dtype=q.dtype, device="cuda")
    L = torch.full((b.T, b.H), 7.0, dtype=torch.float32, device="cuda")
    shape = ex.paged_shape(q, k, v, table)
    ws = torch.full((ex.paged_workspace_size(shape),), 0xFF, dtype=torch.uint8, device="cuda")
    y, L = ex.fwd_paged(q, k, v, table, lens, scale, mask, window, q_starts=starts, y=y, L=L, ws=ws, **kw)
    return y, L, ex.device_status(ws)


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention_over_pages(ex, path, case):
    lens, nqs, H, kv, d, v, dtype, page, mask, window, pad = case
    b = Batch(lens, nqs, H, kv, d, v, dtype, page, seed=ATTEND.index(case) + 100, pad=pad)
    scale = 1 / math.sqrt(d)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, scale,
                        mask, window)
    y, L, status = _attend(ex, b, mask, window, scale)
    assert status == 0
    check_attention(dtype, y, L, ref, d, max(lens), _p_bits(path, dtype, b.T, len(lens), H // kv))
    if pad:  # rows behind the last sequence stay as they were
        assert (y[-pad:] == 7).all() and (L[-pad:] == 7).all()


# Rows of a key head around the edges of a 128-row half and of a 256-row tile, with
# prompts before and behind 128-key blocks.
@pytest.mark.parametrize("nqs,G", [([127], 1), ([128], 1), ([129, 3], 1), ([256, 1, 200], 1), ([257], 1),
                                   ([86, 85], 3), ([37, 74, 1], 7)])
@pytest.mark.parametrize("page,d,v,mask,window", [(8, 128, 128, "causal", 0), (64, 64, 64, "window", 150),
                                                  (128, 72, 120, "causal", 0), (256, 128, 64, "none", 0)])
def test_many_rows(ex, nqs, G, page, d, v, mask, window):
    lens = [n + x for n, x in zip(nqs, (130, 0, 400))]
    b = Batch(lens, nqs, 2 * G, 2, d, v, "bf16", page, seed=len(nqs) + G + page)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, mask,
                        window)
    y, L, status = _attend(ex, b, mask, window, 0.1)
    assert status == 0
    check_attention("bf16", y, L, ref, d, max(lens), _p_bits("auto", "bf16", b.T, len(lens), G))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 5.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(ex, path, dtype, scale):
    b = Batch([70, 300], [2, 50], 8, 2, 64, 64, dtype, 16, seed=3)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, scale,
                        "causal")
    y, L, status = _attend(ex, b, "causal", 0, scale)
    assert status == 0
    check_attention(dtype, y, L, ref, 64, 300, _p_bits(path, dtype, b.T, 2, 4))


@pytest.mark.parametrize("dtype,G,nq", [("bf16", 1, 1), ("bf16", 4, 1), ("bf16", 2, 40), ("f32", 4, 2)])
def test_rows_without_keys(ex, path, dtype, G, nq):
    """A sequence of no cached keys, and one with fewer keys than tokens (its first
    tokens stand before every key)."""
    lens, nqs = [0, 2, 50, 1], [nq, nq + 2, nq, nq]
    b = Batch(lens, nqs, 2 * G, 2, 64, 64, dtype, 16, seed=5)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.125,
                        "causal")
    y, L, status = _attend(ex, b, "causal", 0, 0.125)
    assert status == 5
    check_attention(dtype, y, L, ref, 64, 50, _p_bits(path, dtype, b.T, 4, G))
    assert np.isneginf(L.cpu().numpy()[:nq]).all()


@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 3), ("bf16", 40), ("f32", 2)])
def test_pages_outside_the_pool_are_left_out(ex, path, dtype, nq):
    """The kernels check every entry that they use: keys on such a page are left out
    and the status word says so; entries that a window never reaches are not read."""
    b = Batch([200, 90], [nq, nq], 4, 2, 64, 64, dtype, 16, seed=9)
    num = b.k_pages.shape[0]
    b.table[0, 3], b.table[0, 5], b.table[1, 0] = -1, num, 2 ** 31 - 1
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.125,
                        "causal")
    y, L, status = _attend(ex, b, "causal", 0, 0.125)
    assert status == 8
    check_attention(dtype, y, L, ref, 64, 200, _p_bits(path, dtype, b.T, 2, 2))
    b = Batch([200, 90], [nq, nq], 4, 2, 64, 64, dtype, 16, seed=9)
    b.table[0, :4] = -5
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.125,
                        "window", 70)
    y, L, status = _attend(ex, b, "window", 70, 0.125)
    assert status == 0
    check_attention(dtype, y, L, ref, 64, 200, _p_bits(path, dtype, b.T, 2, 2))


def test_numbers_that_do_not_fit_are_clamped(ex, path):
    b = Batch([40, 60], [2, 2], 2, 1, 64, 64, "bf16", 16, seed=2)
    want = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, np.array([0, 60]), b.starts,
                         0.1, "none")
    b.lens[0] = -3
    y, L, status = _attend(ex, b, "none", 0, 0.1)
    assert status == 8
    check_attention("bf16", y, L, want, 64, 60)
    b = Batch([40, 60], [2, 2], 2, 1, 64, 64, "bf16", 16, seed=2)
    want = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, "none")
    b.starts[2] = 1000  # behind the tokens
    y, L, status = _attend(ex, b, "none", 0, 0.1)
    assert status == 8
    check_attention("bf16", y, L, want, 64, 60)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_key_that_a_row_does_not_allow_leaves_no_trace_in_its_score(ex, path, dtype):
    """Keys of the last token that are infinite or NaN do not reach the tokens before
    it, whose masks leave them out (the value is finite)."""
    b = Batch([100], [2], 2, 1, 64, 64, dtype, 16, seed=12)
    for bad in (float("nan"), float("inf"), -float("inf")):
        b.k_pages[int(b.table[0, 6]), :, 3] = bad  # key 99
        ref = oracle.attend(b.np(b.q[:1]), b.np(b.k_pages), b.np(b.v_pages), b.table, np.array([99]),
                            [0, 1], 0.125, "causal")
        y, L, _ = _attend(ex, b, "causal", 0, 0.125)
        check_attention(dtype, y[:1], L[:1], ref, 64, 99, _p_bits(path, dtype, 2, 1, 2))


@pytest.mark.parametrize("dtype,nq,G", [("bf16", 1, 2), ("bf16", 3, 4), ("bf16", 40, 2), ("f32", 3, 2)])
def test_keys_before_every_window_leave_no_trace(ex, path, dtype, nq, G):
    """Keys and values that no token's window reaches hold NaN and infinities."""
    n, w = 300, 70
    b = Batch([n, 50], [nq, nq], 2 * G, 2, 64, 96, dtype, 32, seed=18)
    first = n - nq + 1 - w
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, "window", w)
    for j in range(first):
        for x in (b.k_pages, b.v_pages):
            x[int(b.table[0, j // 32]), :, j % 32] = (float("nan"), float("inf"), -float("inf"))[j % 3]
    y, L, status = _attend(ex, b, "window", w, 0.1)
    assert status == 0
    check_attention(dtype, y, L, ref, 64, w, _p_bits(path, dtype, b.T, 2, G))


@pytest.mark.parametrize("d,v,page,nq,dtype", [(8, 8, 8, 40, "bf16"), (16, 128, 16, 40, "bf16"), (128, 8, 64, 300, "bf16"),
                                               (64, 64, 4, 40, "bf16"), (4, 4, 2, 3, "f32"), (128, 128, 16, 60, "f32")])
def test_narrow_rows_and_small_pages(ex, path, d, v, page, nq, dtype):
    b = Batch([310, nq], [nq, nq], 4, 2, d, v, dtype, page, seed=d + v)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.2, "causal")
    y, L, status = _attend(ex, b, "causal", 0, 0.2)
    assert status == 0
    check_attention(dtype, y, L, ref, d, 310, _p_bits(path, dtype, b.T, 2, 2))


@pytest.mark.parametrize("nq,page", [(1, 16), (5, 8), (3, 128)])
@pytest.mark.parametrize("dtype,d,v", [("bf16", 72, 96), ("bf16", 96, 80), ("bf16", 104, 128), ("f32", 68, 96),
                                       ("f32", 96, 72), ("f32", 100, 128), ("f32", 128, 108), ("f32", 112, 112)])
def test_widths_between(ex, path, dtype, d, v, nq, page):
    """Widths below those that the kernels are made for: the columns that are missing stay out of
    the products, also where one is wider than the other; an infinite value stays in its column."""
    b = Batch([700, nq, 90], [nq, nq, nq], 4, 2, d, v, dtype, page, seed=d + v + nq)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, "causal")
    y, L, status = _attend(ex, b, "causal", 0, 0.1)
    assert status == 0
    bits = _p_bits(path, dtype, b.T, 3, 2)
    check_attention(dtype, y, L, ref, d, 700, bits)
    b.v_pages[int(b.table[0, 0]), :, 0, v - 1] = float("inf")  # the first key of the first sequence
    y2, L2, status = _attend(ex, b, "causal", 0, 0.1)
    assert status == 0 and torch.equal(L2, L)
    assert not torch.isfinite(y2[:nq, :, v - 1]).any()
    assert torch.equal(y2[nq:], y[nq:]) and torch.equal(y2[..., :v - 1], y[..., :v - 1])


@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("f32", 2), ("bf16", 30)])
def test_large_batches(ex, path, dtype, nq, prefix):
    """The largest batch, most sequences short, some without tokens or keys."""
    B = 1024 if nq < 30 else 60
    rng = np.random.default_rng(B)
    nqs = [0 if x == 0 else int(rng.integers(1, nq + 1)) for x in rng.integers(0, 5, B)]
    lens = [int(rng.integers(0, 40)) + q for q in nqs]
    b = Batch(lens, nqs, 2, 1, 64, 64, dtype, 16, seed=B, prefix=prefix)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, "causal",
                        prefix=(b.prefix_table, prefix) if prefix else None)
    if prefix:
        q, k, v, table, ln, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
        y, L = ex.fwd_prefix(q, k, v, pt, prefix, table, ln, 0.1, "causal", q_starts=starts)
    else:
        y, L, status = _attend(ex, b, "causal", 0, 0.1)
        assert status == 0
    check_attention(dtype, y, L, ref, 64, 80 + prefix, _p_bits(path, dtype, b.T, 1 if prefix else B, 2),
                    extra=2.0 ** -20)


@pytest.mark.parametrize("prefix", [0, 100])
@pytest.mark.parametrize("B", [31, 32, 33, 64, 127, 128, 129])
def test_batches_around_a_warps_share(ex, path, B, prefix):
    """A run's start is found lane by lane in small batches, the prefix among the sequences."""
    rng = np.random.default_rng(B)
    nqs = [int(rng.integers(0, 3)) for _ in range(B)]
    nqs[0] = nqs[-1] = 0 if B % 2 else 2
    lens = [int(rng.integers(0, 300)) + q for q in nqs]
    b = Batch(lens, nqs, 4, 2, 64, 64, "bf16", 16, seed=B, prefix=prefix)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, "causal",
                        prefix=(b.prefix_table, prefix) if prefix else None)
    if prefix:
        q, k, v, table, ln, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
        y, L = ex.fwd_prefix(q, k, v, pt, prefix, table, ln, 0.1, "causal", q_starts=starts)
    else:
        y, L, status = _attend(ex, b, "causal", 0, 0.1)
        assert status == 0
    check_attention("bf16", y, L, ref, 64, 302 + prefix, _p_bits(path, "bf16", b.T, 1 if prefix else B, 2),
                    extra=2.0 ** -20)


def test_tokens_in_front_of_the_first_sequence(ex, path):
    """q_starts may begin behind some tokens, and descend by mistake: rows that no sequence
    owns stay as they were in both operators; nothing outside the tokens is touched."""
    b = Batch([60, 40, 33], [2, 3, 2], 4, 2, 64, 64, "bf16", 16, seed=4, prefix=50)
    for starts, status in (([1, 3, 4, 6], 0), ([1, 4, 2, 6], 8), ([5, 3, 9, -2], 8)):
        own = np.full(b.T, -1)
        s = np.array(starts, dtype=np.int32)
        lo = [min(max(int(x), 0), b.T) for x in s[:-1]]
        hi = [min(max(int(y), x), b.T) for x, y in zip(lo, s[1:])]
        for i, (x, y) in enumerate(zip(lo, hi)):
            own[x:y] = i
        b.starts = s
        y, L, st = _attend(ex, b, "causal", 0, 0.125)
        assert st == status
        assert (y[torch.from_numpy(own < 0).cuda()] == 7).all()
        q, k, v, table, lens, qs, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
        y2 = torch.full_like(q, 7.0)
        L2 = torch.full((b.T, 4), 7.0, device="cuda")
        ws = ex.workspace(ex.prefix_workspace_size(ex.paged_shape(q, k, v, table)), "cuda")
        ws.fill_(0xFF)
        ex.fwd_prefix(q, k, v, pt, 50, table, lens, 0.125, "causal", q_starts=qs, y=y2, L=L2, ws=ws)
        assert ex.device_status(ws) == status
        assert (y2[torch.from_numpy(own < 0).cuda()] == 7).all() and (L2[torch.from_numpy(own < 0).cuda()] == 7).all()
        if status == 0:
            ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, list(map(int, s)),
                                0.125, "causal", prefix=(b.prefix_table, 50))
            check_attention("bf16", y2, L2, ref, 64, 110, _p_bits(path, "bf16", b.T, 1, 2), extra=2.0 ** -20)


def test_equal_tokens_without_q_starts(ex, path):
    b = Batch([70, 33, 128], [2, 2, 2], 4, 2, 128, 128, "bf16", 16, seed=21)
    q, k, v, table, lens, starts = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts")
    y0, L0 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal", q_starts=starts)
    y1, L1 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal")
    assert torch.equal(y0, y1) and torch.equal(L0, L1)


def test_queries_that_are_columns_of_a_projection(ex, path):
    b = Batch([70, 33], [1, 2], 4, 2, 64, 64, "bf16", 16, seed=22)
    q, k, v, table, lens, starts = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts")
    wide = torch.randn(b.T, 4 * 64 + 72, device="cuda").to(q.dtype)
    wide[:, 8:8 + 256] = q.reshape(b.T, 256)
    y0, L0 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal", q_starts=starts)
    y1, L1 = ex.fwd_paged(wide[:, 8:8 + 256].view(b.T, 4, 64), k, v, table, lens, 0.1, "causal",
                          q_starts=starts)
    assert torch.equal(y0, y1) and torch.equal(L0, L1)


@pytest.mark.parametrize("dtype,nq", [("bf16", 1), ("bf16", 40), ("f32", 1)])
def test_pool_beyond_32_bit_offsets(ex, path, dtype, nq):
    """Pages at the far end of a pool of more than 2^31 elements."""
    kv, page, d = 8, 64, 128
    num = (1 << 31) // (kv * page * d) + 40
    b = Batch([500], [nq], 16, kv, d, d, dtype, page, seed=31)
    need = b.table[0, :8].copy()
    far = torch.empty(num, kv, page, d, dtype=DT[dtype], device="cuda")
    farv = torch.empty_like(far)
    table = b.table.copy()
    for i, at in enumerate(need):
        far[num - 1 - i] = b.k_pages[int(at)].cuda()
        farv[num - 1 - i] = b.v_pages[int(at)].cuda()
        table[0, i] = num - 1 - i
    q, lens = b.dev("q", "lens")
    y, L = ex.fwd_paged(q, far, farv, torch.from_numpy(table).cuda(), lens, 0.1, "causal")
    q, k, v, t0 = b.dev("q", "k_pages", "v_pages", "table")
    y0, L0 = ex.fwd_paged(q, k, v, t0, lens, 0.1, "causal")
    assert torch.equal(y, y0) and torch.equal(L, L0)
    k_new, v_new = (x[:nq].contiguous() for x in b.dev("k_new", "v_new"))
    ex.append_paged(k_new, v_new, far, farv, torch.from_numpy(table).cuda(), lens)
    at = 500 - nq
    assert torch.equal(far[num - 1 - at // page, :, at % page], k_new[0])
    assert torch.equal(farv[num - 1 - 499 // page, :, 499 % page], v_new[nq - 1])


# Shared prefix: (prefix, lens, nqs, H, kv, d, v, dtype, page, mask, pad)
PREFIX = [
    (1, [1], [1], 1, 1, 64, 64, "bf16", 16, "causal", 0),
    (300, [5, 1, 40], [1, 1, 1], 8, 2, 128, 128, "bf16", 16, "causal", 0),
    (1000, [3, 70, 1, 0, 9], [3, 5, 1, 0, 2], 6, 2, 64, 64, "bf16", 64, "causal", 2),
    (513, [40, 80], [2, 1], 4, 1, 80, 96, "f32", 32, "none", 0),
    (90, [12] * 40, [1] * 40, 16, 2, 128, 128, "bf16", 16, "causal", 0),
    (257, [20, 30], [20, 30], 8, 2, 64, 128, "bf16", 32, "none", 1),
    (130, [7, 9], [1, 1], 2, 2, 200, 104, "bf16", 16, "causal", 0),
    (2000, [1, 1], [1, 1], 4, 4, 128, 128, "f32", 64, "causal", 0),
    (0, [30, 5], [2, 1], 4, 2, 64, 64, "bf16", 16, "causal", 0),
    # Long enough for tall tiles in a launch of their own.
    (4001, [40, 1, 90, 17] * 4, [1, 1, 1, 0] + [1] * 12, 32, 8, 128, 128, "bf16", 64, "causal", 1),
]


@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_attention_behind_a_shared_prefix(ex, path, case):
    prefix, lens, nqs, H, kv, d, v, dtype, page, mask, pad = case
    b = Batch(lens, nqs, H, kv, d, v, dtype, page, seed=PREFIX.index(case) + 200, pad=pad, prefix=prefix)
    if pad:
        b.q[-pad:] = float("nan")
    scale = 1 / math.sqrt(d)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, scale,
                        mask, prefix=(b.prefix_table, prefix))
    q, k, vv, table, lens_, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts",
                                               "prefix_table")
    y = torch.full((b.T, H, v), 7.0, dtype=q.dtype, device="cuda")
    L = torch.full((b.T, H), 7.0, device="cuda")
    ws = ex.workspace(ex.prefix_workspace_size(ex.paged_shape(q, k, vv, table)), "cuda")
    ex.fwd_prefix(q, k, vv, pt, prefix, table, lens_, scale, mask, q_starts=starts, y=y, L=L, ws=ws)
    assert ex.device_status(ws) == 0
    # The prefix's pass takes every token as one sequence's.
    check_attention(dtype, y, L, ref, d, prefix + max(lens), _p_bits(path, dtype, b.T, 1, H // kv),
                    extra=2.0 ** -20)
    if pad:
        assert (y[-pad:] == 7).all() and (L[-pad:] == 7).all()


def test_a_sequence_without_own_keys_still_has_the_prefix(ex, path):
    """With a prefix no row is empty: a sequence of no own keys (mask none), and one
    with fewer own keys than tokens."""
    b = Batch([0, 1], [2, 3], 4, 2, 64, 64, "bf16", 16, seed=8, prefix=50)
    q, k, v, table, lens, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts",
                                             "prefix_table")
    ws = ex.workspace(ex.prefix_workspace_size(ex.paged_shape(q, k, v, table)), "cuda")
    for mask in ("none", "causal"):
        ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.125,
                            mask, prefix=(b.prefix_table, 50))
        y, L = ex.fwd_prefix(q, k, v, pt, 50, table, lens, 0.125, mask, q_starts=starts, ws=ws)
        assert ex.device_status(ws) == 0
        check_attention("bf16", y, L, ref, 64, 51, extra=2.0 ** -20)
    pt[1] = -1
    y, L = ex.fwd_prefix(q, k, v, pt, 50, table, lens, 0.125, "none", q_starts=starts, ws=ws)
    assert ex.device_status(ws) == 8
    b.prefix_table[1] = -1
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.125,
                        "none", prefix=(b.prefix_table, 50))
    check_attention("bf16", y, L, ref, 64, 51, extra=2.0 ** -20)


# Append: (lens, nqs, H, kv, d, v, dtype, page, pairs, interleaved, offset, pad, with q, strided)
APPEND = [
    ([1], [1], 1, 1, 64, 64, "bf16", 16, 32, False, 0, 0, True, False),
    ([40, 7, 300], [1, 1, 1], 8, 2, 128, 128, "bf16", 16, 64, False, 0, 0, True, True),
    ([40, 7, 300, 9], [5, 7, 30, 0], 6, 2, 80, 96, "f32", 32, 20, True, 1000, 3, True, True),
    ([33, 34], [3, 4], 4, 4, 80, 64, "bf16", 8, 20, False, 0, 0, True, False),   # halves of 20 columns
    ([33, 34], [3, 4], 4, 4, 64, 64, "bf16", 4, 3, False, 5, 0, True, False),    # of 3
    ([33, 34], [3, 4], 4, 4, 64, 64, "f32", 1, 5, True, 0, 0, False, True),
    ([100], [100], 2, 1, 256, 256, "bf16", 64, 128, True, 0, 0, True, False),
    ([100, 50], [20, 1], 3, 1, 12, 4, "f32", 2, 0, False, 0, 1, True, False),    # not rotated
    ([900000], [2], 4, 2, 128, 128, "f32", 1024, 64, False, 100000, 0, True, False),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_append(ex, case):
    lens, nqs, H, kv, d, v, dtype, page, pairs, inter, offset, pad, with_q, strided = case
    b = Batch([min(n, 2000) for n in lens], nqs, H, kv, d, v, dtype, page, seed=APPEND.index(case) + 300, pad=pad)
    if max(lens) > 2000:  # a far position: its page alone is in the table
        b.lens = np.array(lens, dtype=np.int32)
        far = np.full((len(lens), -(-max(lens) // page)), -1, dtype=np.int32)
        far[:, -1] = 0
        b.table = far
    inv = (10000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)
    q, k, vv, table, lens_, starts, kn, vn = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts",
                                                   "k_new", "v_new")
    if strided:
        wide = torch.zeros(b.T, H * d + kv * (d + v) + 8, dtype=q.dtype, device="cuda")
        wide[:, :H * d], wide[:, H * d:H * d + kv * d] = q.reshape(b.T, -1), kn.reshape(b.T, -1)
        wide[:, H * d + kv * d:H * d + kv * (d + v)] = vn.reshape(b.T, -1)
        q = wide[:, :H * d].view(b.T, H, d)
        kn = wide[:, H * d:H * d + kv * d].view(b.T, kv, d)
        vn = wide[:, H * d + kv * d:H * d + kv * (d + v)].view(b.T, kv, v)
    out = torch.full((b.T, H, d), 7.0, dtype=q.dtype, device="cuda") if with_q else None
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    got = ex.append_paged(kn, vn, k, vv, table, lens_, q_starts=starts, q=q if with_q else None, q_out=out,
                          inv_freq=torch.from_numpy(inv).cuda() if pairs else None, interleaved=inter,
                          pos_offset=offset, ws=ws)
    assert ex.device_status(ws) == 0
    assert got is out
    qo, kr, vr = oracle.append(b.np(b.k_new), b.np(b.v_new), b.np(b.k_pages), b.np(b.v_pages), b.table,
                               b.lens, b.starts, b.np(b.q), inv, inter, offset)
    # Rotated values: cos and sin are off by 2^-22 (the turn in fp32, the functions),
    # the two products and their sum by 3 * 2^-24 of the pair's size, then one rounding.
    def close(x, ref, size):
        x = x.double().cpu().numpy()
        same = np.isnan(ref)
        assert np.array_equal(np.isnan(x), same)
        eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        tol = 2.0 ** -20 * size + eps * (np.abs(ref) + 2.0 ** -20 * size)
        assert (np.abs(x - ref)[~same] <= tol[~same]).all()

    size = 2 * max(float(b.k_new.double().abs().max()), float(b.q.double().abs().max()))
    close(k, kr, np.full(kr.shape, size))
    assert np.array_equal(np.nan_to_num(vv.double().cpu().numpy(), nan=1e9), np.nan_to_num(vr, nan=1e9))
    if with_q:
        n = int(b.starts[-1])
        close(out[:n], qo[:n], np.full(qo[:n].shape, size))
        assert (out[n:] == 7).all()


def test_append_frequencies_of_any_size(ex):
    """Frequencies that are zero, negative, subnormal, above a turn a token; an infinite or
    NaN one makes its own pair NaN and no other."""
    inv = np.array([0.0, -0.5, 1e-12, 3e-39, 7.5, 1000.25, np.inf, 1.0, np.nan, -2.0 ** 100, 2.0 ** 30, 1e-3],
                   dtype=np.float32)
    d, n = 2 * len(inv), 1000003
    q = torch.randn(3, 2, d, generator=torch.Generator().manual_seed(1))
    pos = np.arange(n - 3, n, dtype=np.float64)
    table = torch.full((1, -(-n // 1024)), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 0
    pool = torch.zeros(1, 2, 1024, d, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = ex.append_paged(q.cuda(), q.cuda(), pool, torch.zeros_like(pool), table, lens, q=q.cuda(),
                          inv_freq=torch.from_numpy(inv).cuda()).double().cpu().numpy()
    # Angles of 2^30 a token and more lose the low bits of 1 / (2 pi): any angle, but a rotation.
    exact = np.abs(inv) < 2 ** 20
    with np.errstate(invalid="ignore", over="ignore"):
        turn = pos[:, None] * inv.astype(np.float64)
        c, s = np.cos(turn)[:, None], np.sin(turn)[:, None]
    x, y = q[..., :len(inv)].double().numpy(), q[..., len(inv):].double().numpy()
    bad = ~np.isfinite(inv)
    assert np.isnan(out[..., :len(inv)][..., bad]).all() and np.isnan(out[..., len(inv):][..., bad]).all()
    # As in test_append; the oracle's own turn of 10^9 radians is off by 2^-24 of one.
    tol = 2.0 ** -20 * 2 * float(q.abs().max())
    assert (np.abs(out[..., :len(inv)] - (x * c - y * s))[..., exact] <= tol).all()
    assert (np.abs(out[..., len(inv):] - (y * c + x * s))[..., exact] <= tol).all()
    big = ~exact & ~bad
    size = out[..., :len(inv)] ** 2 + out[..., len(inv):] ** 2
    assert (np.abs(size - (x * x + y * y))[..., big] <= 2 * tol * np.sqrt(x * x + y * y)[..., big] + tol * tol).all()


def test_append_rotates_q_in_place(ex):
    b = Batch([40, 9], [3, 2], 4, 2, 64, 64, "bf16", 16, seed=1)
    q, k, v, table, lens, starts, kn, vn = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts",
                                                 "k_new", "v_new")
    inv = torch.pow(10000.0, -torch.arange(32, device="cuda") / 32).float()
    want = ex.append_paged(kn, vn, k, v, table, lens, q_starts=starts, q=q, inv_freq=inv)
    got = ex.append_paged(kn, vn, k, v, table, lens, q_starts=starts, q=q, q_out=q, inv_freq=inv)
    assert got is q and torch.equal(got, want)


def test_append_without_a_place(ex):
    """Tokens before position 0, behind the table, or on a page outside the pool: nothing of
    theirs is written, the others' are, and the status word says so."""
    for lens, edit in (([1, 20], None), ([20, 20], (0, 1, -7)), ([20, 20], (0, 1, 99)), ([900, 20], None)):
        b = Batch([20, 20], [3, 2], 2, 1, 64, 64, "bf16", 16, seed=6)
        b.lens = np.array(lens, dtype=np.int32)
        if edit:
            b.table[edit[0], edit[1]] = edit[2]
        q, k, v, table, lens_, starts, kn, vn = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts",
                                                      "k_new", "v_new")
        ws = ex.workspace(256, "cuda")
        ex.append_paged(kn, vn, k, v, table, lens_, q_starts=starts, ws=ws)
        assert ex.device_status(ws) == 8
        _, kr, vr = oracle.append(b.np(b.k_new), b.np(b.v_new), b.np(b.k_pages), b.np(b.v_pages), b.table,
                                  b.lens, b.starts)
        for x, r in ((k, kr), (v, vr)):
            assert np.array_equal(np.nan_to_num(x.double().cpu().numpy(), nan=1e9), np.nan_to_num(r, nan=1e9))
    ex.append_paged(kn, vn, k, v, table, torch.tensor([20, 20], dtype=torch.int32, device="cuda"),
                    q_starts=starts, ws=ws)
    assert ex.device_status(ws) == 0  # cleared by the next call


@pytest.mark.parametrize("dtype,G,widths", [("bf16", 4, (128, 128)), ("f32", 1, (80, 96)), ("bf16", 16, (64, 64))])
def test_a_run_of_the_three(ex, path, dtype, G, widths):
    """A server's program: a common prompt appended, each request's own tokens behind it, then
    decode steps, each an append and an attention behind the prefix; the last step against
    the oracle over keys that it rotates itself."""
    d, v = widths
    kv, page, P, B, steps = 2, 16, 75, 3, 4
    H, dt = kv * G, DT[dtype]
    g = torch.Generator().manual_seed(77)
    inv = (10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
    inv_d = torch.from_numpy(inv).cuda()
    num = 40
    kp = torch.full((num, kv, page, d), float("nan"), dtype=dt, device="cuda")
    vp = torch.full((num, kv, page, v), float("nan"), dtype=dt, device="cuda")
    perm = np.random.default_rng(1).permutation(num).astype(np.int32)
    pt = torch.from_numpy(perm[:5].copy()).cuda()
    table = torch.from_numpy(perm[5:5 + 4 * B].reshape(B, 4).copy()).cuda()

    def tokens(n):
        return tuple(torch.randn(n, h, w, generator=g).to(dt) for h, w in ((H, d), (kv, d), (kv, v)))

    _, k0, v0 = tokens(P)
    ex.append_paged(k0.cuda(), v0.cuda(), kp, vp, pt[None], torch.tensor([P], dtype=torch.int32).cuda(),
                    inv_freq=inv_d)
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
                             pos_offset=P)
        y, L = ex.fwd_prefix(qr, kp, vp, pt, P, table, ln, 1 / math.sqrt(d), "causal", q_starts=st)
        for b in range(B):
            kk = torch.cat(keys[b]).double().numpy()
            kk = np.stack([oracle.rotate(x, i, inv, False) for i, x in enumerate(kk)])
            vv64 = torch.cat(vals[b]).double().numpy()
            for i in range(nqs[b]):
                t, n = starts[b] + i, P + lens[b] - nqs[b] + i + 1
                qq = oracle.rotate(q[t].double().numpy(), n - 1, inv, False)
                for h in range(H):
                    s = kk[:n, h // G] @ qq[h] / math.sqrt(d)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    A = p @ np.abs(vv64[:n, h // G])
                    # Keys and queries are rounded after their rotation: each score is off by
                    # 2 * 2^-8 (2^-24) of c sum |q k|, at most |q| |k| / sqrt(d).
                    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -20
                    ds = 2 * eps * np.linalg.norm(qq[h]) * np.linalg.norm(kk[:n, h // G], axis=1).max() / math.sqrt(d)
                    tol = (math.expm1(2 * ds) + 2 * eps) * A + eps * A
                    err = np.abs(y[t, h].double().cpu().numpy() - p @ vv64[:n, h // G])
                    assert (err <= tol).all()
        nqs = [1] * B if step else [2, 1, 3]


def test_agrees_with_the_dense_decode(ex):
    """Pages against fwd_splitkv on the same keys laid out densely."""
    B, H, n, d, page = 2, 4, 700, 128, 64
    b = Batch([n] * B, [1] * B, H, H, d, d, "bf16", page, seed=14)
    q, k, v, table, lens = b.dev("q", "k_pages", "v_pages", "table", "lens")
    dense = [torch.stack([x[table[i, :-1].long()].transpose(0, 1).reshape(H, -1, d)[:, :n] for i in range(B)])
             .contiguous() for x in (k, v)]
    y0, L0 = ex.fwd_splitkv(q.view(B, 1, H, d).transpose(1, 2).contiguous(), *dense, 0.1, "causal")
    y1, L1 = ex.fwd_paged(q, k, v, table, lens, 0.1, "causal")
    assert (L0[:, :, 0] - L1).abs().max() <= 1e-5
    # two roundings to bf16 of values that agree far below that
    assert ((y0[:, :, 0].float() - y1.float()).abs() <= 2.0 ** -7 * y1.float().abs() + 1e-5).all()


def test_captured_launch_follows_lengths_and_tables(ex, path):
    """One graph over append and attention, replayed as the sequences grow; a second
    graph with its own workspace runs between the replays, and an uncaptured call."""
    b = Batch([60, 10, 33], [1, 1, 1], 8, 2, 64, 64, "bf16", 16, seed=41)
    b.table[:, -1] = b.k_pages.shape[0] - 1 - np.arange(3)  # room to grow (spare pages)
    b.table[2, -1] = int(b.table[0, -1])
    q, k, v, table, lens, kn, vn = b.dev("q", "k_pages", "v_pages", "table", "lens", "k_new", "v_new")
    shape = ex.paged_shape(q, k, v, table)
    s = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        y, L = torch.empty_like(q), torch.empty(3, 8, device="cuda")
        ws, ws2 = (ex.workspace(ex.paged_workspace_size(shape), "cuda") for _ in range(2))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            ex.append_paged(kn, vn, k, v, table, lens, ws=ws2)
            ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", y=y, L=L, ws=ws)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            ex.append_paged(kn, vn, k, v, table, lens, ws=ws2)
            ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", y=y, L=L, ws=ws)
        graphs.append((graph, y, L, ws, ws2))  # a graph's buffers live as long as it
    for step in range(3):
        lens.add_(1)
        kn.normal_()
        graphs[0][0].replay()
        graphs[1][0].replay()
        y, L = ex.fwd_paged(q, k, v, table, lens, 0.125, "causal")
        torch.cuda.synchronize()
        for graph, yg, Lg, ws, ws2 in graphs:
            assert torch.equal(y, yg) and torch.equal(L, Lg)
            assert ex.device_status(ws) == 0 and ex.device_status(ws2) == 0
        ref = oracle.attend(b.np(b.q), k.double().cpu().numpy(), v.double().cpu().numpy(),
                            b.table, lens.cpu().numpy(), b.starts, 0.125, "causal")
        check_attention("bf16", y, L, ref, 64, 70)


def test_captured_prefix_in_two_launches(ex):
    """A long prefix under few own keys takes two attention launches, the second of which begins
    beside the first; captured with an append before it and another call behind it on the same
    workspace, and replayed as the sequences grow."""
    P, B = 4001, 16
    b = Batch([60 + 3 * k for k in range(B)], [1] * B, 32, 8, 128, 128, "bf16", 64, seed=43, prefix=P, spare=B)
    free = np.setdiff1d(np.arange(b.k_pages.shape[0]),
                        np.concatenate((b.prefix_table, b.table[b.table < b.k_pages.shape[0]])))
    for x in range(B):  # the page behind the last
        b.table[x, -(-int(b.lens[x]) // 64)] = free[x]
    q, k, v, table, lens, kn, vn, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "k_new", "v_new",
                                             "prefix_table")
    shape = ex.paged_shape(q, k, v, table)
    ws = ex.workspace(ex.prefix_workspace_size(shape), "cuda")
    outs = [(torch.empty_like(q), torch.empty(B, 32, device="cuda")) for _ in range(2)]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()

    def calls():
        ex.append_paged(kn, vn, k, v, table, lens, ws=ws)
        for y, L in outs:
            ex.fwd_prefix(q, k, v, pt, P, table, lens, 0.1, "causal", y=y, L=L, ws=ws)

    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    with torch.cuda.graph(graph, stream=s):
        calls()
    for step in range(3):
        lens.add_(1)
        kn.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert ex.device_status(ws) == 0
        assert all(torch.equal(x, y) for x, y in zip(*outs))
        ref = oracle.attend(b.np(b.q), k.double().cpu().numpy(), v.double().cpu().numpy(), b.table,
                            lens.cpu().numpy(), b.starts, 0.1, "causal", prefix=(b.prefix_table, P))
        check_attention("bf16", *outs[0], ref, 128, P + 110, 8)


def test_outputs_belong_to_the_call_stream(ex):
    """What a call allocates is memory of the stream it runs on: a tensor of the current
    stream that was freed while a write to it was still queued is not handed out again."""
    b = Batch([300, 80], [1, 1], 4, 2, 64, 64, "bf16", 16, seed=12, prefix=40)
    q, k, v, table, lens, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "prefix_table")
    new, kp, vp = q[:, :2].contiguous(), torch.zeros_like(k), torch.zeros_like(v)
    side = torch.cuda.Stream()
    calls = [lambda s: ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", stream=s)[0],
             lambda s: ex.fwd_prefix(q, k, v, pt, 40, table, lens, 0.125, "causal", stream=s)[0],
             lambda s: ex.append_paged(new, new, kp, vp, table, lens, q=q, stream=s)]
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
    b = Batch([3000, 10, 900], [1, 2, 1], 8, 2, 128, 128, "bf16", 16, seed=51)
    q, k, v, table, lens, starts = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts")
    want = ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", q_starts=starts)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ex.fwd_paged(q, k, v, table, lens, 0.125, "causal", q_starts=starts, stream=s))
    torch.cuda.synchronize()
    for y, L in got:
        assert torch.equal(y, want[0]) and torch.equal(L, want[1])

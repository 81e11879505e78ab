"""NaN and infinities in rows, keys and values that paged attention does read."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from paged_inputs import Batch, check_attention

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


def _finite_bound(b, scale):
    """c sum |q k| is infinite where an entry of k is: what the finite ones can make it."""
    k = b.np(b.k_pages)
    return abs(scale) * np.abs(k[np.isfinite(k).all(-1)]).sum(-1).max() * np.abs(b.np(b.q)).max()


def _run(ex, b, scale, prefix, mask="causal"):
    """(Y, L, status) of fwd_paged or, with a prefix, fwd_prefix."""
    q, k, v, table, lens, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
    shape = ex.paged_shape(q, k, v, table)
    size = ex.prefix_workspace_size(shape) if prefix else ex.paged_workspace_size(shape)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    if prefix:
        y, L = ex.fwd_prefix(q, k, v, pt, prefix, table, lens, scale, mask, q_starts=starts, ws=ws)
    else:
        y, L = ex.fwd_paged(q, k, v, table, lens, scale, mask, q_starts=starts, ws=ws)
    return y, L, ex.device_status(ws)


# (dtype, d, v, nq, group): the kernels for one row, a few and many, on either side of 128 columns.
WIDTHS = [("bf16", 64, 64, 1, 1), ("bf16", 128, 96, 2, 4), ("bf16", 128, 128, 40, 2), ("f32", 80, 96, 2, 2),
          ("bf16", 256, 200, 1, 1), ("bf16", 192, 256, 3, 2), ("f32", 160, 256, 2, 2)]


@pytest.mark.parametrize("prefix", [0, 37, 2500])
@pytest.mark.parametrize("n", [20, 2500])  # finished by one worker, joined from several
@pytest.mark.parametrize("case", WIDTHS, ids=lambda c: "-".join(map(str, c)))
def test_nan_scores_make_nan_rows(ex, path, case, n, prefix):
    """Scores that are all NaN, of a token whose query holds a NaN and of a sequence whose only
    key does, give NaN in Y and L and no empty row; other rows stay what they are."""
    dtype, d, v, nq, G = case
    lens, nqs = [n + nq, 1, n + nq], [nq, 1, nq]
    b = Batch(lens, nqs, 2 * G, 2, d, v, dtype, 16, seed=61, prefix=prefix)
    b.q[0, 1, d - 1] = float("nan")  # first token, second head
    hurt = np.zeros((b.T, 2 * G), dtype=bool)
    hurt[0, 1] = True
    if not prefix:  # behind a prefix the row has other keys, whose scores count beside the NaN
        b.k_pages[int(b.table[1, 0]), 1, 0, 0] = float("nan")  # key head 1
        hurt[nq, G:] = True
    scale = 1 / math.sqrt(d)
    with np.errstate(invalid="ignore"):
        ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, scale,
                            "causal", prefix=(b.prefix_table, prefix) if prefix else None)
    assert np.array_equal(np.isnan(ref[1]), hurt)
    y, L, status = _run(ex, b, scale, prefix)
    assert status == 0
    hurt_d = torch.from_numpy(hurt).cuda()
    assert torch.isnan(y[hurt_d]).all() and torch.isnan(L[hurt_d]).all()
    tall = path == "auto" and dtype == "bf16" and d <= 128 and nq * G > 16
    # p has 8 bits on the 256-row tiles, else 16 or more; the oracle's NaN rows are left out.
    check_attention(dtype, y, L, ref, d, prefix + n + nq, 8 if tall else 16, extra=2.0 ** -20)


@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("n", [40, 2500])
@pytest.mark.parametrize("case", WIDTHS, ids=lambda c: "-".join(map(str, c)))
def test_infinite_entries_stay_where_they_reach(ex, path, case, n, prefix):
    """An infinite value that every token of a sequence allows makes its column of their rows
    infinite on the SIMT kernels, as the formula does, and infinite or NaN on the tensor cores; an
    infinite key entry reaches the rows of its key head.  Everything else keeps its bits."""
    dtype, d, v, nq, G = case
    b = Batch([n + nq, 5 + nq, n + nq], [nq] * 3, 2 * G, 2, d, v, dtype, 16, seed=62, prefix=prefix)
    scale = 1 / math.sqrt(d)
    y0, L0, _ = _run(ex, b, scale, prefix)
    assert torch.isfinite(y0).all() and torch.isfinite(L0).all()
    page = int(b.table[0, 1])  # keys 16 to 31 of the first sequence
    here = torch.zeros(b.T, 2 * G, dtype=torch.bool, device="cuda")
    here[:nq, G:] = True  # key head 1
    for bad in (math.inf, -math.inf):
        kept = b.v_pages[page, 1, 3, v - 1].clone()
        b.v_pages[page, 1, 3, v - 1] = bad
        y, L, status = _run(ex, b, scale, prefix)
        assert status == 0 and torch.equal(L, L0)
        hit = y[..., v - 1][here]
        simt = path == "simt" or max(d, v) > 128
        assert (hit == bad).all() if simt else not torch.isfinite(hit).any()
        assert torch.equal(y[..., :v - 1], y0[..., :v - 1]) and torch.equal(y[~here], y0[~here])
        b.v_pages[page, 1, 3, v - 1] = kept
    b.k_pages[page, 1, 3, 0] = math.inf
    y, L, status = _run(ex, b, scale, prefix)
    assert torch.equal(y[~here], y0[~here]) and torch.equal(L[~here], L0[~here])
    if path == "simt" or max(d, v) > 128:
        # A score of -inf leaves the key out, +inf has no result.
        up = b.np(b.q)[:nq, G:, 0] > 0
        with np.errstate(invalid="ignore"):
            ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, scale,
                                "causal", prefix=(b.prefix_table, prefix) if prefix else None)
        assert np.array_equal(np.isnan(ref[1][:nq, G:]), up)
        up = torch.from_numpy(up).cuda()
        assert torch.isnan(y[:nq, G:][up]).all() and torch.isfinite(y[:nq, G:][~up]).all()
        clean = list(ref)
        clean[3] = np.where(np.isfinite(ref[3]), ref[3], _finite_bound(b, scale))
        check_attention(dtype, y, L, clean, d, prefix + n + nq, 16, extra=2.0 ** -20)

"""Numbers of a paged batch that do not fit: append and attention take them alike, so that a
token is written where the attention behind it looks for it, or nowhere."""
import numpy as np
import pytest
import torch

from oracle import paged as oracle
from paged_inputs import Batch, check_attention

pytestmark = pytest.mark.gpu

INV = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)


@pytest.fixture(scope="module")
def ex():
    import exact_tiled_softmax_gb300 as mod
    mod.load_library()
    assert torch.cuda.is_available()
    return mod


def _same(x, ref):
    return np.array_equal(np.nan_to_num(x.double().cpu().numpy(), nan=1e9), np.nan_to_num(ref, nan=1e9))


def _append_and_attend(ex, b, starts, lens):
    """An append of b's new tokens (rotated queries, keys as they are) with these numbers, its
    pools against the oracle's, and an attention behind it on the same numbers."""
    q, k, v, table, kn, vn = b.dev("q", "k_pages", "v_pages", "table", "k_new", "v_new")
    st, ln = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (starts, lens))
    ws = ex.workspace(256, "cuda")
    ex.append_paged(kn, vn, k, v, table, ln, q_starts=st, ws=ws)
    assert ex.device_status(ws) == 8
    _, kr, vr = oracle.append(b.np(b.k_new), b.np(b.v_new), b.np(b.k_pages), b.np(b.v_pages), b.table, lens, starts)
    assert _same(k, kr) and _same(v, vr)
    # The queries are rotated for the same positions.
    qo = torch.full_like(q, 7.0)
    scratch = torch.zeros_like(k), torch.zeros_like(v)
    ex.append_paged(kn, vn, *scratch, table, ln, q_starts=st, q=q, q_out=qo, inv_freq=torch.from_numpy(INV).cuda())
    qr, _, _ = oracle.append(b.np(b.k_new), b.np(b.v_new), b.np(b.k_pages), b.np(b.v_pages), b.table, lens, starts,
                             b.np(b.q), INV)
    got, own = qo.double().cpu().numpy(), ~np.isnan(qr)
    size = 2 * float(b.q.double().abs().max())  # as in the tests of append
    assert (np.abs(got - qr)[own] <= (2.0 ** -20 * size + 2.0 ** -8 * (np.abs(qr) + 2.0 ** -20 * size))[own]).all()
    assert (got[~own] == 7).all()
    y, L = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    aws = ex.workspace(ex.paged_workspace_size(ex.paged_shape(q, k, v, table)), "cuda")
    ex.fwd_paged(q, k, v, table, ln, 0.125, "causal", q_starts=st, y=y, L=L, ws=aws)
    s = np.minimum(np.maximum(starts, 0), b.T)
    n = np.minimum(np.maximum(lens, 0), b.table.shape[1] * b.page)
    fits = np.array_equal(s, starts) and np.array_equal(n, lens)  # else fewer keys than tokens: an empty row
    assert ex.device_status(aws) == (5 if fits else 8)
    ref = oracle.attend(b.np(b.q), kr, vr, b.table, n, s, 0.125, "causal")
    check_attention("bf16", y, L, ref, 64, int(n.max()))
    return k


@pytest.mark.parametrize("starts", [[0, 2, 1000], [-7, 2, 4], [-1, 2, 2 ** 31 - 1], [-2 ** 31, 2, 5]])
def test_token_ranges_that_reach_outside_the_tokens(ex, starts):
    b = Batch([40, 60], [2, 2], 4, 2, 64, 64, "bf16", 16, seed=81)
    k = _append_and_attend(ex, b, starts, [40, 60])
    at = int(b.table[1, 3])  # the last two keys of the second sequence are the last two tokens'
    assert torch.equal(k[at, :, 58 % 16:60 % 16].transpose(0, 1), b.k_new[2:].cuda())


@pytest.mark.parametrize("lens", [[65, 60], [66, 60], [64, 1], [2 ** 31 - 1, 60]])
def test_lengths_that_reach_outside_the_cache(ex, lens):
    """A token that stands behind the table, or before position 0, is written nowhere: no cached
    key makes room for it.  Tokens of the same sequence that have a place are written."""
    b = Batch([64, 60], [3, 2], 4, 2, 64, 64, "bf16", 16, seed=82)
    b.table = b.table[:, :4].copy()  # full for the first sequence
    _append_and_attend(ex, b, [0, 3, 5], lens)

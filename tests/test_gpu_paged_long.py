"""Sequences of many row tiles: a worker's start among them, and what finding it costs."""
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


def _part(b, rows):
    """b's queries of the tokens `rows`, each a sequence of its own that ends at its token."""
    q = b.np(b.q)[rows]
    owner = np.searchsorted(b.starts, rows, side="right") - 1
    pos = b.lens[owner] - np.diff(b.starts)[owner] + rows - b.starts[owner]
    return q, b.table[owner], pos


# Around 32 and 1024 row tiles of 4, 8, 16 and 256 rows, one sequence or several, long ones among short.
@pytest.mark.parametrize("nqs", [[513], [4100], [130, 2, 0, 700, 1, 260], [16500, 40]], ids=str)
@pytest.mark.parametrize("dtype,G,d,v,mask,window", [
    ("bf16", 1, 64, 64, "causal", 0), ("bf16", 4, 64, 64, "window", 40), ("f32", 2, 64, 64, "window", 33),
    ("f32", 1, 96, 64, "causal", 0), ("f32", 2, 64, 64, "none", 0), ("bf16", 2, 160, 136, "window", 20)])
def test_long_prompts(ex, path, dtype, G, d, v, mask, window, nqs):
    """Every token's row is written, and a sample of them is the oracle's."""
    lens = [n + x for n, x in zip(nqs, (50, 1, 0, 300, 7, 0))]
    b = Batch(lens, nqs, G, 1, d, v, dtype, 32, seed=71)
    q, k, vv, table, ln, starts = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts")
    y = torch.full((b.T, G, v), 7.0, dtype=q.dtype, device="cuda")
    L = torch.full((b.T, G), float("nan"), device="cuda")
    ws = ex.workspace(ex.paged_workspace_size(ex.paged_shape(q, k, vv, table)), "cuda")
    ex.fwd_paged(q, k, vv, table, ln, 0.1, mask, window, q_starts=starts, y=y, L=L, ws=ws)
    assert ex.device_status(ws) == 0 and torch.isfinite(L).all() and torch.isfinite(y).all()
    rows = np.unique(np.concatenate((np.linspace(0, b.T - 1, 150).astype(int), b.starts[:-1][np.diff(b.starts) > 0],
                                     b.starts[1:][np.diff(b.starts) > 0] - 1)))
    rows = rows if mask == "window" else rows[:: 1 + len(rows) // 40]
    qs, tables, pos = _part(b, rows)
    end = pos + 1 if mask != "none" else b.lens[np.searchsorted(b.starts, rows, side="right") - 1]
    ref = oracle.attend(qs, b.np(b.k_pages), b.np(b.v_pages), tables, end, np.arange(len(rows) + 1), 0.1,
                        mask, window)
    bits = 21 if dtype == "f32" else 8 if path == "auto" and d <= 128 else 16
    at = torch.from_numpy(rows).cuda()
    check_attention(dtype, y[at], L[at], ref, d, min(max(lens), window or max(lens)), bits)


@pytest.mark.parametrize("dtype,G,mask", [("f32", 2, "none"), ("f32", 2, "causal"), ("bf16", 8, "none")])
def test_many_tokens_behind_a_prefix(ex, path, dtype, G, mask):
    """All tokens over the prefix are one sequence: thousands of row tiles over a few keys."""
    n, B, P = 4000, 250, 45
    b = Batch([20] * B, [n // B] * B, G, 1, 64, 64, dtype, 16, seed=72, prefix=P)
    q, k, v, table, ln, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "prefix_table")
    y, L = torch.full_like(q, 7.0), torch.full((n, G), float("nan"), device="cuda")
    ws = ex.workspace(ex.prefix_workspace_size(ex.paged_shape(q, k, v, table)), "cuda")
    ex.fwd_prefix(q, k, v, pt, P, table, ln, 0.1, mask, y=y, L=L, ws=ws)
    assert ex.device_status(ws) == 0 and torch.isfinite(L).all() and torch.isfinite(y).all()
    rows = np.linspace(0, n - 1, 120).astype(int)
    qs, tables, pos = _part(b, rows)
    end = pos + 1 if mask != "none" else np.full(len(rows), 20)
    ref = oracle.attend(qs, b.np(b.k_pages), b.np(b.v_pages), tables, end, np.arange(len(rows) + 1), 0.1, mask,
                        prefix=(b.prefix_table, P))
    at = torch.from_numpy(rows).cuda()
    bits = 21 if dtype == "f32" else 8 if path == "auto" else 16
    check_attention(dtype, y[at], L[at], ref, 64, P + 20, bits, extra=2.0 ** -20)


@pytest.mark.parametrize("dtype,mask,window,limit", [("f32", "none", 0, 2.0), ("f32", "window", 64, 2.0)])
def test_one_long_sequence_costs_what_many_short_ones_do(ex, dtype, mask, window, limit):
    """65536 tokens over 64 keys each, as one sequence and as 64: the same rows and products (1024
    of the tokens in all have fewer keys), so finding a worker's start must not count.  With one
    lane walking over all row tiles it took 13 and 10 times as long."""
    T, G, d, page = 65536, 4, 64, 64
    t = {}
    for B in (1, 64):
        n = 64 if mask == "none" else T // B
        pages = -(-n // page)
        q = torch.randn(T, G, d, device="cuda")
        k, v = (torch.randn(B * pages, 1, page, d, device="cuda") for _ in range(2))
        table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        y, L = torch.empty_like(q), torch.empty(T, G, device="cuda")
        ws = ex.workspace(ex.paged_workspace_size(ex.paged_shape(q, k, v, table)), "cuda")
        best = []
        for _ in range(12):
            e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            e0.record()
            ex.fwd_paged(q, k, v, table, lens, 0.125, mask, window, y=y, L=L, ws=ws)
            e1.record()
            torch.cuda.synchronize()
            best.append(e0.elapsed_time(e1))
        t[B] = min(best[2:])
    assert t[1] <= limit * t[64], t

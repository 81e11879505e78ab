"""Attention behind a long prefix of 8-bit pages where the two launches are of different kernels:
17 to 32 rows of all tokens take 16-row tiles over a prefix of 2^17 keys of all key heads and more,
while the sequences' own keys, in short tables, take the 256-row tiles."""
import numpy as np
import pytest
import torch

from e4m3_inputs import Batch8
from test_gpu_paged_e4m3 import _behind, _check, ex, path  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

# (prefix, lens, nqs, H, kv, d, v, page, mask, pad).  2^17 / 8 key heads = 16384 keys.
CASES = [
    (16384, [3], [3], 64, 8, 64, 64, 16, "causal", 0),
    (16383, [3], [3], 64, 8, 64, 64, 16, "causal", 0),  # one key below: 256-row tiles for both, in one launch
    (16385, [200], [4], 64, 8, 128, 96, 64, "none", 2),
    (16384, [40, 1], [2, 1], 72, 8, 64, 64, 8, "causal", 0),  # two sequences, 27 rows in all
    (16400, [40, 0], [3, 0], 72, 8, 64, 128, 128, "causal", 1),
    (8192, [700], [2], 160, 16, 64, 64, 32, "causal", 0),
    (16384, [5], [4], 64, 8, 64, 64, 4, "causal", 0),  # pages too small for the 256-row tiles
    (16384, [5], [2], 128, 8, 64, 64, 16, "causal", 1),  # 32 rows
    (16384, [5], [3], 88, 8, 64, 64, 16, "causal", 0),  # 33: 256-row tiles
]


def _batch(case):
    prefix, lens, nqs, H, kv, d, v, page, mask, pad = case
    b = Batch8(lens, nqs, H, kv, d, v, "bf16", page, seed=CASES.index(case) + 400, pad=pad, prefix=prefix)
    if pad:
        b.q[-pad:] = float("nan")
    return b


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_long_prefixes_of_few_rows(ex, path, case):  # noqa: F811
    prefix, mask, pad = case[0], case[8], case[9]
    b = _batch(case)
    y, L, status = _behind(ex, b, prefix, mask, 0.02)
    assert status == 0
    _check(path, b, y, L, 0.02, mask, prefix=(b.prefix_table, prefix), extra=2.0 ** -20)
    if pad:
        assert (y[-pad:] == 7).all() and (L[-pad:] == 7).all()


@pytest.mark.parametrize("case", [CASES[0], CASES[3]], ids=["one", "two"])
def test_they_repeat_themselves(ex, case):  # noqa: F811
    """Whatever the workspace held, on a stream of its own, and from a captured graph."""
    prefix, mask = case[0], case[8]
    b = _batch(case)
    k, v, table, lens, starts, ks, vs = b.cache()
    q, pt = b.dev("q", "prefix_table")
    size = ex.prefix_workspace_size(ex.paged_shape(q, k, v, table))
    kw = dict(q_starts=starts, k_scales=ks, v_scales=vs)
    want = ex.fwd_prefix(q, k, v, pt, prefix, table, lens, 0.02, mask, **kw)
    side = torch.cuda.Stream()
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        got = ex.fwd_prefix(q, k, v, pt, prefix, table, lens, 0.02, mask, ws=ws, stream=side, **kw)
        torch.cuda.synchronize()
        assert ex.device_status(ws) == 0
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    y, L = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ex.fwd_prefix(q, k, v, pt, prefix, table, lens, 0.02, mask, y=y, L=L, ws=ws, **kw)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(L, want[1])
    assert np.isfinite(want[1].cpu().numpy()).all()

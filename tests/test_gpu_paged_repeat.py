"""A call gives the same bits every time, whatever its workspace held before."""
import pytest
import torch

from paged_inputs import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import exact_tiled_softmax_gb300 as mod
    mod.load_library()
    assert torch.cuda.is_available()
    return mod


# (lens, nqs, H, kv, d, v, dtype, page, prefix): tiles of every size, finished and shared, one launch and two.
CASES = [
    ([1000], [1], 8, 2, 128, 128, "bf16", 16, 0),
    ([5000, 30, 2000], [2, 1, 4], 16, 4, 64, 96, "bf16", 32, 0),
    ([900, 1400], [200, 300], 8, 2, 128, 128, "bf16", 64, 0),
    ([3000, 10], [2, 3], 4, 2, 80, 96, "f32", 16, 0),
    ([2000], [40], 4, 2, 128, 128, "f32", 16, 0),
    ([1500], [2], 4, 2, 256, 192, "bf16", 16, 0),
    ([40, 1, 90, 17] * 4, [1] * 16, 32, 8, 128, 128, "bf16", 64, 4001),
    ([20, 77, 5], [1, 2, 1], 8, 4, 80, 96, "f32", 32, 3001),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c))[:50].replace(" ", ""))
def test_calls_repeat_themselves(ex, case):
    lens, nqs, H, kv, d, v, dtype, page, prefix = case
    b = Batch(lens, nqs, H, kv, d, v, dtype, page, seed=95, prefix=prefix)
    q, k, vv, table, ln, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
    shape = ex.paged_shape(q, k, vv, table)
    size = ex.prefix_workspace_size(shape) if prefix else ex.paged_workspace_size(shape)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    seen = []
    for fill in (0xFF, 0x00, 0x3C, None, None):  # None: as the call before left it
        if fill is not None:
            ws.fill_(fill)
        if prefix:
            y, L = ex.fwd_prefix(q, k, vv, pt, prefix, table, ln, 0.1, "causal", q_starts=starts, ws=ws)
        else:
            y, L = ex.fwd_paged(q, k, vv, table, ln, 0.1, "causal", q_starts=starts, ws=ws)
        assert ex.device_status(ws) == 0
        seen.append((y, L))
    for y, L in seen[1:]:
        assert torch.equal(y, seen[0][0]) and torch.equal(L, seen[0][1])

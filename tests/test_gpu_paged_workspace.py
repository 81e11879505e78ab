"""What a call needs of its workspace goes by its pages' type: over pages of the inputs' type, heads of
129 to 256 columns need what they did before there were pages in 8 bits."""
import ctypes

import pytest
import torch

from paged_inputs import Batch, check_attention
from oracle import paged as oracle

SHAPE = dict(batch=2, tokens=4, heads=16, kv_heads=4, d=256, v=256, dtype=1, page_size=16, num_pages=50, max_pages=10,
             q_stride=0, k_stride=0, v_stride=0)
# (d, v) -> bytes of attn_fwd_paged, bytes of attn_fwd_prefix without the 2 x tokens x heads rows that it joins: over
# pages of the inputs' type, and over pages in 8 bits (0: these do not exist).
NEEDS = {(256, 256): (3780608, 7552768, 15081984, 30155520), (200, 200): (2963456, 5918464, 0, 0),
         (208, 208): (3080192, 6151936, 12280320, 24552192), (144, 32): (512000, 1015552, 2007552, 4006656)}


@pytest.fixture(scope="module")
def lib():
    import os

    import exact_tiled_softmax_gb300 as ex
    if not os.path.exists(ex.library_path()):
        from exact_tiled_softmax_gb300 import build
        build.build()
    return ex.load_library()


def _joined(s):
    rows, up = s["tokens"] * s["heads"], lambda x: (x + 255) // 256 * 256  # noqa: E731
    return up(4 * 2 * rows * s["v"]) + up(4 * 2 * rows) + up(8 * 2 * rows) + 256


@pytest.mark.parametrize("d,v", NEEDS)
@pytest.mark.parametrize("dtype", [0, 1])
def test_a_call_needs_what_its_pages_take(lib, d, v, dtype):
    """The queries cover every type of pages that the widths allow; a call is refused below its own need alone."""
    import exact_tiled_softmax_gb300 as ex
    p, ws = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)  # never dereferenced
    f = {**SHAPE, "d": d, "v": v, "dtype": dtype}
    s = ctypes.byref(ex.PagedShape(**f))
    paged, prefix, paged8, prefix8 = NEEDS[d, v]
    assert lib.exattn_paged_workspace_size(s) == max(paged, paged8)
    assert lib.exattn_prefix_workspace_size(s) == max(prefix, prefix8) + _joined(f)
    assert lib.attn_fwd_paged(s, p, p, p, p, p, p, 1.0, 0, 0, p, p, ws, paged - 1, None) == 4
    assert lib.attn_fwd_prefix(s, p, p, p, p, 5, p, p, p, 1.0, 0, p, p, ws, prefix + _joined(f) - 1, None) == 4
    refused = 4 if paged8 else 2
    assert lib.attn_fwd_paged_e4m3(s, p, p, p, p, p, p, p, p, 1.0, 0, 0, p, p, ws, (paged8 or 1 << 40) - 1, None) == refused
    assert lib.attn_fwd_prefix_e4m3(s, p, p, p, p, p, p, 5, p, p, p, 1.0, 0, p, p, ws, (prefix8 or 1 << 40) + _joined(f) - 1,
                                    None) == refused


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,v", NEEDS)
def test_workspaces_of_just_that_size(lib, d, v, dtype):
    """Calls over pages of the inputs' type, whose workspaces are followed by bytes that stay as they were."""
    import exact_tiled_softmax_gb300 as ex
    b = Batch([150, 33], [2, 2], 16, 4, d, v, dtype, 16, seed=d, prefix=70)
    names = ("k_pages", "v_pages", "table", "lens", "starts", "q", "prefix_table")
    k, vv, table, lens, starts, q, pt = b.dev(*names)
    need, joined = NEEDS[d, v], _joined({**SHAPE, "v": v})
    for prefix, size in ((0, need[0]), (70, need[1] + joined)):
        whole = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        ws = whole[:size]
        if prefix:
            y, L = ex.fwd_prefix(q, k, vv, pt, prefix, table, lens, 0.02, "causal", q_starts=starts, ws=ws)
        else:
            y, L = ex.fwd_paged(q, k, vv, table, lens, 0.02, "causal", q_starts=starts, ws=ws)
        assert ex.device_status(ws) == 0 and (whole[size:] == 0x5A).all()
        ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.02, "causal", 0,
                            (b.prefix_table, prefix) if prefix else None)
        check_attention(dtype, y, L, ref, d, 220, extra=2.0 ** -20)

"""How many bits of probabilities and values reach Y in each paged kernel, on inputs whose
roundings all fall to the same side, so that a part that is left out shows far above the
bounds of check_attention."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as oracle
from paged_inputs import Batch, check_attention

gpu = pytest.mark.gpu


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


def p_bits(path, dtype, d, v, page, tokens, batch, group, kv, prefix=0):
    """Bits of p that P.V keeps (see check_attention) by the library's choice of a kernel: the
    256-row tiles round p to bf16, everything else keeps its remainder.  Behind a prefix they are
    taken where a sequence's own tokens already have more than 16 rows to a key head, or all tokens
    together do and 16-row tiles would read the prefix again for 40 MB or more."""
    if dtype == "f32":
        return 21
    if path == "simt" or max(d, v) > 128 or page < 8:
        return 16
    rows = -(-tokens // batch) * group
    if prefix and rows <= 16 and tokens * group > 16:
        again = (tokens * group + 15) // 16 - 1
        return 8 if again * prefix * kv * (d + v) * 2 >= 40e6 else 16
    return 8 if rows > 16 else 16


class Sided(Batch):
    """Keys of two kinds, three to four: scores 0 and ln(p).  p lies just below the middle of two
    neighbouring bf16 (tf32) values, and so do fp32 values, with c = 1 + 2^-11 - 2^-23.  Even columns of V
    are c; odd ones c and -c by kind, so that Y is all but 0 there and keeps what is left out of p."""

    def __init__(self, lens, nqs, H, kv, d, v, dtype, page, **kw):
        super().__init__(lens, nqs, H, kv, d, v, dtype, page, **kw)
        self.p = 0.75 + 0.98 * 2.0 ** (-9 if dtype == "bf16" else -12)
        self.scale = -math.log(self.p)
        c = 1.0 if dtype == "bf16" else 1 + 2.0 ** -11 - 2.0 ** -23
        full = ~torch.isnan(self.k_pages[:, :, :, :1])
        num = full.shape[0] * page
        kind = (torch.arange(num) % 7 < 3).view(-1, 1, page, 1)  # of score 0
        k = torch.zeros_like(self.k_pages)
        k[..., :1] = torch.where(kind, 0.0, -1.0).to(k.dtype)
        odd = (torch.arange(v) % 2).bool()
        vv = torch.where(odd & ~kind, -c, c).to(k.dtype).expand(self.v_pages.shape)
        self.k_pages = torch.where(full, k, self.k_pages)
        self.v_pages = torch.where(full, vv, self.v_pages)
        self.q = torch.zeros_like(self.q)
        self.q[..., 0] = 1

    def reference(self, mask, window=0):
        with np.errstate(invalid="ignore"):
            return oracle.attend(self.np(self.q), self.np(self.k_pages), self.np(self.v_pages), self.table, self.lens,
                                 self.starts, self.scale, mask, window,
                                 prefix=(self.prefix_table, self.prefix) if self.prefix else None)


def _nearest(x, bits):
    """x rounded to so many significant bits (x in [0.5, 2))."""
    step = 2.0 ** (np.floor(np.log2(x)) + 1 - bits)
    return np.round(x / step) * step


@pytest.mark.parametrize("dtype,n,mask,window", [("bf16", 138, "none", 0), ("bf16", 60, "causal", 0),
                                                 ("f32", 138, "none", 0), ("f32", 700, "window", 333)])
def test_what_is_left_out_would_show(dtype, n, mask, window):
    """On the CPU: with p, or fp32 values, cut to their first part, the result is outside the
    bounds that the kernels are held to."""
    b = Sided([n], [2], 2, 1, 64, 64, dtype, 16, seed=90)
    ref = b.reference(mask, window)
    keys = min(n, window or n)
    bits = 16 if dtype == "bf16" else 21

    def result(p_first, v_first):
        y = np.zeros((2, 2, 64))
        at = b.table[0].astype(np.int64)
        for i in range(2):
            pos = n - 2 + i
            hi = n if mask == "none" else pos + 1
            j = np.arange(max(0, pos + 1 - window) if mask == "window" else 0, hi)
            p = np.where(b.np(b.k_pages)[at[j // 16], 0, j % 16, 0] == 0, 1.0, b.p)
            vv = b.np(b.v_pages)[at[j // 16], 0, j % 16]
            l = p.sum()
            if p_first:
                p = _nearest(p, 8 if dtype == "bf16" else 11)
            if v_first:
                vv = np.sign(vv) * _nearest(np.abs(vv), 11)
            y[i] = p @ vv / l
        return torch.from_numpy(y)

    L = torch.from_numpy(ref[1])
    check_attention(dtype, result(False, False), L, ref, 64, keys, bits)
    with pytest.raises(AssertionError):
        check_attention(dtype, result(True, False), L, ref, 64, keys, bits)
    if dtype == "f32":
        with pytest.raises(AssertionError):
            check_attention(dtype, result(False, True), L, ref, 64, keys, bits)


# (lens, nqs, H, kv, d, v, dtype, page, mask, window)
PAGED = [
    ([138], [1], 4, 1, 128, 128, "bf16", 16, "causal", 0),
    ([500, 90, 31], [2, 1, 3], 8, 2, 64, 64, "bf16", 16, "causal", 0),
    ([300, 200], [3, 3], 16, 4, 96, 80, "bf16", 32, "none", 0),         # 12 rows to a key head
    ([300, 200], [40, 40], 4, 2, 128, 128, "bf16", 64, "causal", 0),    # 256-row tiles
    ([400], [1], 2, 2, 256, 192, "bf16", 16, "causal", 0),
    ([90, 128, 3], [1, 2, 1], 4, 4, 80, 96, "f32", 16, "causal", 0),
    ([700, 1300], [2, 1], 16, 2, 128, 128, "f32", 32, "window", 333),
    ([90, 200], [33, 50], 3, 3, 112, 64, "f32", 128, "window", 20),
    ([200], [3], 8, 2, 64, 64, "f32", 8, "none", 0),
    ([150, 90], [3, 6], 4, 2, 192, 128, "f32", 16, "window", 64),
]


@gpu
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_parts_of_p_and_v_over_pages(ex, path, case):
    lens, nqs, H, kv, d, v, dtype, page, mask, window = case
    b = Sided(lens, nqs, H, kv, d, v, dtype, page, seed=91)
    q, k, vv, table, ln, starts = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts")
    ws = ex.workspace(ex.paged_workspace_size(ex.paged_shape(q, k, vv, table)), "cuda")
    y, L = ex.fwd_paged(q, k, vv, table, ln, b.scale, mask, window, q_starts=starts, ws=ws)
    assert ex.device_status(ws) == 0
    check_attention(dtype, y, L, b.reference(mask, window), d, min(max(lens), window or max(lens)),
                    p_bits(path, dtype, d, v, page, b.T, len(lens), H // kv, kv))


# (prefix, lens, nqs, H, kv, d, v, dtype, page, mask)
PREFIX = [
    (90, [12] * 40, [1] * 40, 16, 2, 128, 128, "bf16", 16, "causal"),            # 16-row tiles, 320 rows
    (37, [3 + x % 31 for x in range(200)], [1] * 200, 2, 1, 64, 64, "bf16", 16, "causal"),
    (100, [1 + x for x in range(33)], [x % 2 for x in range(33)], 4, 2, 64, 64, "bf16", 16, "causal"),
    (300, [5, 1, 40], [1, 1, 1], 8, 2, 128, 128, "bf16", 16, "causal"),
    (257, [20, 30], [20, 30], 8, 2, 64, 128, "bf16", 32, "none"),                 # 256-row tiles for both
    (2500, [40, 1, 90] * 6, [1] * 18, 32, 8, 128, 128, "bf16", 64, "causal"),     # 256-row tiles for the prefix
    (130, [7, 9], [1, 1], 2, 2, 200, 104, "bf16", 16, "causal"),
    (513, [40, 80], [2, 1], 4, 1, 80, 96, "f32", 32, "none"),
    (90, [12] * 20, [1] * 20, 8, 2, 128, 128, "f32", 16, "causal"),
]


@gpu
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: "-".join(map(str, c))[:60].replace(" ", ""))
def test_parts_of_p_and_v_behind_a_prefix(ex, path, case):
    prefix, lens, nqs, H, kv, d, v, dtype, page, mask = case
    b = Sided(lens, nqs, H, kv, d, v, dtype, page, seed=92, prefix=prefix)
    q, k, vv, table, ln, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
    ws = ex.workspace(ex.prefix_workspace_size(ex.paged_shape(q, k, vv, table)), "cuda")
    y, L = ex.fwd_prefix(q, k, vv, pt, prefix, table, ln, b.scale, mask, q_starts=starts, ws=ws)
    assert ex.device_status(ws) == 0
    # The two parts are joined by one more exponential each.
    check_attention(dtype, y, L, b.reference(mask), d, prefix + max(lens),
                    p_bits(path, dtype, d, v, page, b.T, len(lens), H // kv, kv, prefix), extra=2.0 ** -20)


@gpu
@pytest.mark.parametrize("B,dtype,prefix", [(1024, "bf16", 37), (1024, "f32", 37), (33, "bf16", 100), (129, "bf16", 100)])
def test_large_batches_behind_a_prefix(ex, path, B, dtype, prefix):
    """Status and precision by the kernel that the prefix takes, most sequences short."""
    rng = np.random.default_rng(B)
    nqs = [int(x) for x in rng.integers(0, 3, B)]
    lens = [int(rng.integers(0, 40)) + x for x in nqs]
    b = Batch(lens, nqs, 4, 2, 64, 64, dtype, 16, seed=B, prefix=prefix)
    ref = oracle.attend(b.np(b.q), b.np(b.k_pages), b.np(b.v_pages), b.table, b.lens, b.starts, 0.1, "causal",
                        prefix=(b.prefix_table, prefix))
    q, k, v, table, ln, starts, pt = b.dev("q", "k_pages", "v_pages", "table", "lens", "starts", "prefix_table")
    ws = ex.workspace(ex.prefix_workspace_size(ex.paged_shape(q, k, v, table)), "cuda")
    y, L = ex.fwd_prefix(q, k, v, pt, prefix, table, ln, 0.1, "causal", q_starts=starts, ws=ws)
    assert ex.device_status(ws) == 0
    bits = p_bits(path, dtype, 64, 64, 16, b.T, B, 2, 2, prefix)
    assert dtype == "f32" or bits == 16
    check_attention(dtype, y, L, ref, 64, prefix + max(lens), bits, extra=2.0 ** -20)

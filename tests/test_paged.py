"""The paged-cache operators without a GPU: the oracle's pins, refusals of the C ABI
and of the binding before anything is queued, workspace sizes."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import dense, masks
from oracle import paged as oracle


@pytest.fixture(scope="session")
def lib():
    import exact_tiled_softmax_gb300 as ex
    if not os.path.exists(ex.library_path()):
        from exact_tiled_softmax_gb300 import build
        build.build()
    return ex.load_library()


def _pool(lens, kv, d, v, page, seed=0):
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    perm = rng.permutation(sum(need) + 2)
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = perm[at:at + c]
        at += c
    k, vv = (rng.standard_normal((sum(need) + 2, kv, page, w)) for w in (d, v))
    return k, vv, table


@pytest.mark.parametrize("mask,window", [("none", 0), ("causal", 0), ("window", 5)])
def test_oracle_pages_equal_dense_attention(mask, window):
    lens, nqs, H, kv, d, v, page = [13, 30], [3, 4], 4, 2, 6, 5, 8
    k, vv, table = _pool(lens, kv, d, v, page)
    q = np.random.default_rng(1).standard_normal((7, H, d))
    starts = [0, 3, 7]
    Y, L, A, _ = oracle.attend(q, k, vv, table, lens, starts, 0.3, mask, window)
    kind = {"none": masks.NONE, "causal": masks.CAUSAL, "window": masks.WINDOW}[mask]
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        kk, vb = (oracle.keys_of(x, table[b], n)[0].repeat(H // kv, 0)[None] for x in (k, vv))
        qq = q[starts[b]:starts[b + 1]].transpose(1, 0, 2)[None]
        Yr, Lr = dense.forward_rect(qq, kk, vb, 0.3, kind, window)
        assert np.allclose(Y[starts[b]:starts[b + 1]], Yr[0].transpose(1, 0, 2), atol=1e-13)
        assert np.allclose(L[starts[b]:starts[b + 1]], Lr[0].T, atol=1e-13)
    assert (A >= np.abs(Y) - 1e-15).all()


def test_oracle_prefix_equals_one_long_sequence():
    P, lens, nqs, page = 11, [4, 9], [2, 1], 4
    k, vv, table = _pool(lens + [P], 1, 6, 6, page)
    q = np.random.default_rng(2).standard_normal((3, 2, 6))
    Y, L, _, _ = oracle.attend(q, k, vv, table[:2], lens, [0, 2, 3], 0.4, "causal", prefix=(table[2], P))
    for b, s in ((0, slice(0, 2)), (1, slice(2, 3))):
        kk, vb = (np.concatenate((oracle.keys_of(x, table[2], P)[0], oracle.keys_of(x, table[b], lens[b])[0]), 1)
                  .repeat(2, 0)[None] for x in (k, vv))
        Yr, Lr = dense.forward_rect(q[s].transpose(1, 0, 2)[None], kk, vb, 0.4, masks.CAUSAL)
        assert np.allclose(Y[s], Yr[0].transpose(1, 0, 2), atol=1e-13)
        assert np.allclose(L[s], Lr[0].T, atol=1e-13)


def test_oracle_rotation_keeps_relative_positions():
    """<rot(q, m), rot(k, n)> depends on m - n alone; a quarter turn swaps a pair."""
    rng = np.random.default_rng(3)
    inv = np.array([1.0, 0.1, 0.01])
    for inter in (False, True):
        q, k = rng.standard_normal(8), rng.standard_normal(8)
        a = oracle.rotate(q, 7, inv, inter) @ oracle.rotate(k, 3, inv, inter)
        b = oracle.rotate(q, 1007, inv, inter) @ oracle.rotate(k, 1003, inv, inter)
        assert abs(a - b) < 1e-9
    assert np.allclose(oracle.rotate(np.array([1.0, 2.0, 5.0, 6.0]), 1, [np.pi / 2], True), [-2, 1, 5, 6])
    assert np.allclose(oracle.rotate(np.array([1.0, 2.0, 5.0, 6.0]), 1, [np.pi / 2, 0], False), [-5, 2, 1, 6])


def test_oracle_append_places_tokens():
    k, v, table = _pool([9, 5], 1, 4, 4, 4, seed=5)
    kn, vn = np.ones((3, 1, 4)), np.full((3, 1, 4), 2.0)
    _, kp, vp = oracle.append(kn, vn, k, v, table, [9, 5], [0, 2, 3])
    for b, pos in ((0, 7), (0, 8), (1, 4)):
        assert (kp[table[b][pos // 4], 0, pos % 4] == 1).all()
        assert (vp[table[b][pos // 4], 0, pos % 4] == 2).all()
    assert (kp != k).any(-1).sum() == 3


GOOD = dict(batch=4, tokens=8, heads=8, kv_heads=2, d=64, v=64, dtype=1, page_size=16, num_pages=50,
            max_pages=10, q_stride=0, k_stride=0, v_stride=0)

BAD_SHAPES = [
    (dict(batch=0), 1), (dict(tokens=0), 1), (dict(heads=0), 1), (dict(kv_heads=0), 1),
    (dict(heads=7), 1), (dict(d=0), 1), (dict(v=-8), 1), (dict(dtype=2), 1), (dict(page_size=0), 1),
    (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(q_stride=8), 1), (dict(k_stride=-8), 1),
    (dict(v_stride=64), 1), (dict(d=264), 2), (dict(v=512), 2), (dict(d=68), 2), (dict(dtype=0, v=66), 2),
    (dict(page_size=24), 2), (dict(page_size=2048), 2), (dict(batch=1025, tokens=2050), 2),
    (dict(tokens=1 << 21), 2), (dict(max_pages=1 << 27), 2), (dict(tokens=1 << 20, heads=4096), 2),
    (dict(tokens=972592, heads=2208), 2), (dict(heads=65536 * 2), 2),
    (dict(q_stride=516), 3), (dict(k_stride=130), 3), (dict(v_stride=129), 3),
]


@pytest.mark.parametrize("edit,status", BAD_SHAPES, ids=lambda x: str(x))
def test_shapes_that_the_library_refuses(lib, edit, status):
    import exact_tiled_softmax_gb300 as ex
    p = ctypes.c_void_p(1 << 20)  # never dereferenced
    s = ctypes.byref(ex.PagedShape(**{**GOOD, **edit}))
    assert lib.exattn_paged_workspace_size(s) == 0 and lib.exattn_prefix_workspace_size(s) == 0
    big = 1 << 40
    assert lib.attn_fwd_paged(s, p, p, p, p, p, p, 1.0, 0, 0, p, p, p, big, None) == status
    assert lib.attn_fwd_prefix(s, p, p, p, p, 5, p, p, p, 1.0, 0, p, p, p, big, None) == status
    assert lib.attn_append_paged(s, p, p, p, p, p, p, p, 4, 0, 0, p, p, p, p, big, None) == status


def test_arguments_that_the_library_refuses(lib):
    import exact_tiled_softmax_gb300 as ex
    p, odd, ws = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8), ctypes.c_void_p(1 << 21)
    odd2 = ctypes.c_void_p((1 << 20) + 2)
    s = ctypes.byref(ex.PagedShape(**GOOD))
    big = 1 << 40

    def paged(q=p, k=p, v=p, t=p, n=p, st=p, mask=0, win=0, y=p, L=p, w=ws, size=big, shape=s):
        return lib.attn_fwd_paged(shape, q, k, v, t, n, st, 1.0, mask, win, y, L, w, size, None)

    for name in ("q", "k", "v", "t", "n", "y", "L", "w"):
        assert paged(**{name: None}) == 1, name
    for name in ("q", "k", "v", "y", "L", "w"):
        assert paged(**{name: odd}) == 3, name
    for name in ("t", "n", "st"):
        assert paged(**{name: odd2}) == 3, name
    assert paged(shape=None) == 1
    assert paged(mask=7) == 1 and paged(mask=-1) == 1 and paged(mask=2, win=0) == 1
    assert paged(mask=3) == 2
    assert paged(size=lib.exattn_paged_workspace_size(s) - 1) == 4
    uneven = ctypes.byref(ex.PagedShape(**{**GOOD, "tokens": 9}))
    assert paged(shape=uneven, st=None) == 1

    def prefix(pt=p, n=5, mask=0, w=ws, size=big, q=p, shape=s):
        return lib.attn_fwd_prefix(shape, q, p, p, pt, n, p, p, p, 1.0, mask, p, p, w, size, None)

    assert prefix(pt=None) == 1 and prefix(n=-1) == 1 and prefix(q=None) == 1 and prefix(shape=None) == 1
    assert prefix(mask=2) == 2 and prefix(mask=3) == 2 and prefix(mask=9) == 1
    assert prefix(pt=odd2) == 3 and prefix(n=1 << 30) == 2
    assert prefix(size=lib.exattn_prefix_workspace_size(s) - 1) == 4

    def append(q=p, k=p, v=p, t=p, n=p, st=p, f=p, pairs=4, off=0, qo=p, kp=p, vp=p, w=ws, size=big, shape=s):
        return lib.attn_append_paged(shape, q, k, v, t, n, st, f, pairs, 0, off, qo, kp, vp, w, size, None)

    for name in ("k", "v", "t", "n", "f", "qo", "kp", "vp", "w"):
        assert append(**{name: None}) == 1, name
    for name in ("q", "k", "v", "qo", "kp", "vp", "w"):
        assert append(**{name: odd}) == 3, name
    for name in ("t", "n", "st", "f"):
        assert append(**{name: odd2}) == 3, name
    assert append(pairs=33) == 1 and append(pairs=-1) == 1 and append(off=-1) == 1 and append(shape=None) == 1
    assert append(size=255) == 4
    assert append(shape=uneven, st=None) == 1


def test_packed_calls_reach_the_same_checks(lib):
    """The binding's packed structure has the C layout: each operation's own refusals."""
    import exact_tiled_softmax_gb300 as ex
    p, big = 1 << 20, 1 << 40

    def run(op, shape=GOOD, **edit):
        f = dict(q=p, k=p, v=p, kp=p, vp=p, t=p, n=p, st=p, pt=p, inv=p, y=p, L=p, w=p, size=big, s=0,
                 scale=1.0, mask=0, win=0, plen=5, pairs=4, inter=0)
        f.update(edit)
        return lib.exattn_paged_run(op, ex._PAGED_CALL.pack(*shape.values(), *f.values()))

    assert ex._PAGED_CALL.size == 208
    assert run(3) == 1 and lib.exattn_paged_run(1, None) == 1
    for op in range(3):
        assert run(op, {**GOOD, "page_size": 24}) == 2
        assert run(op, kp=p + 8) == 3 and run(op, y=p + 8) == 3 and run(op, w=p + 128) == 3
        assert run(op, size=8) == 4 and run(op, n=0) == 1 and run(op, st=p + 2) == 3
    assert run(0, pairs=33) == 1 and run(0, plen=-1) == 1 and run(0, inv=p + 2) == 3 and run(0, v=0) == 1
    for op in (1, 2):
        assert run(op, L=0) == 1 and run(op, mask=3) == 2 and run(op, mask=-2) == 1
    assert run(1, mask=2, win=0) == 1 and run(2, plen=-1) == 1 and run(2, pt=0) == 1


def test_workspace_does_not_grow_with_the_cache(lib):
    import exact_tiled_softmax_gb300 as ex
    size = lambda **e: ex.paged_workspace_size(ex.PagedShape(**{**GOOD, **e}))  # noqa: E731
    assert 0 < size() == size(num_pages=10 ** 6, max_pages=10 ** 6)
    assert ex.prefix_workspace_size(ex.PagedShape(**GOOD)) >= size() + 8 * 8 * 4 * 65


def _args(**edit):
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k_pages=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16),
             v_pages=torch.zeros(5, 2, 16, 32, dtype=torch.bfloat16),
             page_table=torch.zeros(3, 4, dtype=torch.int32), seq_lens=torch.ones(3, dtype=torch.int32),
             scale=1.0)
    a.update(edit)
    return a


I32 = dict(dtype=torch.int32)


@pytest.mark.parametrize("edit,match", [
    (dict(q=torch.zeros(3, 4, 32, dtype=torch.bfloat16)), "q has shape"),
    (dict(q=torch.zeros(3, 4, 64)), "dtype mismatch"),
    (dict(q=torch.zeros(3, 4, 64, dtype=torch.float16)), "unsupported dtype"),
    (dict(q=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "dense within a token"),
    (dict(q=torch.zeros(1, 4, 64, dtype=torch.bfloat16).expand(3, 4, 64)), "overlap"),
    (dict(q=torch.zeros(4, 64, dtype=torch.bfloat16)), "expected q"),
    (dict(q=torch.zeros(4, 4, 64, dtype=torch.bfloat16)), "do not divide"),
    (dict(k_pages=torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)), "contiguous"),
    (dict(v_pages=torch.zeros(5, 2, 32, 32, dtype=torch.bfloat16)), "before the width"),
    (dict(page_table=torch.zeros(3, 4, dtype=torch.int64)), "page_table"),
    (dict(page_table=torch.zeros(3, 8, **I32)[:, ::2]), "page_table"),
    (dict(page_table=torch.zeros(4, **I32)), "expected q"),
    (dict(seq_lens=torch.ones(2, **I32)), "seq_lens"),
    (dict(seq_lens=torch.ones(3)), "seq_lens"),
    (dict(q_starts=torch.zeros(3, **I32)), "q_starts"),
    (dict(y=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), "y must be"),
    (dict(y=torch.zeros(3, 4, 32)), "y must be"),
    (dict(L=torch.zeros(3, 4, dtype=torch.bfloat16)), "L must be"),
    (dict(L=torch.zeros(4, 3)), "L must be"),
    (dict(ws=torch.zeros(1 << 24, dtype=torch.uint8)[::2]), "workspace"),
    (dict(window=1 << 31), "32 bits"),
    (dict(), "CUDA device"),
], ids=lambda x: str(x)[:40] if isinstance(x, str) else "")
def test_tensors_that_fwd_paged_refuses(lib, edit, match):
    import exact_tiled_softmax_gb300 as ex
    with pytest.raises(ValueError, match=match):
        ex.fwd_paged(**_args(**edit))


@pytest.mark.parametrize("edit,match", [
    (dict(prefix_table=torch.zeros(2, dtype=torch.int64)), "prefix_table"),
    (dict(prefix_table=torch.zeros(1, 2, **I32)), "prefix_table"),
    (dict(prefix_len=33), "the prefix has 33"),
    (dict(prefix_len=1 << 40), "32 bits"),
    (dict(seq_lens=torch.ones(1, **I32)), "seq_lens"),
    (dict(), "CUDA device"),
], ids=lambda x: str(x)[:40] if isinstance(x, str) else "")
def test_tensors_that_fwd_prefix_refuses(lib, edit, match):
    import exact_tiled_softmax_gb300 as ex
    with pytest.raises(ValueError, match=match):
        ex.fwd_prefix(**{**_args(), "prefix_table": torch.zeros(2, **I32), "prefix_len": 32, **edit})


@pytest.mark.parametrize("edit,match", [
    (dict(k=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), "k has shape"),
    (dict(k=torch.zeros(3, 2, 64)), "must be torch.bfloat16"),
    (dict(v=torch.zeros(3, 2, 64, dtype=torch.bfloat16)), "v has shape"),
    (dict(v=torch.zeros(2, 2, 32, dtype=torch.bfloat16)), "as many tokens"),
    (dict(q=None), "CUDA device"),
    (dict(q=None, q_out=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), "q_out without q"),
    (dict(q_out=torch.zeros(2, 4, 64, dtype=torch.bfloat16)), "q_out"),
    (dict(q_out=torch.zeros(3, 4, 64)), "q_out"),
    (dict(inv_freq=torch.zeros(8, dtype=torch.float64)), "inv_freq"),
    (dict(inv_freq=torch.zeros(2, 4)), "inv_freq"),
    (dict(pos_offset=1 << 31), "32 bits"),
    (dict(), "CUDA device"),
], ids=lambda x: str(x)[:40] if isinstance(x, str) else "")
def test_tensors_that_append_paged_refuses(lib, edit, match):
    import exact_tiled_softmax_gb300 as ex
    a = _args()
    del a["scale"]
    a.update(k=torch.zeros(3, 2, 64, dtype=torch.bfloat16), v=torch.zeros(3, 2, 32, dtype=torch.bfloat16))
    a.update(edit)
    with pytest.raises(ValueError, match=match):
        ex.append_paged(**a)

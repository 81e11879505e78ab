"""The paged cache in 8 bits without a GPU: the oracle's pins, refusals of the C ABI and of the
binding before anything is queued."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import e4m3


@pytest.fixture(scope="session")
def lib():
    import exact_tiled_softmax_gb300 as ex
    if not os.path.exists(ex.library_path()):
        from exact_tiled_softmax_gb300 import build
        build.build()
    return ex.load_library()


def test_oracle_numbers_are_those_of_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    assert np.array_equal(e4m3.NUMBERS, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)


def test_oracle_rounds_as_torch_does():
    """Within 448, where torch's conversion rounds to nearest, ties to even."""
    x = np.random.default_rng(0).uniform(-448, 448, (50, 64)).astype(np.float32)
    x[:, 0] = 448  # the exponent is 127
    x[:, 1:20] = np.random.default_rng(1).choice(e4m3.BORDERS, (50, 19))
    codes, byte = e4m3.quantise(x)
    assert (byte == 127).all()
    assert np.array_equal(codes, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_exponents():
    """The smallest for which nothing saturates, from 1 on; 0 for rows of zeros."""
    for top, byte in ((448.0, 127), (448.0001, 128), (224.0, 126), (225.0, 127), (1.0, 119), (0.0, 0), (2.0 ** -140, 1),
                      (1.75 * 2.0 ** 100, 127 + 92), (1.7500001 * 2.0 ** 100, 127 + 93), (3.4e38, 127 + 120)):
        assert e4m3.exponent(top) == byte, top
    x = np.random.default_rng(2).standard_normal((200, 32)) * 2.0 ** np.random.default_rng(3).integers(-100, 100, (200, 1))
    codes, byte = e4m3.quantise(x)
    unit = 2.0 ** (byte.astype(float) - 127)[:, None]
    assert (np.abs(x) <= 448 * unit).all() and (np.abs(x).max(-1) > 224 * unit[:, 0]).all()
    assert (np.abs(e4m3.values(codes, byte) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * unit)).all()


GOOD = dict(batch=4, tokens=8, heads=8, kv_heads=2, d=64, v=64, dtype=1, page_size=16, num_pages=50,
            max_pages=10, q_stride=0, k_stride=0, v_stride=0)


@pytest.mark.parametrize("edit,status", [
    (dict(batch=0), 1), (dict(heads=7), 1), (dict(dtype=2), 1), (dict(d=264), 2), (dict(d=72), 2), (dict(v=8), 2),
    (dict(dtype=0, v=68), 2), (dict(page_size=24), 2), (dict(tokens=1 << 21), 2), (dict(q_stride=516), 3)],
    ids=lambda x: str(x))
def test_shapes_that_the_library_refuses(lib, edit, status):
    import exact_tiled_softmax_gb300 as ex
    p = ctypes.c_void_p(1 << 20)  # never dereferenced
    s = ctypes.byref(ex.PagedShape(**{**GOOD, **edit}))
    big = 1 << 40
    assert lib.attn_fwd_paged_e4m3(s, p, p, p, p, p, p, p, p, 1.0, 0, 0, p, p, p, big, None) == status
    assert lib.attn_fwd_prefix_e4m3(s, p, p, p, p, p, p, 5, p, p, p, 1.0, 0, p, p, p, big, None) == status
    assert lib.attn_append_paged_e4m3(s, p, p, p, p, p, p, p, 4, 0, 0, p, p, p, p, p, p, big, None) == status


def test_arguments_that_the_library_refuses(lib):
    import exact_tiled_softmax_gb300 as ex
    p, odd, ws = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8), ctypes.c_void_p(1 << 21)
    s = ctypes.byref(ex.PagedShape(**GOOD))
    big = 1 << 40

    def paged(q=p, k=p, v=p, ks=p, vs=p, t=p, n=p, y=p, L=p, w=ws, mask=0, win=0, size=big, shape=s):
        return lib.attn_fwd_paged_e4m3(shape, q, k, v, ks, vs, t, n, p, 1.0, mask, win, y, L, w, size, None)

    def prefix(q=p, k=p, v=p, ks=p, vs=p, pt=p, n=5, mask=0, y=p, L=p, w=ws, size=big, shape=s):
        return lib.attn_fwd_prefix_e4m3(shape, q, k, v, ks, vs, pt, n, p, p, p, 1.0, mask, y, L, w, size, None)

    def append(k=p, v=p, kp=p, vp=p, ks=p, vs=p, w=ws, pairs=4, size=big, shape=s):
        return lib.attn_append_paged_e4m3(shape, p, k, v, p, p, p, p, pairs, 0, 0, p, kp, vp, ks, vs, w, size, None)

    for call, names in ((paged, ("q", "k", "v", "ks", "vs", "y", "L", "w")), (prefix, ("q", "k", "v", "ks", "vs", "y", "L", "w")),
                        (append, ("k", "v", "kp", "vp", "ks", "vs", "w"))):
        for name in names:
            assert call(**{name: None}) == 1, name
            assert call(**{name: odd}) == 3, name
        assert call(shape=None) == 1 and call(size=255) == 4
    assert paged(mask=3) == 2 and paged(mask=2, win=0) == 1 and paged(mask=9) == 1
    assert prefix(mask=2) == 2 and prefix(n=-1) == 1 and prefix(pt=None) == 1 and append(pairs=33) == 1
    assert paged(size=lib.exattn_paged_workspace_size(s) - 1) == 4
    assert prefix(size=lib.exattn_prefix_workspace_size(s) - 1) == 4


def test_packed_calls_reach_the_same_checks(lib):
    """The binding's packed structure has the C layout: each operation's own refusals."""
    import exact_tiled_softmax_gb300 as ex
    p, big = 1 << 20, 1 << 40

    def run(op, shape=GOOD, **edit):
        f = dict(q=p, k=p, v=p, kp=p, vp=p, t=p, n=p, st=p, pt=p, inv=p, y=p, L=p, w=p, size=big, s=0,
                 scale=1.0, mask=0, win=0, plen=5, pairs=4, inter=0, ks=p, vs=p)
        f.update(edit)
        return lib.exattn_paged_e4m3_run(op, ex._PAGED_E4M3_CALL.pack(*shape.values(), *f.values()))

    assert ex._PAGED_E4M3_CALL.size == ex._PAGED_CALL.size + 16
    assert run(3) == 1 and lib.exattn_paged_e4m3_run(1, None) == 1
    for op in range(3):
        assert run(op, {**GOOD, "d": 72}) == 2
        assert run(op, ks=0) == 1 and run(op, vs=0) == 1 and run(op, ks=p + 4) == 3 and run(op, vs=p + 4) == 3
        assert run(op, kp=p + 8) == 3 and run(op, y=p + 8) == 3 and run(op, size=8) == 4
    assert run(0, pairs=33) == 1 and run(1, mask=2, win=0) == 1 and run(2, plen=-1) == 1


F8, U8 = torch.float8_e4m3fn, torch.uint8


def _args(**edit):
    a = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k_pages=torch.zeros(5, 2, 16, 64).to(F8),
             v_pages=torch.zeros(5, 2, 16, 32).to(F8), page_table=torch.zeros(3, 4, dtype=torch.int32),
             seq_lens=torch.ones(3, dtype=torch.int32), k_scales=torch.zeros(5, 2, 16, dtype=U8),
             v_scales=torch.zeros(5, 2, 16, dtype=U8))
    a.update(edit)
    return a


@pytest.mark.parametrize("edit,match", [
    (dict(k_scales=None), "k_scales is missing"),
    (dict(v_scales=None), "v_scales is missing"),
    (dict(k_scales=None, v_scales=None), "k_scales is missing"),
    (dict(k_scales=torch.zeros(5, 2, 15, dtype=U8)), "k_scales must be"),
    (dict(v_scales=torch.zeros(5, 2, 16)), "v_scales must be"),
    (dict(v_scales=torch.zeros(5, 2, 32, dtype=U8)[:, :, ::2]), "v_scales must be"),
    (dict(k_pages=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)), "dtype mismatch"),
    (dict(v_pages=torch.zeros(5, 2, 16, 32, dtype=torch.bfloat16)), "dtype mismatch"),
    (dict(v_pages=torch.zeros(5, 2, 16, 32).to(torch.float8_e5m2)), "dtype mismatch"),
    (dict(k_pages=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16), v_pages=torch.zeros(5, 2, 16, 32, dtype=torch.bfloat16)),
     "dtype mismatch"),
    (dict(), "CUDA device"),
], ids=lambda x: str(x)[:40] if isinstance(x, str) else "")
def test_tensors_that_the_binding_refuses(lib, edit, match):
    import exact_tiled_softmax_gb300 as ex
    with pytest.raises(ValueError, match=match):
        ex.fwd_paged(scale=1.0, **_args(**edit))
    with pytest.raises(ValueError, match=match):
        ex.fwd_prefix(scale=1.0, prefix_table=torch.zeros(2, dtype=torch.int32), prefix_len=32, **_args(**edit))
    with pytest.raises(ValueError, match=match):
        ex.append_paged(k=torch.zeros(3, 2, 64, dtype=torch.bfloat16), v=torch.zeros(3, 2, 32, dtype=torch.bfloat16),
                        **_args(**edit))

"""Paged key/value cache in float64 (oracle; test infrastructure only).

The serving operators written out token by token: append with rotation, and
attention of each token over its sequence's cached keys.  Sequence b owns tokens
starts[b] .. starts[b+1]-1; token i of nq is at position lens[b] - nq + i; key j
is row j % page of page table[b][j // page].

Beside each result stand the sums that bound what rounding can do to it:
A = sum_j p_j |V_j| (per column) and D = max_j c sum_e |q_e k_e| over the allowed keys.
"""
import numpy as np


def rotate(x, pos, inv_freq, interleaved):
    """x [..., d] at position pos: pair f turned by pos * inv_freq[f]."""
    y = np.array(x, dtype=np.float64)
    r = len(inv_freq)
    for f in range(r):
        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + r)
        c, s = np.cos(float(pos) * float(inv_freq[f])), np.sin(float(pos) * float(inv_freq[f]))
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def append(k, v, k_pages, v_pages, table, lens, starts, q=None, inv_freq=(), interleaved=False,
           offset=0):
    """(q_out, k_pages, v_pages) in float64; tokens without a place are not written and
    tokens that no sequence owns give NaN rows of q_out (the caller's rows stay).  Ends of
    `starts` outside the tokens and negative lengths are clamped."""
    kp, vp = k_pages.astype(np.float64), v_pages.astype(np.float64)
    page, num = kp.shape[2], kp.shape[0]
    qo = None if q is None else np.full(q.shape, np.nan)
    for b in range(len(lens)):
        first, end = (min(max(int(x), 0), len(k)) for x in starts[b:b + 2])
        nq = end - first
        for i in range(nq):
            t, pos = first + i, max(int(lens[b]), 0) - nq + i
            if q is not None:
                qo[t] = rotate(q[t], pos + offset, inv_freq, interleaved)
            if pos < 0 or pos >= table.shape[1] * page or not 0 <= table[b][pos // page] < num:
                continue
            at = table[b][pos // page]
            kp[at, :, pos % page] = rotate(k[t], pos + offset, inv_freq, interleaved)
            vp[at, :, pos % page] = v[t]
    return qo, kp, vp


def keys_of(pages, table_row, n):
    """The first n keys [kv_heads][n][width] of a sequence, and which of them have a page."""
    page, num = pages.shape[2], pages.shape[0]
    rows = np.zeros((pages.shape[1], n, pages.shape[3]))
    have = np.zeros(n, dtype=bool)
    for j in range(n):
        at = table_row[j // page]
        if 0 <= at < num:
            rows[:, j] = pages[at, :, j % page]
            have[j] = True
    return rows, have


def attend(q, k_pages, v_pages, table, lens, starts, scale, mask, window=0, prefix=None):
    """(Y [T,H,v], L [T,H], A, D); prefix: (table, length) of keys that every token
    allows before its own.  Rows of tokens that no sequence owns are NaN."""
    T, H, _ = q.shape
    kv, vw = k_pages.shape[1], v_pages.shape[3]
    Y, A = np.full((T, H, vw), np.nan), np.full((T, H, vw), np.nan)
    L, D = np.full((T, H), np.nan), np.full((T, H), np.nan)
    P = 0
    if prefix is not None:
        P = prefix[1]
        kf, have_f = keys_of(k_pages, prefix[0], P)
        vf, _ = keys_of(v_pages, prefix[0], P)
    for b in range(len(lens)):
        nq, n = starts[b + 1] - starts[b], int(lens[b])
        if nq == 0:
            continue
        k, have = keys_of(k_pages, table[b], n)
        v, _ = keys_of(v_pages, table[b], n)
        if P:
            k, v = np.concatenate((kf, k), 1), np.concatenate((vf, v), 1)
            have = np.concatenate((have_f, have))
        j = np.arange(P + n) - P
        for i in range(nq):
            pos = n - nq + i
            ok = have.copy()
            if mask != "none":
                ok &= (j < 0) | (j <= pos)
            if mask == "window":
                ok &= j > pos - window
            t = starts[b] + i
            for h in range(H):
                g = h // (H // kv)
                if not ok.any():
                    Y[t, h], A[t, h], L[t, h], D[t, h] = 0, 0, -np.inf, 0
                    continue
                kk, vv, qq = k[g][ok], v[g][ok], q[t, h].astype(np.float64)
                s = scale * (kk @ qq)
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                Y[t, h], A[t, h] = p @ vv, p @ np.abs(vv)
                L[t, h] = m + np.log(e.sum())
                D[t, h] = abs(scale) * (np.abs(kk) @ np.abs(qq)).max()
    return Y, L, A, D

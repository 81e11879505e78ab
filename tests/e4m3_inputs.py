"""Inputs of the tests of the paged cache in 8 bits: the batches of paged_inputs with their pages
quantised by the oracle."""
import numpy as np
import torch

from oracle import e4m3
from paged_inputs import DT, Batch


class Batch8(Batch):
    """k_pages and v_pages are codes (uint8), k_scales and v_scales bytes, k64 and v64 what they
    stand for.  Rows of the pool that no sequence uses hold NaN codes under a byte that is no
    scale.  spread: rows differ in size by up to 2^spread either way."""

    def __init__(self, lens, nqs, H, kv, d, v, dtype, page, seed=0, spread=3, q_gain=1.0, **kw):
        super().__init__(lens, nqs, H, kv, d, v, "f32", page, seed=seed, **kw)
        self.dtype = dtype
        rng = np.random.default_rng(seed + 1)
        for name in ("k", "v"):
            x = getattr(self, name + "_pages").double().numpy()
            x = x * 2.0 ** rng.integers(-spread, spread + 1, x.shape[:3])[..., None]
            unused = np.isnan(x).all(-1)
            codes, byte = e4m3.quantise(x)
            byte[unused] = 255
            setattr(self, name + "_pages", codes)
            setattr(self, name + "_scales", byte)
        self.requantised()
        self.q = (q_gain * self.q).to(DT[dtype])
        self.k_new, self.v_new = self.k_new.to(DT[dtype]), self.v_new.to(DT[dtype])

    def requantised(self):
        """After a change of codes or bytes."""
        self.k64, self.v64 = (e4m3.values(getattr(self, n + "_pages"), getattr(self, n + "_scales")) for n in "kv")

    def dev(self, *names):
        out = super().dev(*names)
        return [t.view(torch.float8_e4m3fn) if n in ("k_pages", "v_pages") else t for n, t in zip(names, out)]

    def cache(self):
        """k_pages, v_pages, table, lens, starts, k_scales, v_scales on the device."""
        return self.dev("k_pages", "v_pages", "table", "lens", "starts", "k_scales", "v_scales")

    def largest_weight(self, ref, scale, mask="none", window=0, prefix=None):
        """[T][H]: max_j p_j 2^(byte_j - 127) over the allowed keys, given the oracle's L."""
        L, W = ref[1], np.zeros(ref[1].shape)
        Lf = np.where(np.isfinite(L), L, 0.0)

        def rows(table, n, of, vs):
            j = np.arange(n)
            at = np.asarray(table)[j // self.page]
            have = (at >= 0) & (at < self.k64.shape[0])
            at = np.where(have, at, 0)
            return of[at, :, j % self.page], np.where(have[:, None], vs[at, :, j % self.page], 0.0), have

        vs = 2.0 ** (self.v_scales.astype(np.float64) - 127)
        for b in range(len(self.lens)):
            s0, s1, n = int(self.starts[b]), int(self.starts[b + 1]), int(self.lens[b])
            if s0 == s1:
                continue
            parts = [(rows(self.table[b], n, self.k64, vs), 0)]
            if prefix is not None and prefix[1]:
                parts.append((rows(prefix[0], prefix[1], self.k64, vs), None))
            for (k, w, have), own in parts:
                for t in range(s0, s1):
                    ok = have.copy()
                    if own is not None:
                        pos = n - (s1 - s0) + t - s0
                        j = np.arange(n)
                        if mask != "none":
                            ok &= j <= pos
                        if mask == "window":
                            ok &= j > pos - window
                    if not ok.any():
                        continue
                    for h in range(self.H):
                        g = h // (self.H // self.kv)
                        s = scale * (k[ok, g] @ self.q[t, h].double().numpy())
                        W[t, h] = max(W[t, h], (np.exp(s - Lf[t, h]) * w[ok, g]).max())
        return W


def weight_bits(path, dtype, d, v, page, rows, scale=1.0):
    """Significant bits of a weight in the product with V, by the kernel that `rows` rows to a key
    head take: the tall tiles round probabilities to bf16, the others hold weights in fp16 parts (one
    of bf16 queries, two of fp32 ones); the SIMT kernels hold them in fp32."""
    if path == "simt":
        return 22
    if dtype == "f32":
        return 21
    return 8 if rows > 16 and scale > 0 and d <= 128 and v <= 128 and page >= 8 else 11


def small_weights(W, n):
    """[T][H][1]: n weights that are each held to 2^-32 of their row's largest only, times the largest
    number, 448; twice that for pieces that are joined."""
    return (2 * n * 2.0 ** -32 * 448 * W)[..., None]

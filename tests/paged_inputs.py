"""Seeded inputs of the paged-cache tests, and the bounds that their results are
held to.  Nothing of the operators is computed here."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Batch:
    """A pool of pages in random order, tables, and packed tokens.  `lens` and `nqs`
    give each sequence's cached and new tokens; `pad` tokens follow the last
    sequence's.  Every row of the pool that no sequence uses holds NaN."""

    def __init__(self, lens, nqs, H, kv, d, v, dtype, page, seed=0, pad=0, prefix=0, spare=2,
                 gain=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = DT[dtype]
        self.dtype, self.page, self.H, self.kv = dtype, page, H, kv
        self.starts = np.concatenate(([0], np.cumsum(nqs))).astype(np.int32)
        self.lens = np.array(lens, dtype=np.int32)
        T = int(self.starts[-1]) + pad
        need = [-(-n // page) for n in lens]
        np_ = -(-prefix // page)
        num = sum(need) + np_ + spare
        perm = rng.permutation(num).astype(np.int32)
        most = max(1, max(need)) + 1  # one column that no sequence reaches
        self.table = np.full((len(lens), most), 2 ** 30, dtype=np.int32)  # no page at all
        k = torch.full((num, kv, page, d), float("nan"), dtype=dt)
        vv = torch.full((num, kv, page, v), float("nan"), dtype=dt)
        at = 0

        def fill(ids, n):
            for x, w in ((k, d), (vv, v)):
                rows = (gain * torch.randn(kv, max(n, 1), w, generator=g)).to(dt)[:, :n]
                for j in range(0, n, page):
                    c = min(page, n - j)
                    x[int(ids[j // page]), :, :c] = rows[:, j:j + c]

        for b, (n, c) in enumerate(zip(lens, need)):
            self.table[b, :c] = perm[at:at + c]
            fill(perm[at:at + c], n)
            at += c
        self.prefix = prefix
        self.prefix_table = perm[at:at + np_].copy()
        fill(self.prefix_table, prefix)
        self.k_pages, self.v_pages = k, vv
        self.q = (gain * torch.randn(T, H, d, generator=g)).to(dt)
        self.k_new = torch.randn(T, kv, d, generator=g).to(dt)
        self.v_new = torch.randn(T, kv, v, generator=g).to(dt)
        self.T = T

    def np(self, t):
        return t.double().numpy()

    def dev(self, *names):
        out = []
        for n in names:
            t = getattr(self, n)
            out.append((torch.from_numpy(t) if isinstance(t, np.ndarray) else t).cuda())
        return out


def check_attention(dtype, Y, L, ref, d, n, p_bits=16, extra=0.0):
    """Y and L against the float64 (Y, L, A, D) of n keys of width d at most.

    A score is c times a sum of d products; the products of bf16 are exact in fp32
    and those of fp32 are off by 2^-24 (2^-21 as three products of tf32 parts, the sum
    of the two lowest parts' product left out), the running sum adds 2^-24 of the
    partial sums at each of d steps (2^-23 where the tensor cores cut instead of
    rounding), folding c in costs 2^-23: |ds| <= (d + 8) 2^-23 D, D = max_j c sum |q k|.
    Probabilities move by a factor of exp(2 ds) at most, ex2.approx by 2^-22 + the
    rounding of its argument (2^-24 of |s| <= 2 D, the reference point included),
    and the two sums of n terms by n 2^-24 (taken as if all in one chain, far above
    the tree that is).  p rounded to p_bits significant bits adds 2^-p_bits.  Each acts
    on A = sum p |V|; Y is rounded last."""
    Y, L = Y.double().cpu().numpy(), L.double().cpu().numpy()
    Yr, Lr, A, D = ref
    own = ~np.isnan(Lr)
    fin = own & np.isfinite(Lr)
    assert np.array_equal(np.isneginf(L[own]), np.isneginf(Lr[own]))
    Dm = np.where(fin, D, 0.0)
    ds = (d + 16) * 2.0 ** -23 * Dm
    rel = 2 * ds + 2.0 ** -21 + (2 * n + 64) * 2.0 ** -24 + extra
    tol = (rel + 2.0 ** -p_bits)[..., None] * A + 1e-30
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(Yr) + tol)
    else:
        tol = tol + 2.0 ** -24 * np.abs(Yr)
    err = np.abs(Y - Yr)
    assert np.isfinite(Y[own]).all()
    assert (err[own] <= tol[own]).all(), float((err[own] / tol[own]).max())
    tl = rel + 2.0 ** -22 * (1 + np.abs(np.where(fin, Lr, 0)))
    assert (np.abs(L[fin] - Lr[fin]) <= tl[fin]).all(), float((np.abs(L[fin] - Lr[fin]) / tl[fin]).max())
    assert (Y[own & ~fin] == 0).all()

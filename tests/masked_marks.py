"""Marked sequences for capped, biased and masked attention: every position's share of a row shows in the row.

A position t of a sequence has a score of -e_t ln 2, e_t in 0 .. 3, and a value that is 1 in one dim and 0 in the others:
dim t mod D ("modulo": a row over n positions has about n / D of them to a dim, so that one position more or less
shows), or dim t D / L ("stretch": long sequences, where a run of positions shows).  Elements are sums of positive terms,
so a right kernel's are off by the relative errors of its weights and their own rounding."""
import numpy as np

from masked_checks import EPS, P_ROUNDING, Pools, TINY, f64, tdtype

LN2 = float(np.log(2.0))


class Marked(Pools):
    def __init__(self, lens, hkv, d, bs, dtype, seed, first_visible=None, marks="modulo"):
        import torch
        super().__init__(lens, hkv, d, bs, dtype, seed, first_visible=first_visible)
        rng = np.random.default_rng(seed + 1000)
        self.e = [rng.integers(0, 4, (hkv, n)) for n in lens]
        self.dim = [np.arange(n) % d if marks == "modulo" else np.arange(n) * d // n for n in lens]
        k, v = self.k.float().numpy(), self.v.float().numpy()
        for s, n in enumerate(lens):
            lo = first_visible[s] if first_visible is not None else 0
            t = np.arange(lo, n)
            blk, off, h = self.table[s, t // bs][:, None], (t % bs)[:, None], np.arange(hkv)[None]
            k[blk, h, :, off] = 0.0
            k[blk, h, 0, off, 0] = -self.e[s][:, t].T
            v[blk, h, :, off] = 0.0
            v[blk, h, self.dim[s][t][:, None], off] = 1.0
        self.k, self.v = torch.from_numpy(k).to(tdtype(dtype)), torch.from_numpy(v).to(tdtype(dtype))

    def queries(self, rows, heads, dtype):
        import torch
        q = torch.zeros(rows, heads, self.d, dtype=tdtype(dtype))
        q[..., 0] = 1.0
        return q

    def row(self, s, p, heads, softcap=0.0, slopes=None, window=0, prefix=0, weight=None, shift=(0, 0)):
        """[heads, D] of the row at position p of sequence s; `weight` [L] multiplies the positions' weights and `shift`
        moves the first and the last position (to plant mistakes)."""
        n = self.lens[s]
        lo = (max(0, p - window + 1) if window else 0) + shift[0]
        hi = max(p, min(prefix, n) - 1) + shift[1]
        t = np.arange(max(lo, 0), min(hi, n - 1) + 1)
        x = np.repeat(-LN2 * self.e[s][:, t], heads // self.hkv, axis=0)
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - np.asarray(slopes, np.float64)[:, None] * np.abs(p - t)[None]
        w = np.exp(x - x.max(1, keepdims=True))
        if weight is not None:
            w = w * weight[t]
        out = np.stack([np.bincount(self.dim[s][t], row, self.d) for row in w])
        return out / w.sum(1, keepdims=True)

    def excess(self, got, ref, dtype, bias=0.0):
        """How far rows are past what the arithmetic allows (at most 0 when right).  Weights: one product of the score's
        dot is not 0; the cap 2^-20 of a score below 3; the bias two roundings of its size; exp, sums and a piece's
        merge 2^-18 together; P's rounding.  The row twice that (its sum of weights is off too), and its own rounding."""
        rel = 2 * (P_ROUNDING[self.dtype] + 2.0 ** -18 + bias * 2.0 ** -22) + EPS[dtype] * (1 + 2.0 ** -6)
        return np.abs(got - ref) - rel * np.abs(ref) - TINY[dtype]


def rounded(x, dtype):
    """What a right kernel that computed x stores."""
    import torch
    return f64(torch.from_numpy(np.asarray(x, np.float64)).to(tdtype(dtype)))

"""Checks of decode over FP4 pools that a lost, doubled or misweighted piece cannot pass.

Markers.  The tokens of a sequence are cut into `D` stretches, and dim j of V is 6 for the tokens of stretch j and 0
for all others.  K and q are such that the weight of token t is the power of two 2^-e(t), e(t) in 0 .. 3:
q is 1 in dim 0 and 0 elsewhere, K is -e(t) there, the softmax's scale times k_scale times log2(e) is 1
up to 2^-22.  So, with C_j the sum of the weights of stretch j,
    out_j = 6 v_scale C_j / sum C.

How near the kernel has to come: the exponents e hs are off by at most 3 * 2^-22, an exponential by
2^-22 of itself, so every weight rounds to its power of two in fp16; products and sums of them are integers
times one power of two and below 2^24 of it, exact in fp32 whatever the order; a piece's factor when it is
merged is off by 2^-20 at most, and the two divisions and products at the end by 2^-22.  So
|out - ref| <= 2^-18 |ref| and half a step of the output's type.

sharp_bound, for any values.  With w the exact softmax weights, A = sum_t w_t |v_t|, L tokens and D dims, and
since the weights that are summed are the rounded ones, an error d_t of weight t moves out by d_t (v_t - out):
  * a weight is rounded once to fp16, after it was scaled so that the largest is 2^7 at least: by 2^-11 of
    itself, or below fp16's normal range by 2^-25 at most, that is 2^-32 of the weights' sum --
    2^-11 (A + |ref|) + L 2^-31 max|v|;
  * a score is a sum of D fp32 products scaled once, off by d = (D + 8) 2^-23 scale |q| max|k| + 2^-20 at most
    (the exponential's own error included) -- 2 d (A + |ref|) with room for the square;
  * both sums are accumulated in fp32, at most one addition per 8 tokens and a merge of partial
    results -- (L / 8 + 64) 2^-22 (A + |ref|);
  * the output is rounded once (half_ulp, added by the caller).
"""
import numpy as np

import oracle
import workloads as W
from helpers import half_ulp
from oracle import fp4

SF_ONE = 0x38        # the E4M3 code of 1
E2M1_OF = {0: 0, 1: 2, 2: 4, 3: 5, 6: 7}


class Markers:
    def __init__(self, lens, G, Hkv, D, bs, q_dtype, seed=0):
        rng = np.random.default_rng([seed, len(lens), G, Hkv, D, bs])
        self.lens, self.G, self.Hkv, self.D, self.bs, self.q_dtype = list(lens), G, Hkv, D, bs, q_dtype
        n = [-(-L // bs) for L in lens]
        NB = sum(n) + 3
        perm = rng.permutation(NB).astype(np.int32)
        self.table = np.full((len(lens), max(n) + 1), -1, np.int32)
        codes = {of: np.full((NB, Hkv, bs, D), 7, np.uint8) for of in "kv"}       # past a sequence's end: anything
        scales = {of: np.full((NB, Hkv, bs, D // 16), fp4.NAN_SCALE, np.uint8) for of in "kv"}
        self.e = []                                            # [Hkv, L] per sequence
        at = 0
        for i, L in enumerate(lens):
            self.table[i, :n[i]] = perm[at:at + n[i]]
            at += n[i]
            # runs of one exponent, the largest weight at any place (a run of a single token among them)
            e = np.repeat(rng.integers(1, 4, (Hkv, L // 37 + 1)), 37, axis=1)[:, :L]
            e[np.arange(Hkv), rng.integers(0, L, Hkv)] = 0
            self.e.append(e)
            t = np.arange(L)
            block, off = self.table[i, t // bs], t % bs
            for h in range(Hkv):
                k = np.zeros((L, D), np.uint8)
                k[:, 0] = np.array([0, 8 + E2M1_OF[1], 8 + E2M1_OF[2], 8 + E2M1_OF[3]], np.uint8)[e[h]]
                v = np.zeros((L, D), np.uint8)
                v[t, self.stretch(i)] = E2M1_OF[6]
                for of, x in (("k", k), ("v", v)):
                    codes[of][block, h, off] = x
                    scales[of][block, h, off] = SF_ONE
        self.k, self.v = (fp4.pack(codes[of], scales[of], of) for of in "kv")
        q = np.zeros((len(lens), G * Hkv, D))
        q[..., 0] = 1.0
        self.q = W.cast(q.astype(np.float32), q_dtype)
        self.k_scale, self.v_scale = 0.0173, 0.0214
        self.scale = float(1.0 / (float(np.float32(self.k_scale)) * np.log2(np.e)))
        self.max_len = max(lens)

    def stretch(self, i):
        L = self.lens[i]
        return (np.arange(L) * self.D) // L

    def expected(self, i, weight=None):
        """[H, D] of sequence i in fp64; `weight` [L] multiplies the tokens' weights (to plant a mistake)."""
        w = 2.0 ** -self.e[i]
        if weight is not None:
            w = w * weight
        C = np.stack([np.bincount(self.stretch(i), w[h], self.D) for h in range(self.Hkv)])
        out = 6 * float(np.float32(self.v_scale)) * C / C.sum(1, keepdims=True)
        return np.repeat(out, self.G, axis=0)

    def excess(self, i, got):
        """How far `got` [H, D] of sequence i is past what the arithmetic allows (at most 0 when right)."""
        ref = self.expected(i)
        bound = 2.0 ** -18 * np.abs(ref)
        return float((np.abs(got - ref) - bound - half_ulp(np.abs(ref) + bound, self.q_dtype)).max())

    def rounded(self, x):
        """What a right kernel that computed x stores."""
        return oracle.widen(W.cast(x.astype(np.float32), self.q_dtype), self.q_dtype)


# (lens, query heads per kv head, kv heads, head size, block size, query type): one segment over every CTA,
# segments cut at CTAs' ends, many pieces of one warp
LONG = [
    ([150001], 2, 1, 64, 16, "f16"), ([3, 60000, 1], 1, 1, 128, 16, "bf16"), ([9001], 4, 2, 128, 16, "f16"),
    ([20000, 3], 10, 1, 64, 32, "f16"), ([5000, 4999, 5001], 20, 1, 128, 32, "bf16"), ([40000], 1, 2, 128, 16, "f16"),
    ([1, 65, 3000, 700, 2222], 7, 2, 128, 16, "f16"),
]


def sharp_bound(q, q64, k_tiles, v_tiles, table, lens, scale, D, bs, k_scale, v_scale, q_dtype):
    """(exact out, bound without the final rounding) [S, H, D] for tiles whose unused slots may be NaN."""
    k64, v64 = fp4.f64_pools(k_tiles, v_tiles, D, bs, k_scale, v_scale)
    lens = np.asarray(lens, np.int32)
    out, mass = (oracle.decode(q, k64, v, table, lens, scale, "f64", q_dtype=q_dtype) for v in (v64, np.abs(v64)))
    kn = np.nanmax(np.sqrt((np.moveaxis(k64, 3, 2).reshape(*k64.shape[:2], bs, -1) ** 2).sum(-1)))
    qn = np.sqrt((q64 ** 2).sum(-1, keepdims=True))
    d = (D + 8) * 2.0 ** -23 * abs(scale) * qn * kn + 2.0 ** -20
    L = lens.astype(np.float64)[:, None, None]
    rel = 2.0 ** -11 + 2 * d + (L / 8 + 64) * 2.0 ** -22
    return out, rel * (mass + np.abs(out)) + L * 2.0 ** -31 * np.nanmax(np.abs(v64))


# the sizes of the long decode tests over random rows
RANDOM = [
    ("f16", 128, 16, 7, 4, [4096, 512, 1000, 2047, 1]), ("bf16", 128, 16, 4, 8, [9001]),
    ("bf16", 64, 32, 10, 1, [20000, 3]), ("f16", 64, 16, 1, 5, [1, 1, 1, 7000, 1]),
    ("f16", 128, 32, 20, 1, [5000, 4999, 5001]), ("f16", 128, 16, 1, 32, [513, 600]),
    ("f16", 64, 16, 2, 1, [150001]), ("bf16", 128, 16, 1, 1, [3, 60000, 1]), ("f16", 128, 16, 1, 2, [40000]),
]


def sharp_bound_of(case, ks, vs):
    """sharp_bound of an object with the fields of a decode test case."""
    return sharp_bound(case.q, case.q64, case.k, case.v, case.table, case.lens, case.scale, case.D, case.bs, ks, vs,
                       case.q_dtype)

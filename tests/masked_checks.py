"""Shared by the tests of rotary positions and of capped, biased and masked attention: seeded
inputs, tolerances from the kernels' roundings, and comparisons with oracle/masked.py."""
import numpy as np

EPS = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}     # half a step, relative
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the least step


def tdtype(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[name]


def f64(t):
    return t.detach().double().cpu().numpy()


class Pools:
    """Sequences of the given lengths in randomly placed blocks.  Slots past a sequence's end, and pool
    blocks no sequence uses, hold NaN; before_window: so do the positions before each sequence's window
    (given as the first visible position), whose whole blocks leave the table."""

    def __init__(self, lens, hkv, d, bs, dtype, seed, k_scale=1.0, v_scale=1.0, first_visible=None, spare=3):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.bs, self.hkv, self.d, self.dtype = list(lens), bs, hkv, d, dtype
        self.k_scale, self.v_scale = float(np.float32(k_scale)), float(np.float32(v_scale))
        n = [-(-x // bs) for x in lens]
        nb = sum(n) + spare
        order = rng.permutation(nb).astype(np.int32)
        self.table = np.full((len(lens), max(max(n), 1)), -1, np.int32)
        at = 0
        k, v = np.full((nb, hkv, bs, d), np.nan, np.float32), np.full((nb, hkv, bs, d), np.nan, np.float32)
        for s, m in enumerate(n):
            self.table[s, :m] = order[at:at + m]
            at += m
            lo = first_visible[s] if first_visible is not None else 0
            for j in range(m):
                a, b = max(lo - j * bs, 0), min(lens[s] - j * bs, bs)
                if a < b:
                    k[self.table[s, j], :, a:b] = rng.standard_normal((hkv, b - a, d))
                    v[self.table[s, j], :, a:b] = rng.standard_normal((hkv, b - a, d))
            self.table[s, :min(lo // bs, m)] = rng.choice([-1, 2 ** 31 - 1, -2 ** 31], min(lo // bs, m))
        x = 16 // {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}[dtype]
        kt = torch.from_numpy(k / np.float32(self.k_scale)).view(nb, hkv, bs, d // x, x).permute(0, 1, 3, 2, 4)
        vt = torch.from_numpy(v / np.float32(self.v_scale)).permute(0, 1, 3, 2)
        self.k = kt.contiguous().to(tdtype(dtype))
        self.v = vt.contiguous().to(tdtype(dtype))

    def exact(self):
        return f64(self.k.float()) * self.k_scale, f64(self.v.float()) * self.v_scale

    def on(self, device):
        import torch
        return self.k.to(device), self.v.to(device), torch.from_numpy(self.table).to(device)


def queries(n, h, d, dtype, seed, size=2.0):
    import torch
    x = np.random.default_rng(seed).standard_normal((n, h, d)).astype(np.float32) * size
    return torch.from_numpy(x).to(tdtype(dtype))


def attention_bound(q, k, v, ref, scale, softcap, bias, dtype, wide_p):
    """How far a row may be from the reference, from the kernels' arithmetic.

    A weight is off by the relative error of exp's argument and of its own rounding; out, a mean of V
    with the weights, by twice that times max|V|, and by its own rounding.
      argument: the fp32 dot of D products, at most (D + 4) roundings of partial sums of |q||k|;
                the tanh, softcap 2^-21; the bias, two roundings of its size;
      weight:   exp and the sums (2^-20 together: a sum's roundings average out over terms of one sign),
                P as one fp16 number (2^-12; none for fp32 pools, 2^-16 for bf16's two parts)."""
    k, v = np.nan_to_num(k), np.nan_to_num(v)
    d = q.shape[-1]
    # |scale|: a rounding's size does not know the score's sign (scale may be negative)
    reach = abs(scale) * np.abs(q).sum(-1).max() * np.abs(k).max()
    arg = (d + 4) * 2.0 ** -24 * reach + softcap * 2.0 ** -21 + bias * 2.0 ** -22
    weight = arg + 2.0 ** -20 + wide_p
    return 2 * weight * np.abs(v).max() + EPS[dtype] * np.abs(ref) * (1 + 2.0 ** -6) + TINY[dtype]


P_ROUNDING = {"f32": 0.0, "f16": 2.0 ** -12, "bf16": 2.0 ** -16, "fp8": 2.0 ** -12}


def check_attention(out, ref, q, pools, scale, softcap=0.0, bias=0.0, dtype="f16", what=""):
    got = f64(out)
    k, v = pools.exact()
    bound = attention_bound(f64(q), k, v, ref, scale, softcap, bias, dtype, P_ROUNDING[pools.dtype])
    assert np.isfinite(got).all(), f"{what}: {np.isnan(got).sum()} NaN of {got.size}"
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound (error {np.abs(got - ref).max():.2e})"
    # and as a whole: a lost piece or a wrong mask is far above the mean error of roundings
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    most = 4 * EPS[dtype] + 4 * P_ROUNDING[pools.dtype] + 2.0 ** -18 + softcap * 2.0 ** -20
    assert rel <= most, f"{what}: relative error {rel:.2e}, at most {most:.2e}"


def slopes_of(h):
    return np.array([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], np.float32)

"""The FP4 cache format in plain numpy, fp64 -- TEST INFRASTRUCTURE ONLY.

A token's row of D dims in one kv head is D/16 groups of 16 dims; a group holds 16
E2M1 codes and one E4M3 scale sf and reads back as code * sf * s.  The write:
    u = max|x| / s,  sf = E4M3(u / 6) clamped to 448,  F = sf * s,
    code = E2M1(x / F), nearest, ties to even, clamped to +-6 (zeros where F = 0),
each of the four fp32 operations rounded to nearest (a quotient or product taken in
fp64 and then rounded to fp32 equals the fp32 operation).  A NaN makes the group NaN.

Logical pools here are (codes uint8 [NB, Hkv, bs, D], scales uint8 [NB, Hkv, bs, D/16]);
`pack` and `unpack` go to and from the tiles' byte order, which is built from its
description, not from the library's formulas.
"""
import functools

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    v = [m / 8.0 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    v[127] = np.nan
    return np.array(v + [-x for x in v])


E4M3 = _e4m3_table()
NAN_SCALE = 0x7F


def _nearest(x, grid):
    """Index of the grid value (ascending) nearest to x, ties to the even index; past the end, the last."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        down, up = x - grid[lo], grid[hi] - x
        take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def _f32(x):
    with np.errstate(over="ignore"):
        return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def quantise(x, s):
    """(codes uint8 [..., D], scale bytes uint8 [..., D/16]) of float64 rows x [..., D]."""
    s = float(np.float32(s))
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 16)
    nan = np.isnan(g).any(-1)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        u = _f32(np.max(np.abs(g), axis=-1) / s)
        sf = _nearest(np.minimum(np.where(nan, 0.0, _f32(u / 6.0)), 448.0), E4M3[:127])
        f = _f32(E4M3[sf] * s)[..., None]
        y = _f32(np.where(f > 0, np.abs(np.where(nan[..., None], 0.0, g)) / np.where(f > 0, f, 1.0), 0.0))
    mag = _nearest(np.minimum(y, 6.0), E2M1)
    codes = (mag + 8 * np.signbit(g)).astype(np.uint8)
    codes[nan] = 7
    return codes.reshape(x.shape), np.where(nan, NAN_SCALE, sf).astype(np.uint8)


def values(codes, scales, s):
    """float64 values of logical codes [..., D] and scale bytes [..., D/16]."""
    v = np.where(codes > 7, -1.0, 1.0) * E2M1[codes & 7]
    return v * np.repeat(E4M3[scales], 16, axis=-1) * float(np.float32(s))


def tile_bytes(D, bs):
    return bs * D // 2 + bs * D // 16


@functools.lru_cache(maxsize=None)
def places(D, bs, of):
    """(codes [bs, D/2], scales [bs, D/16]): where a tile keeps each byte."""
    G = D // 16
    codes = np.zeros((bs, D // 2), np.int64)
    scales = np.zeros((bs, G), np.int64)
    for sub in range(bs // 16):
        # sixteen rows in four runs of four: run i holds tokens i, 4 + i, 8 + i, 12 + i, the odd runs backwards
        order = []
        for i in range(4):
            run = [i, 4 + i, 8 + i, 12 + i]
            order += run[::-1] if i % 2 else run
        for r, t in enumerate(order):
            at = np.arange(D // 2)
            if D == 128 and (r // 2) % 2:
                at = np.concatenate([at[32:], at[:32]])
            codes[16 * sub + t] = (16 * sub + r) * (D // 2) + at
        base = bs * D // 2 + sub * 16 * G
        if of == "v":
            for g in range(G):
                for t in range(16):
                    scales[16 * sub + t, g] = base + 16 * g + t
        else:
            # the pairs of tokens (t, t + 2); then the runs of D/64 groups; then the pair's two tokens; then the run
            n = 0
            for t in [a + b for a in range(0, 16, 4) for b in range(2)]:
                for g0 in range(0, G, G // 4):
                    for tok in (t, t + 2):
                        for g in range(g0, g0 + G // 4):
                            scales[16 * sub + tok, g] = base + n
                            n += 1
    return codes, scales


def pack(codes, scales, of):
    """Tiles uint8 [NB, Hkv, tile bytes] of logical codes and scales."""
    bs, D = codes.shape[2:]
    ci, si = places(D, bs, of)
    out = np.zeros(codes.shape[:2] + (tile_bytes(D, bs),), np.uint8)
    out[..., ci] = codes[..., 0::2] | (codes[..., 1::2] << 4)
    out[..., si] = scales
    return out


def unpack(tiles, D, bs, of):
    ci, si = places(D, bs, of)
    two = tiles[..., ci]
    codes = np.empty(tiles.shape[:2] + (bs, D), np.uint8)
    codes[..., 0::2] = two & 15
    codes[..., 1::2] = two >> 4
    return codes, tiles[..., si]


def write(rows, pool, slots, s):
    """Quantise rows [T, Hkv, D] (float64) into the logical pool (codes, scales) in place."""
    codes, scales = pool
    bs = codes.shape[2]
    c, f = quantise(rows, s)
    for t, slot in enumerate(slots):
        if slot >= 0:
            codes[slot // bs, :, slot % bs] = c[t]
            scales[slot // bs, :, slot % bs] = f[t]


def pool_values(tiles, D, bs, of, s):
    """float64 [NB, Hkv, bs, D] of a pool's tiles."""
    return values(*unpack(tiles, D, bs, of), s)


def f64_pools(k_tiles, v_tiles, D, bs, k_scale, v_scale):
    """The pools' values in the fp64 oracle's own cache layouts (x = 2)."""
    k = pool_values(k_tiles, D, bs, "k", k_scale)
    v = pool_values(v_tiles, D, bs, "v", v_scale)
    nb, hkv = k.shape[:2]
    k = k.reshape(nb, hkv, bs, D // 2, 2).transpose(0, 1, 3, 2, 4)
    return np.ascontiguousarray(k), np.ascontiguousarray(v.transpose(0, 1, 3, 2))

"""fp64 reference of the calls around the cache -- TEST INFRASTRUCTURE ONLY: rotary positions, and
attention whose scores are capped, biased by distance or masked.  numpy only; it shares no code with
the CUDA library.

Rows and pools come as float64 (numpy), pools in the cache's layouts: k [NB, Hkv, D/x, bs, x],
v [NB, Hkv, D, bs].
"""
import numpy as np


def rope(x, positions, inv_freq, pairs, amplitude=1.0):
    """x float64 [T, heads, D] with the first 2 len(inv_freq) dims of each row turned, pair by pair, as
    complex numbers."""
    n = len(inv_freq)
    out = np.array(x, dtype=np.float64)
    first = np.arange(n) * 2 if pairs else np.arange(n)
    second = first + 1 if pairs else first + n
    # the angle in extended precision: positions may be far, and its whole turns cancel
    angle = np.asarray(positions, np.longdouble)[:, None] * np.asarray(inv_freq, np.longdouble)[None, :]
    two_pi = np.longdouble("6.283185307179586476925286766559")
    angle = (angle - two_pi * np.rint(angle / two_pi)).astype(np.float64)
    z = (out[..., first] + 1j * out[..., second]) * (amplitude * np.exp(1j * angle))[:, None, :]
    out[..., first], out[..., second] = z.real, z.imag
    return out


def frequencies(rotary_dim, base, scaling=None, factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """(inv_freq, amplitude) of a scaling, from its description one pair at a time."""
    out = []
    for i in range(rotary_dim // 2):
        f = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "bands":
            wave = 2 * np.pi / f
            if wave > original_len / low:
                f = f / factor
            elif wave > original_len / high:
                smooth = (original_len / wave - low) / (high - low)
                f = (1 - smooth) * f / factor + smooth * f
        elif scaling == "yarn":
            def at(turns):
                return rotary_dim * np.log(original_len / (turns * 2 * np.pi)) / (2 * np.log(base))
            lo, hi = max(np.floor(at(high)), 0), min(np.ceil(at(low)), rotary_dim - 1)
            ramp = min(max((i - lo) / ((hi - lo) if hi > lo else 0.001), 0.0), 1.0)
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return np.array(out), (0.1 * np.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rows_of(k_cache, v_cache, table, n, bs):
    """K and V [Hkv, n, D] of a sequence's first n positions (positions in blocks that the table does not
    name, entry < 0, come as NaN)."""
    hkv, d = v_cache.shape[1], v_cache.shape[2]
    k, v = np.full((hkv, n, d), np.nan), np.full((hkv, n, d), np.nan)
    for t in range(n):
        b = int(table[t // bs])
        if 0 <= b < len(v_cache):
            k[:, t] = k_cache[b, :, :, t % bs, :].reshape(hkv, d)
            v[:, t] = v_cache[b, :, :, t % bs]
    return k, v


def attend(q, p, k, v, scale, softcap=0.0, slopes=None, window=0, prefix=0):
    """Attention of one query [H, D] at position p over rows k, v [Hkv, n, D]; returns [H, D]."""
    h, hkv = q.shape[0], k.shape[0]
    lo = max(0, p - window + 1) if window else 0
    hi = max(p, min(prefix, k.shape[1]) - 1)
    t = np.arange(lo, hi + 1)
    kk, vv = k[:, lo:hi + 1], v[:, lo:hi + 1]
    s = scale * np.einsum("kgd,ktd->kgt", q.reshape(hkv, h // hkv, -1), kk).reshape(h, -1)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    if slopes is not None:
        s = s - np.asarray(slopes, np.float64)[:, None] * np.abs(p - t)[None, :]
    w = np.exp(s - s.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    return np.einsum("kgt,ktd->kgd", w.reshape(hkv, h // hkv, -1), vv).reshape(h, -1)


def decode(q, k_cache, v_cache, tables, lens, scale, bs, **mod):
    out = np.empty(q.shape)
    for s, n in enumerate(lens):
        k, v = rows_of(k_cache, v_cache, tables[s], int(n), bs)
        out[s] = attend(q[s], int(n) - 1, k, v, scale, **mod)
    return out


def prefill(q, k_cache, v_cache, tables, lens, starts, scale, bs, prefixes=None, **mod):
    out = np.empty(q.shape)
    for s, n in enumerate(lens):
        n = int(n)
        a, b = int(starts[s]), int(starts[s + 1])
        if a == b:
            continue
        k, v = rows_of(k_cache, v_cache, tables[s], n, bs)
        for i in range(a, b):
            out[i] = attend(q[i], n - (b - a) + (i - a), k, v, scale,
                            prefix=int(prefixes[s]) if prefixes is not None else 0, **mod)
    return out

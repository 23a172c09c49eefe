"""The fp64 reference of capped, biased and masked attention and of rotary positions, held against
independent code and against properties of the definitions (no GPU)."""
import math

import numpy as np
import pytest

from oracle import brute, masked
from masked_checks import Pools, queries, f64, slopes_of


def pools(lens, seed=0, hkv=2, d=64, bs=16):
    p = Pools(lens, hkv, d, bs, "f32", seed)
    return (p, *p.exact())


def test_plain_scores_agree_with_the_brute_force():
    p, k, v = pools([1, 17, 40])
    q = f64(queries(3, 4, 64, "f32", 1))
    out = masked.decode(q, k, v, p.table, p.lens, 0.125, 16)
    for s, n in enumerate(p.lens):
        kr, vr = masked.rows_of(k, v, p.table[s], n, 16)
        for h in range(4):
            ref = brute.dense_decode_one(q[s, h].tolist(), kr[h // 2].tolist(), vr[h // 2].tolist(), 0.125)
            assert np.allclose(out[s, h], ref, atol=1e-12)


@pytest.mark.parametrize("window", [1, 5, 16, 39, 40, 1000])
def test_capped_biased_window_term_by_term(window):
    p, k, v = pools([40], seed=2)
    q, sl = f64(queries(1, 4, 64, "f32", 3)), slopes_of(4)
    out = masked.decode(q, k, v, p.table, [40], 0.3, 16, softcap=7.0, slopes=sl, window=window)
    kr, vr = masked.rows_of(k, v, p.table[0], 40, 16)
    for h in range(4):
        acc = brute.RunningSoftmax(64)
        for t in range(40):
            if t > 39 - window:
                x = 0.3 * math.fsum(a * b for a, b in zip(q[0, h], kr[h // 2, t]))
                acc.add(7.0 * math.tanh(x / 7.0) - float(sl[h]) * (39 - t), vr[h // 2, t])
        assert np.allclose(out[0, h], acc.result(), atol=1e-12)


def test_a_window_is_a_shorter_sequence():
    p, k, v = pools([48], seed=4)
    q = f64(queries(1, 4, 64, "f32", 5))
    kr, vr = masked.rows_of(k, v, p.table[0], 48, 16)
    a = masked.attend(q[0], 47, kr, vr, 0.2, window=20)
    b = masked.attend(q[0], 19, kr[:, 28:], vr[:, 28:], 0.2)
    assert np.allclose(a, b, atol=1e-13)


def test_a_prefix_shows_later_positions_to_earlier_rows():
    p, k, v = pools([30], seed=6)
    q = f64(queries(30, 4, 64, "f32", 7))
    whole = masked.prefill(q, k, v, p.table, [30], [0, 30], 0.2, 16, prefixes=[12])
    kr, vr = masked.rows_of(k, v, p.table[0], 30, 16)
    for i in range(30):
        assert np.allclose(whole[i], masked.attend(q[i], max(i, 11), kr, vr, 0.2), atol=1e-13)


def test_large_caps_and_zero_slopes_change_nothing():
    p, k, v = pools([33], seed=8)
    q = f64(queries(1, 4, 64, "f32", 9))
    a = masked.decode(q, k, v, p.table, [33], 0.2, 16)
    b = masked.decode(q, k, v, p.table, [33], 0.2, 16, softcap=1e9, slopes=np.zeros(4))
    assert np.allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_turns_by_the_angle(pairs):
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((5, 3, 64)), masked.frequencies(32, 10000.0)[0]
    pos = np.array([0, 1, 7, 1000, -3])
    y = masked.rope(x, pos, f, pairs, 1.25)
    for t in range(5):
        for i in range(16):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + 16)
            c, s = math.cos(pos[t] * f[i]), math.sin(pos[t] * f[i])
            assert np.allclose(y[t, :, a], 1.25 * (x[t, :, a] * c - x[t, :, b] * s), atol=1e-12)
            assert np.allclose(y[t, :, b], 1.25 * (x[t, :, a] * s + x[t, :, b] * c), atol=1e-12)
    assert np.array_equal(y[..., 32:], x[..., 32:])


def test_rope_scores_depend_on_the_distance_only():
    rng = np.random.default_rng(1)
    f = masked.frequencies(64, 10000.0)[0]
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    dots = [np.sum(masked.rope(q, [p + 9], f, False) * masked.rope(k, [p], f, False)) for p in (0, 5, 100000)]
    assert np.allclose(dots, dots[0], atol=1e-9)

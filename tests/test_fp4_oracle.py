"""The FP4 format's oracle (oracle/fp4.py) pinned on the CPU: its tables against
torch's float8 type and the E2M1 definition, its quantiser against a search over all
codes, its byte order against a bijection, and its pools through the fp64 decode."""
import math

import numpy as np
import pytest

import oracle
from oracle import fp4


def test_tables():
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp4.E4M3, t, equal_nan=True)
    e2m1 = [m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]
    assert fp4.E2M1.tolist() == e2m1


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("of", ["k", "v"])
def test_places_cover_the_tile_once(D, bs, of):
    codes, scales = fp4.places(D, bs, of)
    at = np.concatenate([codes.ravel(), scales.ravel()])
    assert sorted(at) == list(range(fp4.tile_bytes(D, bs)))
    assert codes.max() < bs * D // 2 <= scales.min()


@pytest.mark.parametrize("s", [1.0, 0.0173, 2.0 ** -64, 2.0 ** 64])
def test_codes_are_the_nearest_and_scales_too(s):
    rng = np.random.default_rng(1)
    s = float(np.float32(s))
    x = np.float32(rng.standard_normal((200, 64)) * np.exp(rng.standard_normal((200, 64))) * 40 * s).astype(np.float64)
    codes, sf = fp4.quantise(x, s)
    top = np.abs(x.reshape(200, 4, 16)).max(-1) / s / 6
    best = np.abs(fp4.E4M3[:127][None, None] - top[..., None]).min(-1)
    assert np.allclose(np.abs(fp4.E4M3[sf] - top), best, rtol=1e-5)
    got = fp4.values(codes, sf, s).reshape(200, 4, 16)
    f = fp4.E4M3[sf] * s
    every = np.concatenate([fp4.E2M1, -fp4.E2M1])
    err = np.abs(every * f[..., None, None] - x.reshape(200, 4, 16, 1)).min(-1)
    assert np.all(np.abs(got - x.reshape(200, 4, 16)) <= err + 1e-6 * f[..., None])


def test_ties_go_to_even_codes():
    x = np.zeros((1, 64))
    x[0, :8] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x[0, 8:16] = -x[0, :8]
    codes, sf = fp4.quantise(x, 1.0)
    assert fp4.E4M3[sf[0, 0]] == 1.0
    assert fp4.values(codes, sf, 1.0)[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert (codes[0, 8:16] == codes[0, :8] + 8).all()


def test_zeros_saturation_infinities_and_nans():
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1] = 1e9, 1.0                      # past 448 * 6: clamped
    x[0, 16], x[0, 17] = np.inf, -300.0
    x[0, 32], x[0, 33] = np.nan, 1.0
    x[0, 48] = 5.9 * 2.0 ** -10                      # sf rounds to zero
    codes, sf = fp4.quantise(x, 1.0)
    v = fp4.values(codes, sf, 1.0)[0]
    assert v[0] == 2688 and v[1] == 0 and v[16] == 2688 and v[17] == -224
    assert np.isnan(v[32:48]).all() and (v[48:] == 0).all()


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32)])
def test_pack_and_write_round_trip_and_decode(D, bs):
    """Rows written through slots, packed, unpacked and attended to by the fp64 oracle equal
    attention over the quantised rows themselves."""
    rng = np.random.default_rng(2)
    NB, Hkv, G, L = 9, 2, 3, 2 * bs + 5
    pools = []
    rows = rng.standard_normal((2, L, Hkv, D))
    table = rng.permutation(NB)[:3].astype(np.int32)
    slots = [int(table[t // bs]) * bs + t % bs for t in range(L)]
    for of, x, s in (("k", rows[0], 0.03), ("v", rows[1], 0.02)):
        logical = (np.full((NB, Hkv, bs, D), 7, np.uint8), np.full((NB, Hkv, bs, D // 16), fp4.NAN_SCALE, np.uint8))
        fp4.write(x, logical, slots, s)
        pools.append(fp4.pack(*logical, of))
        back = fp4.unpack(pools[-1], D, bs, of)
        assert np.array_equal(back[0], logical[0]) and np.array_equal(back[1], logical[1])
    k64, v64 = fp4.f64_pools(*pools, D, bs, 0.03, 0.02)
    q = rng.standard_normal((1, Hkv * G, D)).astype(np.float32)
    out = oracle.decode(q, k64, v64, table[None], np.array([L], np.int32), 0.2, "f64", q_dtype="f32")
    kq = fp4.values(*fp4.quantise(rows[0], 0.03), 0.03)
    vq = fp4.values(*fp4.quantise(rows[1], 0.02), 0.02)
    for h in range(Hkv * G):
        w = np.array([math.exp(0.2 * float(q[0, h].astype(np.float64) @ kq[t, h // G])) for t in range(L)])
        ref = (w[:, None] * vq[:, h // G]).sum(0) / w.sum()
        assert np.abs(ref - out[0, h]).max() < 1e-12

"""Caps of every accepted size: where a cap is large against the scores, the result is plain attention's."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, f64, queries, slopes_of
from masked_rows import check_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# cap, size of most rows, size of every fifth row (whose scores lie around the cap or past it)
CAPS = [(2.0 ** -64, 2.0, 2.0), (0.37, 2.0, 0.02), (50.0, 2.0, 30.0), (200.0, 2.0, 100.0), (1e4, 2.0, 3000.0),
        (1e5, 20.0, 6000.0), (1e6, 2.0, 9000.0), (1e8, 2.0, 2.0), (1e8, 2.0, 9000.0), (2.0 ** 64, 2.0, 9000.0)]
TYPES = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")]


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


def mixed_queries(n, h, d, dtype, seed, size, other):
    q = queries(n, h, d, "f32", seed, 1.0)
    q *= size
    q.view(n * h, d)[::5] *= other / size
    return q.to(queries(1, 1, d, dtype, 0).dtype)


@pytest.mark.parametrize("caps", CAPS, ids=lambda c: "-".join(f"{x:g}" for x in c))
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "/".join(t))
def test_decode_caps(pa, types, caps):
    cap, size, other = caps
    for group, hkv, d, bs, alibi in ((4, 2, 64, 16, False), (1, 3, 128, 32, False), (10, 1, 128, 16, True)):
        lens = [1, 2, 17, 100, 700]
        ks, vs = (0.0173, 0.0214) if types[1] == "fp8" else (1.0, 1.0)
        pools = Pools(lens, hkv, d, bs, types[1], group, ks, vs)
        h = group * hkv
        q = mixed_queries(len(lens), h, d, types[0], group + 1, size, other)
        sl = slopes_of(h) if alibi else None
        out = torch.empty_like(q).cuda()
        kc, vc, bt = pools.on("cuda")
        pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), d ** -0.5,
                            700, cap, None if sl is None else torch.from_numpy(sl).cuda(), 0, pools.k_scale, pools.v_scale)
        assert pa.pa_get_device_error() == 0
        ref = masked.decode(f64(q), *pools.exact(), pools.table, lens, d ** -0.5, bs, softcap=cap, slopes=sl)
        check_rows(out, ref, q, pools, d ** -0.5, cap, 700.0 if alibi else 0.0, types[0], f"group {group}")


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "/".join(t))
def test_decode_with_the_largest_cap_is_plain_decode(pa, types):
    """A cap that no score comes near leaves the scores: the same row up to the rounding of fp32 steps."""
    pools = Pools([3, 500, 77], 2, 64, 16, types[1], 1)
    kc, vc, bt = pools.on("cuda")
    lens = torch.tensor(pools.lens, dtype=torch.int32, device="cuda")
    for h in (2, 8):
        q = queries(3, h, 64, types[0], 2).cuda()
        outs = [torch.empty_like(q) for _ in range(2)]
        for out, cap in zip(outs, (0.0, 2.0 ** 64)):
            pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 500, cap)
            ref = masked.decode(f64(q), *pools.exact(), pools.table, pools.lens, 0.125, 16)
            check_rows(out, ref, q, pools, 0.125, 2.0 ** 64 if cap else 0.0, 0.0, types[0])
    assert pa.pa_get_device_error() == 0


def test_decode_scales_that_a_small_cap_divides(pa):
    """A score of any size over the smallest cap: scale / cap itself need not be a number of 32 bits."""
    pools = Pools([40, 9], 1, 64, 16, "f16", 3)
    kc, vc, bt = pools.on("cuda")
    lens = torch.tensor(pools.lens, dtype=torch.int32, device="cuda")
    for h, scale, cap in ((4, 2.0 ** 70, 2.0 ** -64), (1, 2.0 ** 70, 2.0 ** -64), (4, 2.0 ** -70, 2.0 ** 64),
                          (1, 2.0 ** -70, 2.0 ** 64)):
        q = queries(2, h, 64, "f16", 4)
        out = torch.empty_like(q).cuda()
        pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, lens, scale, 40, cap)
        assert pa.pa_get_device_error() == 0
        ref = masked.decode(f64(q), *pools.exact(), pools.table, pools.lens, scale, 16, softcap=cap)
        check_rows(out, ref, q, pools, scale, cap)


@pytest.mark.parametrize("caps", CAPS, ids=lambda c: "-".join(f"{x:g}" for x in c))
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefill_caps(pa, dtype, caps):
    """Chunks that the rows see whole, chunks that the diagonal or a window cuts, and biased ones."""
    cap, size, other = caps
    for group, hkv, d, bs, kw in ((4, 2, 64, 16, dict()), (1, 1, 128, 32, dict(window=200)), (7, 1, 128, 16, dict(alibi=True))):
        ctx, news = [600, 3], [70, 150]
        lens = [a + b for a, b in zip(ctx, news)]
        pools = Pools(lens, hkv, d, bs, dtype, group)
        h = group * hkv
        q = mixed_queries(sum(news), h, d, dtype, group + 1, size, other)
        sl = slopes_of(h) if kw.get("alibi") else None
        starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        out = torch.empty_like(q).cuda()
        kc, vc, bt = pools.on("cuda")
        pa.pa_prefill_masked(out, q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             torch.from_numpy(starts).cuda(), d ** -0.5, max(lens), cap,
                             None if sl is None else torch.from_numpy(sl).cuda(), kw.get("window", 0))
        assert pa.pa_get_device_error() == 0
        ref = masked.prefill(f64(q), *pools.exact(), pools.table, lens, starts, d ** -0.5, bs, softcap=cap, slopes=sl,
                             window=kw.get("window", 0))
        check_rows(out, ref, q, pools, d ** -0.5, cap, float(max(lens)) if sl is not None else 0.0, dtype, f"group {group}")


def test_prefill_scales_that_a_small_cap_divides(pa):
    pools = Pools([140, 9], 1, 64, 16, "f16", 5)
    kc, vc, bt = pools.on("cuda")
    lens = torch.tensor(pools.lens, dtype=torch.int32, device="cuda")
    starts = np.array([0, 100, 109], np.int32)
    q = queries(109, 4, 64, "f16", 6)
    for scale, cap in ((2.0 ** 70, 2.0 ** -64), (2.0 ** -70, 2.0 ** 64), (2.0 ** 30, 2.0 ** 40), (2.0 ** -30, 2.0 ** -20)):
        out = torch.empty_like(q).cuda()
        pa.pa_prefill_masked(out, q.cuda(), kc, vc, bt, lens, torch.from_numpy(starts).cuda(), scale, 140, cap)
        assert pa.pa_get_device_error() == 0
        ref = masked.prefill(f64(q), *pools.exact(), pools.table, pools.lens, starts, scale, 16, softcap=cap)
        check_rows(out, ref, q, pools, scale, cap)

"""Slopes of any finite size: the row then is the value of the position with the largest score, with no overflow on the
way (a position's own bias is 0 whatever the slope)."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, f64, queries
from masked_rows import check_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
SLOPES = np.array([3.4e38, -3.4e38, 2.4e38, 1e37, -1e37, 1e30, 0.5, 0.0], np.float32)


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(softcap=9.0), dict(softcap=2.0 ** 64)], ids=str)
@pytest.mark.parametrize("types", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "fp8")], ids="/".join)
def test_decode(pa, types, kw):
    lens = [1, 2, 40, 700]
    for hkv in (2, 8):
        pools = Pools(lens, hkv, 64, 16, types[1], hkv)
        kc, vc, bt = pools.on("cuda")
        q = queries(4, 8, 64, types[0], 3)
        out = torch.empty_like(q).cuda()
        pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125, 700,
                            alibi_slopes=torch.from_numpy(SLOPES).cuda(), **kw)
        assert pa.pa_get_device_error() == 0
        ref = masked.decode(f64(q), *pools.exact(), pools.table, lens, 0.125, 16, slopes=SLOPES, **kw)
        check_rows(out, ref, q, pools, 0.125, kw.get("softcap", 0.0), 350.0, types[0])


@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(softcap=9.0), dict(softcap=2.0 ** 64)], ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("prefixes", [None, [300, 30, 5]], ids=["", "prefixes"])
def test_prefill(pa, dtype, prefixes, kw):
    ctx, news = [200, 0, 31], [130, 70, 1]
    lens = [a + b for a, b in zip(ctx, news)]
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    pools = Pools(lens, 2, 64, 16, dtype, 4)
    kc, vc, bt = pools.on("cuda")
    q = queries(sum(news), 8, 64, dtype, 5)
    out = torch.empty_like(q).cuda()
    pa.pa_prefill_masked(out, q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(starts).cuda(), 0.125, max(lens), alibi_slopes=torch.from_numpy(SLOPES).cuda(),
                         prefix_lens=None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32, device="cuda"), **kw)
    assert pa.pa_get_device_error() == 0
    ref = masked.prefill(f64(q), *pools.exact(), pools.table, lens, starts, 0.125, 16, prefixes, slopes=SLOPES, **kw)
    check_rows(out, ref, q, pools, 0.125, kw.get("softcap", 0.0), 350.0, dtype)

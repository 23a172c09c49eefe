"""Keys that are no numbers at positions that a row sees: the row is no number either, however its sequence is cut into
pieces, and no other row is touched."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, f64, queries
from masked_rows import check_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TYPES = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")]


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


def spoil(pools, seq, head, positions):
    """NaN keys of kv head `head` at positions of a sequence; returns the pools' values before."""
    clean = pools.exact()
    k = pools.k.float().numpy()
    t = np.asarray(positions)
    k[pools.table[seq, t // pools.bs], head, :, t % pools.bs] = np.nan
    pools.k = torch.from_numpy(k).to(pools.k.dtype)
    return clean


@pytest.mark.parametrize("call", ["plain", "masked"])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("lens,seq,positions", [
    ([20011, 300], 0, [0]), ([20011, 300], 0, [12345]), ([20011, 300], 0, range(9000, 9400)), ([300, 9000], 1, [8999]),
    ([100], 0, [5]), ([250], 0, range(0, 64)), ([40, 700, 900], 1, [333]),
    ([150000], 0, [70000]),
], ids=lambda x: str(x)[:20])
def test_decode(pa, lens, seq, positions, types, call):
    for group in (1, 4, 12):
        pools = Pools(lens, 2, 64, 16, types[1], group)
        clean = spoil(pools, seq, 1, list(positions))
        kc, vc, bt = pools.on("cuda")
        q = queries(len(lens), 2 * group, 64, types[0], group + 1)
        out = torch.zeros_like(q).cuda()
        sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if call == "masked":
            pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, sl, 0.125, max(lens), 9.0)
        else:
            pa.pa_decode_scaled(out, q.cuda(), kc, vc, bt, sl, 0.125, max(lens), 1.0, 1.0)
        assert pa.pa_get_device_error() == 0
        nan = np.zeros(out.shape[:2], bool)
        nan[seq, group:] = True                               # the query heads of kv head 1
        got = torch.isnan(out.float()).cpu().numpy()
        assert got[nan].all(), "a row that sees them is a number"
        assert not got[~nan].any(), "a row that does not see them is none"
        if max(lens) <= 20011:
            ref = masked.decode(f64(q), *clean, pools.table, lens, 0.125, 16, softcap=9.0 if call == "masked" else 0.0)
            fine = torch.where(torch.from_numpy(nan)[..., None], torch.from_numpy(ref).to(out.dtype), out.cpu())
            held = type("P", (), dict(exact=lambda self: clean, dtype=types[1]))()
            check_rows(fine, ref, q, held, 0.125, 9.0 if call == "masked" else 0.0, 0.0, types[0])


@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0), dict(window=200)], ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prefill(pa, dtype, kw):
    ctx, news = [300, 20], [90, 140]
    lens = [a + b for a, b in zip(ctx, news)]
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    for seq, at in ((0, 150), (0, 340), (1, 100), (1, 159)):
        pools = Pools(lens, 2, 64, 16, dtype, 1)
        clean = spoil(pools, seq, 1, [at])
        kc, vc, bt = pools.on("cuda")
        q = queries(sum(news), 8, 64, dtype, 2)
        out = torch.zeros_like(q).cuda()
        pa.pa_prefill_masked(out, q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             torch.from_numpy(starts).cuda(), 0.125, max(lens), **kw)
        assert pa.pa_get_device_error() == 0
        p = ctx[seq] + np.arange(news[seq])
        nan = np.zeros(out.shape[:2], bool)
        nan[starts[seq]:starts[seq + 1], 4:] = ((p >= at) & (p - at < kw.get("window", 10 ** 9)))[:, None]
        got = torch.isnan(out.float()).cpu().numpy()
        assert got[nan].all(), "a row that sees them is a number"
        assert not got[~nan].any(), "a row that does not see them is none"
        ref = masked.prefill(f64(q), *clean, pools.table, lens, starts, 0.125, 16, **kw)
        fine = torch.where(torch.from_numpy(nan)[..., None], torch.from_numpy(ref).to(out.dtype), out.cpu())
        held = type("P", (), dict(exact=lambda self: clean, dtype=dtype))()
        check_rows(fine, ref, q, held, 0.125, kw.get("softcap", 0.0), 0.0, dtype)

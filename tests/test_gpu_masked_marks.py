"""Masked decode and prefill over marked sequences (masked_marks; what they can tell apart is tested in
test_masked_marks.py): every position counts once, at every edge of a window, cut of a sequence and merge of its pieces."""
import numpy as np
import pytest

from masked_checks import f64, slopes_of
from masked_marks import LN2, Marked

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
TYPES = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")]
KINDS = [dict(), dict(softcap=3.0), dict(slopes=True), dict(softcap=5.0, slopes=True)]


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


def split(kw, heads):
    """A kind's arguments for the reference and for the calls."""
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = slopes_of(heads) * 2.0 ** -8
    call = {k: v for k, v in kw.items() if k != "slopes"}
    if "slopes" in kw:
        call["alibi_slopes"] = torch.from_numpy(kw["slopes"].astype(np.float32)).cuda()
    return kw, call


def decode(pa, m, heads, dtype, kw, max_len=None):
    kw, call = split(kw, heads)
    kc, vc, bt = m.on("cuda")
    q = m.queries(len(m.lens), heads, dtype)
    out = torch.full_like(q, 99.0).cuda()
    pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, torch.tensor(m.lens, dtype=torch.int32, device="cuda"), LN2,
                        max_len or max(m.lens), **call)
    assert pa.pa_get_device_error() == 0
    got = f64(out)
    assert np.isfinite(got).all()
    for s, n in enumerate(m.lens):
        assert m.excess(got[s], m.row(s, n - 1, heads, **kw), dtype, 8.0).max() <= 0, f"sequence {s} of {n}"


@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("group", [1, 4, 12])
def test_decode(pa, group, types, kw):
    for d, bs, window in ((64, 16, 0), (128, 32, 129), (64, 32, 33), (128, 16, 1000), (64, 16, 1), (64, 16, 16)):
        lens = [1, 2, 16, 17, 100, 700, 1500]
        first = [max(0, n - window) if window else 0 for n in lens]
        m = Marked(lens, 2, d, bs, types[1], group + d, first)
        decode(pa, m, 2 * group, types[0], dict(kw, window=window))


@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_decode_of_few_blocks(pa, types):
    """Launches of one CTA, which merges its pieces itself."""
    n0 = pa.pa_launch_count()
    calls = 0
    for lens in ([100], [250], [40, 60], [1, 5, 17, 2, 33], [3, 130]):
        for group, window in ((1, 0), (4, 37), (4, 0)):
            first = [max(0, n - window) if window else 0 for n in lens]
            decode(pa, Marked(lens, 1, 64, 16, types[1], sum(lens), first), group, types[0], dict(softcap=3.0, window=window))
            calls += 1
    assert pa.pa_launch_count() - n0 < 2 * calls, "no launch was of one CTA"


@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("lens,group,hkv", [([20011, 9000], 4, 1), ([40000], 1, 2), ([3, 60000, 1], 8, 1),
                                             ([5000, 4999, 5001], 20, 1)], ids=str)
def test_decode_of_long_sequences(pa, lens, group, hkv, types):
    """Sequences cut over many CTAs, whose pieces the second kernel merges."""
    decode(pa, Marked(lens, hkv, 64, 16, types[1], 5, marks="stretch"), group * hkv, types[0], dict())
    w = 3 * max(lens) // 5
    m = Marked(lens, hkv, 64, 16, types[1], 6, [max(0, n - w) for n in lens], marks="stretch")
    decode(pa, m, group * hkv, types[0], dict(softcap=3.0, window=w))


@pytest.mark.parametrize("longest,window", [(100, 0), (900, 300), (2000, 0)])
@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_decode_of_a_batch(pa, types, longest, window):
    lens = [int(x) for x in np.random.default_rng(longest).integers(1, longest + 1, 90)]
    first = [max(0, n - window) if window else 0 for n in lens]
    decode(pa, Marked(lens, 3, 64, 16, types[1], 7, first), 6, types[0], dict(softcap=3.0, window=window))


@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,prefixes", [(0, None), (1, None), (129, None), (600, None), (0, [300, 1000, 0, 30]),
                                             (200, [260, 900, -1, 300])], ids=str)
def test_prefill(pa, window, prefixes, dtype, kw):
    for group, hkv, d, bs in ((4, 2, 64, 16), (1, 1, 128, 32), (7, 1, 64, 32)):
        ctx, news = [200, 0, 1000, 127], [70, 300, 1, 130]
        lens = [a + b for a, b in zip(ctx, news)]
        first = [max(0, a - window + 1) if window else 0 for a in ctx]
        m = Marked(lens, hkv, d, bs, dtype, group, first)
        heads = group * hkv
        ref_kw, call = split(dict(kw, window=window), heads)
        kc, vc, bt = m.on("cuda")
        q = m.queries(sum(news), heads, dtype)
        starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        out = torch.full_like(q, 99.0).cuda()
        pa.pa_prefill_masked(out, q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             torch.from_numpy(starts).cuda(), LN2, max(lens),
                             prefix_lens=None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32, device="cuda"),
                             **call)
        assert pa.pa_get_device_error() == 0
        got = f64(out)
        assert np.isfinite(got).all()
        for s, (a, n) in enumerate(zip(ctx, news)):
            for i in range(n):
                ref = m.row(s, a + i, heads, prefix=0 if prefixes is None else prefixes[s], **ref_kw)
                assert m.excess(got[starts[s] + i], ref, dtype, 8.0).max() <= 0, f"row {i} of sequence {s}"

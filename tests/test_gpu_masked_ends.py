"""Sequences as long as a length can be (2^31 - 1 tokens), whose windows leave a few blocks of them: the last blocks of a
short sequence stand at the end of a long one's table, and the result is the short one's."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, f64, queries, slopes_of
from masked_rows import check_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


def long_table(pools, long_lens):
    """A table whose row s ends, at long_lens[s] tokens, with the blocks of the pools' sequence s (as many tokens less
    a multiple of the block size); what stands before them is no block."""
    bs = pools.bs
    bt = torch.full((len(long_lens), (BIG + bs) // bs), -1, dtype=torch.int32, device="cuda")
    for s, (n, big) in enumerate(zip(pools.lens, long_lens)):
        assert (big - n) % bs == 0
        used = torch.from_numpy(pools.table[s, :-(-n // bs)].copy()).cuda()
        bt[s, (big - n) // bs:(big - n) // bs + len(used)] = used
    return bt


# ends: how far the sequences' lengths are below 2^31 - 1 (the last ones are short sequences' own)
CASES = [("f16", 16, [0, 3, 14]), ("bf16", 32, [0, 1, 30]), ("f32", 16, [0, 2, 14])]


@pytest.mark.parametrize("window", [1, 50, 64])
@pytest.mark.parametrize("dtype,bs,ends", CASES, ids=lambda x: str(x))
def test_decode_at_the_longest_lengths(pa, dtype, bs, ends, window):
    long_lens = [BIG - e for e in ends] + [100, 1]
    lens = [big if big < 1000 else 96 + big % bs for big in long_lens]
    for group in (4, 1):
        pools = Pools(lens, 2, 64, bs, dtype, group)
        kc, vc, _ = pools.on("cuda")
        q = queries(len(lens), 2 * group, 64, dtype, group + 1)
        sl = slopes_of(2 * group)
        for slopes in (None, sl):
            out = torch.full_like(q, 99.0).cuda()
            pa.pa_decode_masked(out, q.cuda(), kc, vc, long_table(pools, long_lens),
                                torch.tensor(long_lens, dtype=torch.int32, device="cuda"), 0.125, BIG, 9.0,
                                None if slopes is None else torch.from_numpy(slopes).cuda(), window)
            assert pa.pa_get_device_error() == 0
            ref = masked.decode(f64(q), *pools.exact(), pools.table, lens, 0.125, bs, softcap=9.0, window=window,
                                slopes=slopes)
            check_rows(out, ref, q, pools, 0.125, 9.0, 64.0 if slopes is not None else 0.0, dtype)


@pytest.mark.parametrize("window", [1, 50, 64])
@pytest.mark.parametrize("dtype,bs,ends", CASES[:2], ids=lambda x: str(x))
def test_prefill_at_the_longest_lengths(pa, dtype, bs, ends, window):
    long_lens = [BIG - e for e in ends] + [100, 1]
    lens = [big if big < 1000 else 96 + big % bs for big in long_lens]
    news = [30, 1, 7, 100, 1]
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    # (V past a sequence's end is NaN in the pools: it may not reach a row)
    for group, cap in ((4, 9.0), (1, 0.0)):
        pools = Pools(lens, 2, 64, bs, dtype, group)
        kc, vc, _ = pools.on("cuda")
        q = queries(sum(news), 2 * group, 64, dtype, group + 1)
        sl = slopes_of(2 * group)
        for slopes in (None, sl):
            out = torch.full_like(q, 99.0).cuda()
            pa.pa_prefill_masked(out, q.cuda(), kc, vc, long_table(pools, long_lens),
                                 torch.tensor(long_lens, dtype=torch.int32, device="cuda"),
                                 torch.from_numpy(starts).cuda(), 0.125, BIG, cap,
                                 None if slopes is None else torch.from_numpy(slopes).cuda(), window)
            assert pa.pa_get_device_error() == 0
            ref = masked.prefill(f64(q), *pools.exact(), pools.table, lens, starts, 0.125, bs, softcap=cap,
                                 window=window, slopes=slopes)
            check_rows(out, ref, q, pools, 0.125, cap, 64.0 if slopes is not None else 0.0, dtype)


@pytest.mark.parametrize("dtype,bs,ends", CASES[:2], ids=lambda x: str(x))
def test_prefill_at_the_longest_lengths_with_windows_and_prefixes(pa, dtype, bs, ends):
    """Prefixes that end before the window, within the chunk and past the sequence."""
    window = 60
    long_lens = [BIG - e for e in ends] + [100, 1]
    lens = [big if big < 1000 else 96 + big % bs for big in long_lens]
    news = [30, 25, 7, 100, 1]
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    cut = [big - n for big, n in zip(long_lens, lens)]
    for prefixes in ([10, long_lens[1] - 10, BIG, 60, 0], [long_lens[0] - 20, 0, 3, 100, -7]):
        short = [min(max(x - c, 0), n) for x, c, n in zip(prefixes, cut, lens)]
        pools = Pools(lens, 2, 64, bs, dtype, 8)
        kc, vc, _ = pools.on("cuda")
        q = queries(sum(news), 8, 64, dtype, 9)
        out = torch.full_like(q, 99.0).cuda()
        pa.pa_prefill_masked(out, q.cuda(), kc, vc, long_table(pools, long_lens),
                             torch.tensor(long_lens, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(),
                             0.125, BIG, 9.0, None, window, torch.tensor(prefixes, dtype=torch.int32, device="cuda"))
        assert pa.pa_get_device_error() == 0
        ref = masked.prefill(f64(q), *pools.exact(), pools.table, lens, starts, 0.125, bs, short, softcap=9.0, window=window)
        check_rows(out, ref, q, pools, 0.125, 9.0, 0.0, dtype)

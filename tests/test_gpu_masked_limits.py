"""The masked and rotary calls at their limits: waits that run out, calls at once on several streams and from several
host threads, pools past 2^31 elements, lengths and windows up to 2^31 - 1."""
import threading

import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, check_attention, f64, queries

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TIMEOUT = 4           # PA_DEVERR_TIMEOUT
LIMIT_NS = 2_000_000  # as in the other tests of waits that run out: none of them faults or hangs


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    yield m
    m.pa_set_test_wait_limit(0)


def decode_call(pa, lens, seed, types=("f16", "f16"), stream=None, **kw):
    pools = Pools(lens, 2, 64, 16, types[1], seed)
    kc, vc, bt = pools.on("cuda")
    q = queries(len(lens), 8, 64, types[0], seed + 1)
    args = (q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125, max(lens))

    def call(stream=None):
        out = torch.full_like(args[0], 99.0)
        pa.pa_decode_masked(out, *args, stream=stream, **kw)
        return out

    def check(out):
        ref = masked.decode(f64(q), *pools.exact(), pools.table, lens, 0.125, 16, **kw)
        check_attention(out, ref, q, pools, 0.125, kw.get("softcap", 0.0), 0.0, types[0])
    return call, check


def prefill_call(pa, ctx, news, seed, dtype="f16", prefixes=None, **kw):
    lens = [a + b for a, b in zip(ctx, news)]
    pools = Pools(lens, 2, 64, 16, dtype, seed)
    kc, vc, bt = pools.on("cuda")
    q = queries(sum(news), 8, 64, dtype, seed + 1)
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    args = (q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(),
            0.125, max(lens))
    pre = None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32, device="cuda")

    def call(stream=None):
        out = torch.full_like(args[0], 99.0)
        pa.pa_prefill_masked(out, *args, prefix_lens=pre, stream=stream, **kw)
        return out

    def check(out):
        ref = masked.prefill(f64(q), *pools.exact(), pools.table, lens, starts, 0.125, 16, prefixes, **kw)
        check_attention(out, ref, q, pools, 0.125, kw.get("softcap", 0.0), 0.0, dtype)
    return call, check


CALLS = {
    "decode": lambda pa: decode_call(pa, [1, 17, 300, 2500, 40, 900], 1, softcap=9.0, window=700),
    "decode of few blocks": lambda pa: decode_call(pa, [60], 2, softcap=9.0),
    "decode f32": lambda pa: decode_call(pa, [900, 33], 3, ("f32", "f32"), softcap=9.0),
    "prefill": lambda pa: prefill_call(pa, [0, 40, 700], [70, 9, 130], 4, window=100),
    "prefill capped": lambda pa: prefill_call(pa, [0, 40, 700], [70, 9, 130], 5, "bf16", [30, 0, 800], softcap=9.0),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(pa, name):
    call, check = CALLS[name](pa)
    try:
        pa.pa_set_test_wait_limit(LIMIT_NS)
        call()
    finally:
        pa.pa_set_test_wait_limit(0)
    assert pa.pa_get_device_error() == TIMEOUT
    out = call()
    assert pa.pa_get_device_error() == 0
    check(out)


def test_calls_at_once_on_several_streams(pa):
    made = [CALLS[n](pa) for n in CALLS for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in made]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(3):
        for (call, _), s in zip(made, streams):
            with torch.cuda.stream(s):
                outs.append(call(stream=s))
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for i, out in enumerate(outs):
        made[i % len(made)][1](out)


def test_calls_from_several_host_threads(pa):
    made = [CALLS[n](pa) for n in CALLS]
    got, failed = {}, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(s):
                for _ in range(20):
                    got[i] = made[i][0](stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    assert pa.pa_get_device_error() == 0
    for i, (_, check) in enumerate(made):
        check(got[i])


def test_blocks_past_two_to_the_31_elements(pa):
    """Block numbers whose tiles lie past 2^31 elements: the write and the decode of a sequence there."""
    nb, hkv, d, bs = 135000, 8, 128, 16                   # 2.2e9 elements a pool
    kc = torch.empty(nb, hkv, d // 8, bs, 8, dtype=torch.float16, device="cuda")
    vc = torch.empty(nb, hkv, d, bs, dtype=torch.float16, device="cuda")
    t = 50
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((t, 8 + 2 * hkv, d)).astype(np.float32)).half().cuda()
    table = torch.tensor([[nb - 1, 3, nb - 7, nb - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(t, device="cuda")
    slots = table[0, pos // bs].long() * bs + pos % bs
    f = pa.pa_rope_frequencies(d)[0].cuda()
    q = torch.empty(t, 8, d, dtype=torch.float16, device="cuda")
    pa.pa_rope_and_cache(q, x[:, :8], x[:, 8:8 + hkv], x[:, 8 + hkv:], kc, vc, pos, slots, f)
    used = table[0].long()
    small_k, small_v = f64(kc[used]), f64(vc[used])
    k_ref = masked.rope(f64(x[:, 8:8 + hkv]), np.arange(t), f.cpu().numpy(), False)
    got_k = small_k[np.arange(t) // bs, :, :, np.arange(t) % bs].reshape(t, hkv, d)
    assert np.abs(got_k - k_ref).max() <= 2.0 ** -11 * np.abs(k_ref).max() * 1.01
    assert np.array_equal(small_v[np.arange(t) // bs, :, :, np.arange(t) % bs], f64(x[:, 8 + hkv:]))
    lens = torch.tensor([t], dtype=torch.int32, device="cuda")
    held = type("P", (), dict(exact=lambda self: (np.nan_to_num(small_k), np.nan_to_num(small_v)), dtype="f16"))()
    local = np.arange(4, dtype=np.int32)[None]
    out = torch.empty_like(q[-1:])
    pa.pa_decode_masked(out, q[-1:].contiguous(), kc, vc, table, lens, 0.09, 64, softcap=9.0, window=40)
    ref = masked.decode(f64(q[-1:]), small_k, small_v, local, [t], 0.09, bs, softcap=9.0, window=40)
    check_attention(out, ref, q[-1:], held, 0.09, 9.0)
    starts = np.array([0, t], dtype=np.int32)
    out = torch.empty_like(q)
    pa.pa_prefill_masked(out, q, kc, vc, table, lens, torch.from_numpy(starts).cuda(), 0.09, 64, softcap=9.0, window=40)
    ref = masked.prefill(f64(q), small_k, small_v, local, [t], starts, 0.09, bs, softcap=9.0, window=40)
    check_attention(out, ref, q, held, 0.09, 9.0)
    assert pa.pa_get_device_error() == 0


def test_length_bounds_up_to_two_to_the_31(pa):
    """max_seq_len, windows and prefixes at their largest, over short sequences (the table's width is the bound's)."""
    big = 2 ** 31 - 1
    pools = Pools([40, 100], 2, 64, 32, "f16", 5)
    kc, vc, _ = pools.on("cuda")
    width = big // 32 + 1
    bt = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    bt[:, :pools.table.shape[1]] = torch.from_numpy(pools.table).cuda()
    lens = torch.tensor([40, 100], dtype=torch.int32, device="cuda")
    q = queries(2, 8, 64, "f16", 6)
    out = torch.empty_like(q).cuda()
    for window in (big, 50):
        pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, lens, 0.125, big, softcap=9.0, window=window)
        ref = masked.decode(f64(q), *pools.exact(), pools.table, [40, 100], 0.125, 32, softcap=9.0, window=window)
        check_attention(out, ref, q, pools, 0.125, 9.0)
        qsl = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        pre = torch.tensor([big, -big], dtype=torch.int32, device="cuda")
        pa.pa_prefill_masked(out, q.cuda(), kc, vc, bt, lens, qsl, 0.125, big, softcap=9.0, window=window, prefix_lens=pre)
        check_attention(out, ref, q, pools, 0.125, 9.0)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2500])
def test_more_sequences_than_the_table_of_a_launch_holds(pa, n):
    """Many short chunks, some empty, with windows, slopes and prefixes of their own."""
    rng = np.random.default_rng(n)
    ctx, news = rng.integers(0, 40, n), rng.integers(0, 4, n)
    ctx = np.where(ctx + news == 0, 1, ctx)
    pre = rng.integers(0, 50, n)
    call, check = prefill_call(pa, ctx.tolist(), news.tolist(), n, prefixes=pre.tolist(), softcap=9.0, window=15)
    check(call())
    lens = (ctx + news).tolist()
    call, check = decode_call(pa, lens, n + 1, softcap=9.0, window=15)
    check(call())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 300])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0)])
def test_the_longest_windows_behind_rows_before_their_prefix(pa, window, kw):
    """Rows near position 0 that see a prefix of several chunks through a window longer than any sequence."""
    call, check = prefill_call(pa, [0, 3], [400, 200], 9, prefixes=[390, 150], window=window, **kw)
    check(call())
    assert pa.pa_get_device_error() == 0

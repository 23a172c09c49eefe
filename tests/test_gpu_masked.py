"""Decode and prefill with capped, biased and masked scores against oracle/masked.py."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, check_attention, f64, queries, slopes_of, tdtype

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


def run_decode(pa, pools, q, scale, max_len=None, **kw):
    kc, vc, bt = pools.on("cuda")
    out = torch.full_like(q, 99.0).cuda()
    scales = dict(k_scale=pools.k_scale, v_scale=pools.v_scale)
    slopes = kw.pop("slopes", None)
    pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, torch.tensor(pools.lens, dtype=torch.int32, device="cuda"), scale,
                        max_len or max(pools.lens), alibi_slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
                        **scales, **kw)
    assert pa.pa_get_device_error() == 0
    return out


def decode_case(pa, lens, group, hkv, d, bs, dtype, cdt, seed, cap=0.0, alibi=False, window=0, size=2.0, scale=None):
    first = [max(0, n - window) if window else 0 for n in lens]
    ks, vs = (0.0173, 0.0214) if cdt == "fp8" else (1.0, 1.0)
    pools = Pools(lens, hkv, d, bs, cdt, seed, ks, vs, first)
    h = group * hkv
    q = queries(len(lens), h, d, dtype, seed + 1, size)
    scale = d ** -0.5 if scale is None else scale
    mod = dict(softcap=cap, window=window, slopes=slopes_of(h) if alibi else None)
    out = run_decode(pa, pools, q, scale, **mod)
    ref = masked.decode(f64(q), *pools.exact(), pools.table, lens, scale, bs, **mod)
    bias = max(lens) if alibi else 0.0
    check_attention(out, ref, q, pools, scale, cap, bias, dtype, f"{dtype}/{cdt} group {group}")


MODS = [dict(cap=30.0), dict(alibi=True), dict(window=33), dict(cap=5.0, alibi=True, window=100), dict()]
TYPES = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")]


@pytest.mark.parametrize("mod", MODS, ids=str)
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "/".join(t))
@pytest.mark.parametrize("group", [1, 4, 7, 12, 20])
def test_decode(pa, group, types, mod):
    for d, bs in ((64, 32), (128, 16)):
        decode_case(pa, [1, 2, 15, 16, 17, 31, 32, 33, 100, 257, 700], group, 2, d, bs, *types, seed=group + d, **mod)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "/".join(t))
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 64, 699, 700, 701, 2 ** 31 - 1])
def test_decode_windows(pa, window, types):
    """Every place of the window's first position in a block, windows as long as a sequence and longer."""
    decode_case(pa, [1, 16, 47, 48, 49, 64, 700], 4, 1, 64, 16, *types, seed=window % 1000, window=window)
    decode_case(pa, [1, 31, 32, 33, 65, 700], 1, 2, 128, 32, *types, seed=window % 1000, window=window, cap=20.0)


@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "fp8"), ("f32", "f32")], ids=lambda t: "/".join(t))
def test_decode_long_contexts_in_pieces(pa, types):
    """Contexts cut over many CTAs, whose pieces the second kernel merges."""
    decode_case(pa, [20011, 9000], 8, 1, 64, 16, *types, seed=5, cap=30.0)
    decode_case(pa, [20011, 9000], 2, 1, 64, 32, *types, seed=6, window=12345, alibi=True)


def test_decode_scores_past_the_cap(pa):
    """Scores far past the cap: the tanh is +-1 and every such position weighs the same."""
    for types in TYPES:
        decode_case(pa, [50, 300], 4, 2, 64, 16, *types, seed=9, cap=2.0, size=60.0)
        decode_case(pa, [50, 300], 1, 2, 64, 16, *types, seed=10, cap=2.0 ** -20, size=4.0)


def test_decode_negative_scale(pa):
    for types in TYPES:
        decode_case(pa, [50, 300], 4, 2, 64, 16, *types, seed=11, cap=9.0, scale=-0.2)
        decode_case(pa, [50, 300], 4, 2, 64, 16, *types, seed=12, alibi=True, scale=-0.2)


def test_decode_biases_of_any_sign(pa):
    pools = Pools([64, 500], 2, 64, 16, "f16", 13)
    q = queries(2, 8, 64, "f16", 14)
    slopes = np.array([0.5, -0.5, 0.0, 3.0, -3.0, 1e-4, 100.0, -100.0], np.float32)
    out = run_decode(pa, pools, q, 0.125, slopes=slopes)
    ref = masked.decode(f64(q), *pools.exact(), pools.table, pools.lens, 0.125, 16, slopes=slopes)
    check_attention(out, ref, q, pools, 0.125, 0.0, 100.0 * 500, "f16")


def test_decode_unchanged_scores_equal_pa_decode(pa):
    for dtype in ("f16", "bf16", "f32"):
        pools = Pools([1, 100, 3000], 2, 128, 16, dtype, 15)
        q = queries(3, 8, 128, dtype, 16)
        out = run_decode(pa, pools, q, 0.09)
        plain = torch.empty_like(out)
        kc, vc, bt = pools.on("cuda")
        pa.pa_decode(plain, q.cuda(), kc, vc, bt, torch.tensor(pools.lens, dtype=torch.int32, device="cuda"), 0.09, 3000)
        ref = masked.decode(f64(q), *pools.exact(), pools.table, pools.lens, 0.09, 16)
        check_attention(plain, ref, q, pools, 0.09, dtype=dtype)
        check_attention(out, ref, q, pools, 0.09, dtype=dtype)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "/".join(t))
def test_decode_of_few_blocks(pa, types):
    """Launches of one CTA, which merges its pieces itself: one sequence of every length around a block's, and
    batches of short ones with a few warps' work or less."""
    for d, bs in ((64, 16), (128, 32)):
        for n in (1, 2, bs - 1, bs, bs + 1, 3 * bs + 5, 100):
            decode_case(pa, [n], 4, 1, d, bs, *types, seed=n + d, cap=12.0, window=40)
        decode_case(pa, [1, 5, 17, 2, 33], 1, 1, d, bs, *types, seed=31, alibi=True)
        decode_case(pa, [60, 3], 20, 1, d, bs, *types, seed=32, cap=4.0)
        decode_case(pa, [100], 8, 2, d, bs, *types, seed=33)


def test_decode_of_few_blocks_replayed(pa):
    """A captured launch of one CTA over other lengths: warps without work leave no piece behind."""
    pools = Pools([120], 1, 64, 16, "f16", 34)
    kc, vc, bt = pools.on("cuda")
    q = queries(1, 4, 64, "f16", 35).cuda()
    lens, out = torch.tensor([120], dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 120, softcap=6.0)
    n0 = pa.pa_launch_count()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 120, softcap=6.0, workspace=ws)
    assert pa.pa_launch_count() == n0 + 1
    for n in (120, 16, 1, 97, 33, 120):
        lens.fill_(n)
        out.fill_(99.0)
        graph.replay()
        ref = masked.decode(f64(q), *pools.exact(), pools.table, [n], 0.125, 16, softcap=6.0)
        check_attention(out, ref, q, pools, 0.125, 6.0)
    assert pa.pa_get_device_error() == 0


def test_decode_many_sequences(pa):
    """More sequences than one launch takes."""
    lens = [(37 * i) % 70 + 1 for i in range(1100)]
    decode_case(pa, lens, 4, 1, 64, 16, "f16", "f16", seed=17, cap=10.0, alibi=True, window=20)


def test_decode_lengths_outside_the_contract(pa):
    pools = Pools([40, 40, 40, 40], 1, 64, 16, "f16", 18)
    q = queries(4, 4, 64, "f16", 19)
    kc, vc, bt = pools.on("cuda")
    lens = torch.tensor([40, 0, 41, -3], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 99.0).cuda()
    pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, lens, 0.125, 40, window=17, softcap=5.0)
    assert pa.pa_get_device_error() == 2
    ref = masked.decode(f64(q)[:1], *pools.exact(), pools.table, [40], 0.125, 16, window=17, softcap=5.0)
    check_attention(out[:1], ref, q[:1], pools, 0.125, 5.0)
    assert not out[1:].any()


def test_decode_bad_block_inside_the_window_is_recorded(pa):
    pools = Pools([100], 1, 64, 16, "f16", 20)
    pools.table[0, 5] = 9999
    kc, vc, bt = pools.on("cuda")
    q = queries(1, 4, 64, "f16", 21).cuda()
    out, lens = torch.empty_like(q), torch.tensor([100], dtype=torch.int32, device="cuda")
    pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 100, window=30)
    assert pa.pa_get_device_error() == 1
    pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 100, window=4)      # blocks 6 on
    assert pa.pa_get_device_error() == 0


def test_decode_captured_and_replayed_over_other_lengths(pa):
    pools = Pools([900, 2000, 333], 2, 64, 16, "f16", 22)
    kc, vc, bt = pools.on("cuda")
    q = queries(3, 8, 64, "f16", 23).cuda()
    sl = torch.from_numpy(slopes_of(8)).cuda()
    lens = torch.tensor(pools.lens, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    kw = dict(softcap=20.0, alibi_slopes=sl, window=500)
    ws = pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 2000, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_masked(out, q, kc, vc, bt, lens, 0.125, 2000, workspace=ws, **kw)
    for new in ([900, 2000, 333], [1, 16, 17], [900, 1500, 1], [33, 2, 300]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(99.0)
        graph.replay()
        ref = masked.decode(f64(q), *pools.exact(), pools.table, new, 0.125, 16, softcap=20.0, slopes=slopes_of(8),
                            window=500)
        check_attention(out, ref, q, pools, 0.125, 20.0, 2000.0)
    assert pa.pa_get_device_error() == 0


def run_prefill(pa, pools, q, news, scale, prefixes=None, slopes=None, **kw):
    kc, vc, bt = pools.on("cuda")
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    out = torch.full((q.shape[0] + 3, *q.shape[1:]), 99.0, dtype=q.dtype, device="cuda")
    pa.pa_prefill_masked(out[:q.shape[0]], q.cuda(), kc, vc, bt,
                         torch.tensor(pools.lens, dtype=torch.int32, device="cuda"), torch.from_numpy(starts).cuda(),
                         scale, max(pools.lens), alibi_slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
                         prefix_lens=None if prefixes is None else torch.tensor(prefixes, dtype=torch.int32, device="cuda"),
                         **kw)
    assert pa.pa_get_device_error() == 0
    assert (out[q.shape[0]:] == 99.0).all(), "rows behind the last sequence changed"
    return out[:q.shape[0]], starts


def prefill_case(pa, ctx, news, group, hkv, d, bs, dtype, seed, cap=0.0, alibi=False, window=0, prefixes=None, size=2.0):
    lens = [a + b for a, b in zip(ctx, news)]
    # the first position that any row of the sequence's chunk sees
    first = [max(0, a - window + 1) if window else 0 for a in ctx]
    pools = Pools(lens, hkv, d, bs, dtype, seed, first_visible=first)
    h = group * hkv
    q = queries(sum(news), h, d, dtype, seed + 1, size)
    sl = slopes_of(h) if alibi else None
    out, starts = run_prefill(pa, pools, q, news, d ** -0.5, prefixes, sl, softcap=cap, window=window)
    ref = masked.prefill(f64(q), *pools.exact(), pools.table, lens, starts, d ** -0.5, bs, prefixes, softcap=cap,
                         slopes=sl, window=window)
    check_attention(out, ref, q, pools, d ** -0.5, cap, max(lens) if alibi else 0.0, dtype)


PREFILLS = [  # context, new tokens, group, kv heads
    ([0], [1], 1, 1),
    ([0, 5, 127, 128], [1, 3, 129, 40], 4, 2),
    ([300, 0, 17], [70, 200, 1], 7, 1),
    ([1000, 0], [33, 260], 2, 1),
    ([64, 9, 0], [64, 0, 130], 20, 1),    # a sequence without new tokens (its length is still one of the cache)
]
PMODS = [dict(cap=30.0), dict(alibi=True), dict(window=1), dict(window=100), dict(cap=5.0, alibi=True, window=129),
         dict(prefix=True), dict(prefix=True, cap=8.0, alibi=True, window=150), dict()]


@pytest.mark.parametrize("mod", PMODS, ids=str)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", range(len(PREFILLS)))
def test_prefill(pa, shape, dtype, mod):
    mod = dict(mod)
    ctx, news, group, hkv = PREFILLS[shape]
    lens = [a + b for a, b in zip(ctx, news)]
    if mod.pop("prefix", False):
        mod["prefixes"] = [(7 * n) // 8 if i % 2 == 0 else n + 1000 for i, n in enumerate(lens)]
        mod["prefixes"][-1] = -5 if len(lens) > 1 else lens[-1]
    for d, bs in ((64, 32), (128, 16)):
        prefill_case(pa, ctx, news, group, hkv, d, bs, dtype, seed=shape + d, **mod)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 600, 10000, 2 ** 31 - 1])
def test_prefill_windows(pa, window):
    prefill_case(pa, [513, 0, 128], [300, 257, 1], 4, 1, 64, 16, "f16", seed=window % 1000, window=window)
    prefill_case(pa, [500, 31], [140, 300], 1, 1, 128, 32, "bf16", seed=window % 999, window=window, cap=20.0)


def test_prefill_long_context_window(pa):
    """A window far behind which nothing is read: those blocks hold NaN and have left the table."""
    prefill_case(pa, [9000, 5000], [150, 300], 8, 1, 64, 16, "f16", seed=3, window=700, cap=30.0)
    prefill_case(pa, [9000], [20], 1, 1, 128, 32, "bf16", seed=4, window=4000, alibi=True)


def test_prefill_many_units(pa):
    """More units than clusters, of uneven lengths: the schedule hands out each one once."""
    prefill_case(pa, [0] * 24, [(61 * i) % 250 + 1 for i in range(24)], 4, 8, 64, 16, "f16", seed=5, cap=30.0,
                 prefixes=[(97 * i) % 300 for i in range(24)])
    prefill_case(pa, [(113 * i) % 500 for i in range(40)], [(31 * i) % 90 + 1 for i in range(40)], 8, 4, 64, 32, "bf16",
                 seed=6, window=130)


def test_prefill_scores_past_the_cap(pa):
    prefill_case(pa, [40], [200], 4, 1, 64, 16, "f16", seed=7, cap=2.0, size=60.0)
    prefill_case(pa, [40], [200], 4, 1, 128, 16, "bf16", seed=8, cap=2.0 ** -20)


def test_prefill_unchanged_scores_equal_pa_prefill(pa):
    pools = Pools([400, 130], 2, 128, 16, "f16", 9)
    q = queries(230, 8, 128, "f16", 10)
    out, starts = run_prefill(pa, pools, q, [100, 130], 0.09)
    plain = torch.empty_like(out)
    kc, vc, bt = pools.on("cuda")
    pa.pa_prefill(plain, q.cuda(), kc, vc, bt, torch.tensor(pools.lens, dtype=torch.int32, device="cuda"),
                  torch.from_numpy(starts).cuda(), 0.09, 400)
    # (not bit by bit: the two kernels add a row's weights in another order)
    ref = masked.prefill(f64(q), *pools.exact(), pools.table, pools.lens, starts, 0.09, 16)
    check_attention(plain, ref, q, pools, 0.09)
    check_attention(out, ref, q, pools, 0.09)


def test_prefill_equals_decode_of_the_last_row(pa):
    """The last row of a chunk is the query a decode of the same sequence has."""
    pools = Pools([300, 77], 2, 64, 16, "bf16", 11)
    q = queries(60, 8, 64, "bf16", 12)
    kw = dict(softcap=15.0, window=90, slopes=slopes_of(8))
    out, starts = run_prefill(pa, pools, q, [40, 20], 0.125, **kw)
    last = q[[39, 59]]
    dec = run_decode(pa, pools, last, 0.125, **kw)
    ref = masked.decode(f64(last), *pools.exact(), pools.table, pools.lens, 0.125, 16, **kw)
    check_attention(dec, ref, last, pools, 0.125, 15.0, 300.0, "bf16")
    check_attention(out[[39, 59]], ref, last, pools, 0.125, 15.0, 300.0, "bf16")


def test_prefill_captured_and_on_another_stream(pa):
    pools = Pools([300, 200], 2, 64, 16, "f16", 13)
    kc, vc, bt = pools.on("cuda")
    q = queries(150, 8, 64, "f16", 14).cuda()
    lens = torch.tensor([300, 200], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    prefix = torch.tensor([250, 10], dtype=torch.int32, device="cuda")
    out, side = torch.empty_like(q), torch.cuda.Stream()
    kw = dict(softcap=20.0, window=120, prefix_lens=prefix)

    def check(ns, st, pre):
        ref = masked.prefill(f64(q), *pools.exact(), pools.table, ns, st, 0.125, 16, pre, softcap=20.0, window=120)
        check_attention(out, ref, q, pools, 0.125, 20.0)

    side.wait_stream(torch.cuda.current_stream())
    pa.pa_prefill_masked(out, q, kc, vc, bt, lens, starts, 0.125, 300, stream=side, **kw)
    side.synchronize()
    check([300, 200], [0, 100, 150], [250, 10])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prefill_masked(out, q, kc, vc, bt, lens, starts, 0.125, 300, **kw)
    lens.copy_(torch.tensor([211, 200], dtype=torch.int32))
    starts.copy_(torch.tensor([0, 20, 150], dtype=torch.int32))
    prefix.copy_(torch.tensor([0, 180], dtype=torch.int32))
    out.fill_(99.0)
    graph.replay()
    check([211, 200], [0, 20, 150], [0, 180])
    assert pa.pa_get_device_error() == 0


def test_a_layer_as_it_is_used(pa):
    """Rotary positions with the write, a masked prefill of a prompt in two chunks, then generation steps with
    rotary positions, write and masked decode: each against the reference over what the pools hold."""
    for dtype, cdt in (("f16", "f16"), ("bf16", "bf16")):
        h, hkv, d, bs, window = 8, 2, 64, 16, 50
        kw = dict(softcap=20.0, window=window)
        rng = np.random.default_rng(15)
        kc = torch.full((12, hkv, d // 8, bs, 8), float("nan"), dtype=tdtype(cdt), device="cuda")
        vc = torch.full((12, hkv, d, bs), float("nan"), dtype=tdtype(cdt), device="cuda")
        table = torch.from_numpy(rng.permutation(12).astype(np.int32).reshape(1, 12)).cuda()
        f, amp = pa.pa_rope_frequencies(d, 10000.0, "yarn", 4.0, 64)
        f = f.cuda()
        sl = torch.from_numpy(slopes_of(h)).cuda()
        done = 0
        for n in (70, 41, 1, 1, 1):
            x = torch.from_numpy(rng.standard_normal((n, h + 2 * hkv, d)).astype(np.float32)).to(tdtype(dtype)).cuda()
            pos = torch.arange(done, done + n, device="cuda")
            slots = table[0, pos // bs].long() * bs + pos % bs
            q = torch.empty(n, h, d, dtype=x.dtype, device="cuda")
            pa.pa_rope_and_cache(q, x[:, :h], x[:, h:h + hkv], x[:, h + hkv:], kc, vc, pos, slots, f, amplitude=amp)
            done += n
            lens = torch.tensor([done], dtype=torch.int32, device="cuda")
            out = torch.empty_like(q)
            if n > 1:
                starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
                pa.pa_prefill_masked(out, q, kc, vc, table, lens, starts, 0.125, 12 * bs, alibi_slopes=sl, **kw)
            else:
                pa.pa_decode_masked(out, q, kc, vc, table, lens, 0.125, 12 * bs, alibi_slopes=sl, **kw)
            assert pa.pa_get_device_error() == 0
            k64, v64 = f64(kc), f64(vc)
            ref = masked.prefill(f64(q), k64, v64, table.cpu().numpy(), [done], [0, n], 0.125, bs, slopes=slopes_of(h),
                                 **kw)
            held = type("P", (), dict(exact=lambda self: (k64, v64), dtype=cdt))()
            check_attention(out, ref, q, held, 0.125, 20.0, float(window), dtype, f"after {done} tokens")


@pytest.fixture(params=["extension", "ctypes"])
def path(request, monkeypatch):
    """Both of the binding's paths: the extension, and the Python code that takes its place."""
    from paged_kv_cache_306_gb300 import _binding as B
    if request.param == "extension":
        assert B._fp4_calls() is not None, "the extension was not built"
    else:
        monkeypatch.setattr(B, "_fp4_calls", lambda: None)
    return request.param


def test_both_paths(pa, path):
    for types in (("f16", "f16"), ("bf16", "fp8"), ("f32", "f32")):
        decode_case(pa, [40, 77], 4, 2, 64, 16, *types, seed=25, cap=9.0, alibi=True, window=50)
    prefill_case(pa, [40, 0], [60, 33], 4, 2, 64, 16, "bf16", seed=26, cap=9.0, alibi=True, window=50, prefixes=[70, 20])
    pools = Pools([40, 500], 2, 64, 16, "f16", 27)
    kc, vc, bt = pools.on("cuda")
    q, lens = queries(2, 8, 64, "f16", 28).cuda(), torch.tensor([40, 500], dtype=torch.int32, device="cuda")
    out = [torch.empty_like(q) for _ in range(2)]
    ws = pa.pa_decode_masked(out[0], q, kc, vc, bt, lens, 0.125, 500, 5.0)
    assert ws is not None and pa.pa_decode_masked(out[1], q, kc, vc, bt, lens, 0.125, 500, 5.0, workspace=ws) is ws
    assert torch.equal(*out)


def test_binding_refusals(pa, path):
    pools = Pools([40, 40], 2, 64, 16, "f16", 23)
    kc, vc, bt = pools.on("cuda")
    q = queries(2, 8, 64, "f16", 24).cuda()
    lens = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    sl = torch.zeros(8, device="cuda")
    good = dict(out=torch.empty_like(q), q=q, k_cache=kc, v_cache=vc, block_tables=bt, seq_lens=lens, scale=0.1,
                max_seq_len=40, alibi_slopes=sl)
    both = [dict(q=q[:, :, :32]), dict(out=torch.empty_like(q)[:1]), dict(out=torch.empty_like(q).float()),
            dict(k_cache=kc[:, :1]), dict(k_cache=kc.view(kc.shape[0], 2, 16, 16, 4)), dict(v_cache=vc[:1]),
            dict(block_tables=bt[:1]), dict(block_tables=bt.long()), dict(seq_lens=lens[:1]), dict(seq_lens=lens.long()),
            dict(alibi_slopes=sl[:7]), dict(alibi_slopes=sl.double()), dict(alibi_slopes=sl.cpu()), dict(softcap=-1.0),
            dict(softcap=float("nan")), dict(window=-1), dict(window=2 ** 31), dict(max_seq_len=2 ** 31),
            dict(max_seq_len=1000), dict(q=q.cpu()), dict(scale=float("nan"))]
    for b in both:
        with pytest.raises(pa.PAError):
            pa.pa_decode_masked(**{**good, **b})
        with pytest.raises(pa.PAError):
            pa.pa_prefill_masked(query_start_loc=starts, **{**good, **b})
    with pytest.raises(pa.PAError):
        pa.pa_decode_masked(**{**good, "q": q[:1].contiguous(), "out": torch.empty_like(q)[:1].contiguous()})
    with pytest.raises(pa.PAError):
        pa.pa_prefill_masked(query_start_loc=starts[:2], **good)
    with pytest.raises(pa.PAError):
        pa.pa_prefill_masked(query_start_loc=starts, **{**good, "prefix_lens": lens[:1]})
    with pytest.raises(pa.PAError):
        pa.pa_prefill_masked(query_start_loc=starts, **{**good, "scale": 0.0})
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    used = pa.pa_decode_masked(**good, workspace=small)          # too small: one of its own
    assert used is not small

"""Rotary positions, alone and with the write into the pool, against oracle/masked.py."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import EPS, TINY, f64, tdtype

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


def rows(t, h, hkv, d, dtype, seed, fused):
    x = np.random.default_rng(seed).standard_normal((t, h + 2 * hkv, d)).astype(np.float32)
    x = torch.from_numpy(x).to(tdtype(dtype)).cuda()
    q, k, v = x[:, :h], x[:, h:h + hkv], x[:, h + hkv:]
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def positions(t, seed, far):
    p = np.random.default_rng(seed + 1).integers(0, far, t)
    p[:min(t, 3)] = [0, far, 1][:min(t, 3)]
    return p


def turned_bound(x, ref, dtype, amplitude):
    """A turned element is x cos - y sin: the cosine and sine are off by at most 2^-22 of the amplitude
    (the fixed-point angle by 2^-25 of a radian, sincospif and the product with the amplitude by two
    steps), the two products by a step each; then the element's own rounding."""
    size = np.abs(x).max(axis=-1, keepdims=True)
    return 2 * size * abs(amplitude) * (2.0 ** -22 + 2.0 ** -23) + EPS[dtype] * np.abs(ref) * (1 + 2.0 ** -6) + TINY[dtype]


def check_rows(got, x, ref, dtype, amplitude, r, what):
    got, x = f64(got), f64(x)
    worst = np.max(np.abs(got - ref) / turned_bound(x, ref, dtype, amplitude))
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"
    assert np.array_equal(got[..., r:], x[..., r:]), f"{what}: dims past the rotary ones changed"


CASES = [  # tokens, heads, kv heads, head size, rotary dims, dtype, fused rows
    (1, 4, 1, 64, 64, "f16", True),
    (2, 1, 1, 128, 128, "bf16", False),
    (3, 28, 4, 128, 128, "f16", True),
    (17, 8, 2, 64, 16, "f32", False),
    (31, 5, 5, 128, 48, "bf16", True),
    (64, 28, 4, 128, 128, "f16", True),
    (65, 3, 1, 128, 96, "f32", True),
    (257, 32, 8, 128, 64, "bf16", False),
    (1000, 7, 1, 64, 32, "f16", True),
    (4099, 16, 16, 64, 64, "f32", False),
]


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope(pa, case, pairs):
    t, h, hkv, d, r, dtype, fused = case
    q, k, _ = rows(t, h, hkv, d, dtype, t, fused)
    pos = positions(t, t, 200000)
    f, _ = pa.pa_rope_frequencies(r, 10000.0)
    amp = 1.25 if pairs else 1.0
    qo = torch.full((t, h, d), 7.0, dtype=q.dtype, device="cuda")
    ko = torch.full((t, hkv, d), 7.0, dtype=q.dtype, device="cuda")
    pa.pa_rope(qo, ko, q, k, torch.from_numpy(pos).cuda(), f.cuda(), pa.ROPE_PAIRS if pairs else pa.ROPE_HALVES, amp)
    for got, x, name in ((qo, q, "q"), (ko, k, "key")):
        check_rows(got, x, masked.rope(f64(x), pos, f.numpy(), pairs, amp), dtype, amp, r, name)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_in_place_and_back(pa, pairs):
    q, k, _ = rows(100, 8, 2, 128, "f32", 3, False)
    pos = torch.from_numpy(positions(100, 5, 100000)).cuda()
    f = pa.pa_rope_frequencies(128)[0].cuda()
    q0, k0 = q.clone(), k.clone()
    layout = pa.ROPE_PAIRS if pairs else pa.ROPE_HALVES
    expect_q, expect_k = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope(expect_q, expect_k, q, k, pos, f, layout)
    pa.pa_rope(q, k, q, k, pos, f, layout)
    assert torch.equal(q, expect_q) and torch.equal(k, expect_k)
    pa.pa_rope(q, k, q, k, pos, -f, layout)
    # turned twice: 2 * 2 * (2^-22 + 2^-23) of the row's largest, and two fp32 roundings
    assert (q - q0).abs().max() <= 4 * (2.0 ** -22 + 2.0 ** -23 + 2.0 ** -24) * q0.abs().max() * 2
    assert (k - k0).abs().max() <= 4 * (2.0 ** -22 + 2.0 ** -23 + 2.0 ** -24) * k0.abs().max() * 2


@pytest.mark.parametrize("pos", [[-1, -100000], [2 ** 31, 2 ** 31 + 1], [2 ** 40 + 12345, 2 ** 20 + 1], [0, 1]])
def test_rope_far_and_negative_positions(pa, pos):
    """|p| 2^-53 f radians: what inv_freq's own 53 bits leave of the angle at p = 2^40 is 2^-12 of one."""
    q, k, _ = rows(2, 4, 1, 64, "f32", 11, False)
    f = pa.pa_rope_frequencies(64)[0]
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope(qo, ko, q, k, torch.tensor(pos, device="cuda"), f.cuda())
    ref = masked.rope(f64(q), pos, f.numpy(), False)
    slack = 2 * np.abs(f64(q)).max() * max(abs(p) for p in pos) * 2.0 ** -52
    assert np.all(np.abs(f64(qo) - ref) <= turned_bound(f64(q), ref, "f32", 1.0) + slack)


def test_rope_of_frequencies_past_a_turn(pa):
    q, k, _ = rows(5, 2, 1, 64, "f32", 13, False)
    f = torch.linspace(-9.0, 9.0, 32, dtype=torch.float64)
    pos = np.array([0, 1, 2, 1000, 12345])
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pa.pa_rope(qo, ko, q, k, torch.from_numpy(pos).cuda(), f.cuda())
    check_rows(qo, q, masked.rope(f64(q), pos, f.numpy(), False), "f32", 1.0, 64, "q")


WRITES = [  # tokens, heads, kv heads, head size, rotary dims, rows, pool, block size, fused, padded
    (1, 4, 1, 64, 64, "f16", "f16", 16, True, False),
    (3, 8, 2, 128, 128, "bf16", "bf16", 16, True, True),
    (16, 8, 8, 64, 32, "f32", "f32", 16, False, False),
    (37, 28, 4, 128, 128, "f16", "fp8", 16, True, True),
    (64, 5, 5, 128, 64, "bf16", "fp8", 32, False, False),
    (100, 4, 2, 64, 48, "f32", "fp8", 32, True, True),
    (129, 7, 1, 128, 112, "f16", "f16", 32, True, True),
    (700, 32, 8, 128, 128, "bf16", "bf16", 32, False, True),
    (2050, 12, 3, 64, 64, "f16", "f16", 16, True, False),
    (50, 4, 2, 64, 64, "f16", "f16", 7, True, True),      # the write path takes any block size
    (40, 4, 2, 128, 128, "bf16", "fp8", 1, False, True),
]


def e4m3_step(x):
    """Half a step of E4M3 at |x| (normal: 2^-4 relative to the power of two; 2^-10 below 2^-6), and clamping."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    return 2.0 ** (np.minimum(e, 8) - 4)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("case", WRITES, ids=lambda c: "-".join(map(str, c)))
def test_rope_and_cache(pa, case, pairs):
    t, h, hkv, d, r, dtype, cdt, bs, fused, padded = case
    rng = np.random.default_rng(t + d)
    q, k, v = rows(t, h, hkv, d, dtype, t, fused)
    pos = positions(t, t, 131072)
    nb = -(-t // bs) + 5
    if t <= 64:
        slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    else:
        slots = (rng.permutation(nb)[np.arange(t) // bs] * bs + np.arange(t) % bs).astype(np.int64)
    if padded:
        slots[:-1][rng.random(t - 1) < 0.2] = -1
        slots[0] = -7
    ks, vs = (0.0173, 0.0214) if cdt == "fp8" else (1.0, 1.0)
    x = 16 // {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}[cdt]
    fill = torch.from_numpy(rng.integers(0, 120, (2, nb, hkv, d, bs, tdtype(cdt).itemsize)).astype(np.uint8))
    kc = fill[0].cuda().view(torch.uint8).view(tdtype(cdt)).view(nb, hkv, d // x, bs, x)
    vc = fill[1].cuda().view(torch.uint8).view(tdtype(cdt)).view(nb, hkv, d, bs)
    k0, v0 = kc.clone(), vc.clone()
    f, _ = pa.pa_rope_frequencies(r, 10000.0)
    qo = torch.full((t, h, d), 7.0, dtype=q.dtype, device="cuda")
    pa.pa_rope_and_cache(qo, q, k, v, kc, vc, torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), f.cuda(),
                         pa.ROPE_PAIRS if pairs else pa.ROPE_HALVES, 1.0, ks, vs)
    assert pa.pa_get_device_error() == 0
    check_rows(qo, q, masked.rope(f64(q), pos, f.numpy(), pairs), dtype, 1.0, r, "q")
    keep = np.nonzero(slots >= 0)[0]
    blk, off = slots[keep] // bs, slots[keep] % bs
    # as bytes, so that NaN patterns in the pools compare
    kb, vb = (c.view(torch.uint8).cpu().numpy() for c in (kc, vc))
    kb0, vb0 = (c.view(torch.uint8).cpu().numpy() for c in (k0, v0))
    e = tdtype(cdt).itemsize
    vb, vb0 = vb.reshape(nb, hkv, d, bs, e), vb0.reshape(nb, hkv, d, bs, e)
    got_k = f64(kc.float())[blk, :, :, off].reshape(len(keep), hkv, d)
    ref_k = masked.rope(f64(k), pos, f.numpy(), pairs)[keep]
    xk = f64(k)[keep]
    if cdt == "fp8":
        s = float(np.float32(ks))
        # the quotient's fp32 rounding and the turned key's error move it across a border at most
        ref = np.clip(ref_k / s, -448, 448)
        slack = turned_bound(xk, ref_k, "f32", 1.0) / s + np.abs(ref) * 2.0 ** -23
        assert np.all(np.abs(got_k - ref) <= e4m3_step(ref) + slack)
        exact_v = (f64(v)[keep] / float(np.float32(vs))).astype(np.float32)
        want = torch.from_numpy(exact_v).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert np.array_equal(vb[blk, :, :, off, 0], want.view(torch.uint8).numpy())
    else:
        check_rows(torch.from_numpy(got_k), torch.from_numpy(xk), ref_k, dtype, 1.0, r, "key")
        assert np.array_equal(vb[blk, :, :, off], v[torch.from_numpy(keep).cuda()].contiguous().view(torch.uint8).cpu()
                              .numpy().reshape(len(keep), hkv, d, e))
    # nothing else in the pools changes
    kb[blk, :, :, off] = kb0[blk, :, :, off]
    vb[blk, :, :, off] = vb0[blk, :, :, off]
    assert np.array_equal(kb, kb0) and np.array_equal(vb, vb0)


def test_the_write_equals_rope_then_write(pa):
    """16-bit pools: the same bits as the rows turned by pa_rope and written by pa_reshape_and_cache."""
    for dtype, t in (("f16", 33), ("bf16", 1025)):
        q, k, v = rows(t, 8, 2, 128, dtype, 21, True)
        pos = torch.from_numpy(positions(t, 22, 5000)).cuda()
        f = pa.pa_rope_frequencies(128)[0].cuda()
        slots = torch.from_numpy(np.random.default_rng(5).permutation(16 * 70)[:t].astype(np.int64)).cuda()
        pools = [torch.zeros(70, 2, 16, 16, 8, dtype=q.dtype, device="cuda") for _ in range(2)]
        vpools = [torch.zeros(70, 2, 128, 16, dtype=q.dtype, device="cuda") for _ in range(2)]
        qo = [torch.empty(t, 8, 128, dtype=q.dtype, device="cuda") for _ in range(2)]
        ko = torch.empty(t, 2, 128, dtype=q.dtype, device="cuda")
        pa.pa_rope_and_cache(qo[0], q, k, v, pools[0], vpools[0], pos, slots, f)
        pa.pa_rope(qo[1], ko, q, k, pos, f)
        pa.pa_reshape_and_cache(ko, v.contiguous(), pools[1], vpools[1], slots)
        assert torch.equal(qo[0], qo[1]) and torch.equal(pools[0], pools[1]) and torch.equal(vpools[0], vpools[1])


def test_a_slot_past_the_pool_is_recorded_and_skipped(pa):
    q, k, v = rows(4, 2, 1, 64, "f16", 31, True)
    kc = torch.zeros(2, 1, 8, 16, 8, dtype=torch.float16, device="cuda")
    vc = torch.zeros(2, 1, 64, 16, dtype=torch.float16, device="cuda")
    qo = torch.empty(4, 2, 64, dtype=torch.float16, device="cuda")
    pos = torch.arange(4, device="cuda")
    slots = torch.tensor([0, 32, 2 ** 62, 5], device="cuda")
    pa.pa_rope_and_cache(qo, q, k, v, kc, vc, pos, slots, pa.pa_rope_frequencies(64)[0].cuda())
    assert pa.pa_get_device_error() == 3
    assert (vc[0, 0, :, 5] == v[3, 0]).all() and (vc[0, 0, :, 0] == v[0, 0]).all()
    vc[0, 0, :, [0, 5]] = 0
    assert not vc.any()


def test_rope_captured_and_on_another_stream(pa):
    q, k, v = rows(20, 8, 2, 128, "bf16", 41, True)
    f = pa.pa_rope_frequencies(128)[0].cuda()
    pos, slots = torch.arange(20, device="cuda"), torch.arange(20, device="cuda")
    kc = torch.zeros(3, 2, 16, 16, 8, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(3, 2, 128, 16, dtype=torch.bfloat16, device="cuda")
    qo = torch.empty(20, 8, 128, dtype=torch.bfloat16, device="cuda")

    def fresh(p, s):
        a, b, c = torch.zeros_like(kc), torch.zeros_like(vc), torch.empty_like(qo)
        pa.pa_rope_and_cache(c, q, k, v, a, b, p, s, f)
        return a, b, c

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_and_cache(qo, q, k, v, kc, vc, pos, slots, f, stream=side)
    side.synchronize()
    for a, b in zip((kc, vc, qo), fresh(pos, slots)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rope_and_cache(qo, q, k, v, kc, vc, pos, slots, f)
    pos += 1000
    slots.copy_(torch.arange(20, device="cuda").flip(0) + 9)
    kc.zero_(), vc.zero_()
    graph.replay()
    for a, b in zip((kc, vc, qo), fresh(pos, slots)):
        assert torch.equal(a, b)


@pytest.fixture(params=["extension", "ctypes"])
def path(request, monkeypatch):
    """Both of the binding's paths: the extension, and the Python code that takes its place."""
    from paged_kv_cache_306_gb300 import _binding as B
    if request.param == "extension":
        assert B._fp4_calls() is not None, "the extension was not built"
    else:
        monkeypatch.setattr(B, "_fp4_calls", lambda: None)
    return request.param


@pytest.mark.parametrize("t,h,hkv", [(1, 1, 1), (1, 4, 2), (9, 1, 1), (9, 4, 2)])
def test_both_paths_take_rows_that_lie_apart(pa, path, t, h, hkv):
    wide = torch.from_numpy(np.random.default_rng(3).standard_normal((t, h + 2 * hkv + 3, 64)).astype(np.float32)).cuda()
    q, k, v = wide[:, 1:h + 1], wide[:, h + 1:h + 1 + hkv], wide[:, h + 2 + hkv:h + 2 + 2 * hkv]
    pos, slots = torch.arange(t, device="cuda") + 7, torch.arange(t, device="cuda")
    f = pa.pa_rope_frequencies(64)[0].cuda()
    out = []
    for rows3 in ((q, k, v), (q.clone(), k.contiguous(), v.contiguous())):
        kc, vc = torch.zeros(1, hkv, 16, 16, 4, device="cuda"), torch.zeros(1, hkv, 64, 16, device="cuda")
        qo, ko = torch.empty(t, h, 64, device="cuda"), torch.empty(t, hkv, 64, device="cuda")
        pa.pa_rope_and_cache(qo, *rows3, kc, vc, pos, slots, f, amplitude=1.5)
        pa.pa_rope(qo, ko, *rows3[:2], pos, f, amplitude=1.5)
        out.append((qo, ko, kc, vc))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    check_rows(out[0][0], q, masked.rope(f64(q), np.arange(t) + 7, f.cpu().numpy(), False, 1.5), "f32", 1.5, 64, path)


def test_binding_refusals(pa, path):
    q, k, v = rows(4, 4, 2, 64, "f16", 51, False)
    f = pa.pa_rope_frequencies(64)[0].cuda()
    pos, slots = torch.arange(4, device="cuda"), torch.arange(4, device="cuda")
    kc = torch.zeros(2, 2, 8, 16, 8, dtype=torch.float16, device="cuda")
    vc = torch.zeros(2, 2, 64, 16, dtype=torch.float16, device="cuda")
    qo = torch.empty_like(q)
    good = dict(q_out=qo, q=q, key=k, value=v, k_cache=kc, v_cache=vc, positions=pos, slot_mapping=slots, inv_freq=f)
    pa.pa_rope_and_cache(**good)
    bad = [dict(q=q.transpose(0, 1)), dict(q=q[..., :32]), dict(q_out=torch.empty_like(q).transpose(0, 1)),
           dict(q_out=qo[:3]), dict(key=k[:3]), dict(key=k.float()), dict(value=v[:, :1]), dict(value=v[:3]),
           dict(positions=pos[:3]), dict(positions=pos.int()), dict(slot_mapping=slots[:3]),
           dict(inv_freq=f.float()), dict(inv_freq=f[:5]), dict(inv_freq=f[:0]), dict(k_cache=kc[:, :1]),
           dict(v_cache=vc[:1]), dict(k_cache=kc.bfloat16(), v_cache=vc.bfloat16()), dict(layout=5),
           dict(amplitude=float("nan")), dict(k_scale=2.0), dict(q=q.expand(4, 4, 64)[:1].expand(4, 4, 64)),
           dict(positions=pos.cpu()), dict(q=q.cpu())]
    for b in bad:
        with pytest.raises(pa.PAError):
            pa.pa_rope_and_cache(**{**good, **b})
    with pytest.raises(pa.PAError):
        pa.pa_rope(qo, torch.empty_like(k)[:3], q, k, pos, f)


@pytest.mark.parametrize("scale", [1.0, 0.0173, 3.7e-5, 1234.567, 2.0 ** -70, 3.1e25, 1e-30])
def test_codes_of_any_value_and_scale(pa, scale):
    """Values over all magnitudes, borders between codes, infinities and NaN: the codes that the write path stores."""
    t, d = 64, 64
    rng = np.random.default_rng(7)
    x = (rng.standard_normal(t * d) * 2.0 ** rng.integers(-14, 12, t * d)).astype(np.float32)
    grid = np.array([m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
    border = (grid[1:] + grid[:-1]) / 2
    near = np.concatenate([border, border * (1 + 2.0 ** -23), border * (1 - 2.0 ** -23), [448, 480, 464, 1e5, 0.0]])
    x[:len(near)] = near
    with np.errstate(over="ignore", under="ignore"):
        x = (x.astype(np.float64) * np.float64(np.float32(scale))).astype(np.float32)
    x[-8:] = [np.inf, -np.inf, np.nan, 3.4e38, -3.4e38, 1e-45, -1e-45, -0.0]
    v = torch.from_numpy(x.reshape(t, 1, d)).cuda()
    q = torch.zeros(t, 1, d, device="cuda")
    pools = [torch.zeros(4, 1, d // 16, 16, 16, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    vpools = [torch.zeros(4, 1, d, 16, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    slots, pos = torch.arange(t, device="cuda"), torch.zeros(t, dtype=torch.int64, device="cuda")
    f = pa.pa_rope_frequencies(16)[0].cuda()
    # position 0 turns nothing: x cos - y sin = x (an infinite or NaN partner apart, so k's turned dims are zero)
    k = v.clone()
    k[..., :16] = 0
    pa.pa_rope_and_cache(q, q, k, v, pools[0], vpools[0], pos, slots, f, k_scale=scale, v_scale=scale)
    pa.pa_reshape_and_cache_scaled(k, v, pools[1], vpools[1], slots, scale, scale)
    assert pa.pa_get_device_error() == 0
    for a, b in ((pools[0], pools[1]), (vpools[0], vpools[1])):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

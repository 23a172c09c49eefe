"""GPU parity of the FP4 cache calls against the oracle (oracle/fp4.py and the fp64 decode).

The write and the reads back are exact: the tiles' bytes, and the values rounded as
documented.  Decode is held to a bound derived per output row.  With w the exact
softmax weights, A = sum_t w_t |v_t|, L tokens and D dims:
  * a weight is rounded once to fp16: 2^-11 of it, or at most 2^-25 of the largest weight
    when it is below fp16's normal range -- 2^-11 A + L 2^-24 max|v| with room for the second;
  * a score is a sum of D fp32 products scaled once: off by at most
    d = (D + 8) 2^-23 * scale * |q| max|k| + 2^-20 (the exponential's own error included), which moves
    weights and their sum by that factor each -- 2 d A;
  * the weighted sums are accumulated in fp32, at most one addition per 8 tokens and a merge
    of partial results -- (L / 8 + 64) 2^-22 A;
  * the output is rounded once: half a step of its type.
"""
import math
import zlib

import numpy as np
import pytest

import oracle
import workloads as W
from helpers import TOL, as_f64, half_ulp, same_bytes
from oracle import fp4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KS, VS = 0.0173, 0.0214


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_306_gb300 as pa
    pa.load()


def rng_of(*key):
    return np.random.default_rng(zlib.crc32(repr(key).encode()))


def store(x, dtype):
    """float32 values rounded to the dtype: (numpy storage, float64 values)."""
    with np.errstate(over="ignore"):
        a = W.cast(np.asarray(x, np.float32), dtype)
    return a, oracle.widen(a, dtype)


def cuda(a, dtype=None):
    return W.to_torch(a, dtype, "cuda") if dtype else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def no_error():
    import paged_kv_cache_306_gb300 as pa
    code = pa.pa_get_device_error()
    assert code == 0, pa.DEVICE_ERRORS[code]


def rounded(v64, dtype):
    """fl_T(fl32(v)): what a read gives for an exact value."""
    with np.errstate(over="ignore"):
        return oracle.widen(W.cast(v64.astype(np.float32), dtype), dtype)


def random_pool(rng, NB, Hkv, D, bs, s, of, std=1.0):
    """(tiles, logical codes, logical scales): quantised normal rows whose channels differ in size."""
    x = rng.standard_normal((NB, Hkv, bs, D)).astype(np.float32) * std
    x *= np.exp(0.7 * rng.standard_normal((1, Hkv, 1, D))).astype(np.float32)
    c, f = fp4.quantise(x.astype(np.float64), s)
    return fp4.pack(c, f, of), c, f


# --- the write -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("scales", [(KS, VS), (2.0 ** -6, 2.0 ** -7), (1.0, 3.0e-5), (2.0 ** -64, 2.0 ** 64)])
def test_write_is_exact_and_touches_nothing_else(dtype, D, bs, scales):
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of(dtype, D, bs, scales)
    NB, Hkv, T = 23, 3, 77
    x = rng.standard_normal((2, T, Hkv, D)).astype(np.float32)
    x[:, :40] *= np.exp(2 * rng.standard_normal((2, 40, Hkv, D // 16))).repeat(16, -1)
    x[:, 8:16] *= 2.0 ** -11 * scales[0]         # scales that are subnormal codes, or zero
    x[:, 16:20] *= 2.0e4 * scales[0]             # past the largest code
    x[:, 20] = 0.0
    x[:, 21] = -0.0
    x[:, 22, :, 5] = np.nan
    x[:, 23, :, 17] = np.inf
    x[:, 24, :, 33] = -np.inf
    x[:, 25] = np.round(x[:, 25] * 4) / 4        # ties between codes
    x[:, 25, :, ::16] = 6.0
    (key, k64), (value, v64) = store(x[0], dtype), store(x[1], dtype)
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    slots[[3, 11]] = -1
    slots[12] = -(1 << 40)
    before = rng.integers(0, 256, (2, NB, Hkv, fp4.tile_bytes(D, bs)), dtype=np.uint8)
    kt, vt = cuda(before[0]), cuda(before[1])
    pa.pa_reshape_and_cache_fp4(cuda(key, dtype), cuda(value, dtype), kt, vt, cuda(slots), *scales)
    no_error()
    for of, got, rows, s, b in (("k", kt, k64, scales[0], before[0]), ("v", vt, v64, scales[1], before[1])):
        logical = fp4.unpack(b, D, bs, of)
        fp4.write(rows, logical, slots, s)
        assert np.array_equal(got.cpu().numpy(), fp4.pack(*logical, of)), of


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_write_and_read_of_many_rows(dtype):
    """More rows than a wave of CTAs; every fp16 / bf16 mantissa meets every scale mantissa many times."""
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("many", dtype)
    NB, Hkv, D, bs, T = 1300, 5, 128, 16, 20001
    x = (rng.standard_normal((2, T, Hkv, D)) * np.exp(rng.standard_normal((2, T, Hkv, 1)))).astype(np.float32)
    (key, k64), (value, v64) = store(x[0], dtype), store(x[1], dtype)
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    kt = torch.zeros(NB, Hkv, fp4.tile_bytes(D, bs), dtype=torch.uint8, device="cuda")
    vt = torch.zeros_like(kt)
    st = cuda(slots)
    pa.pa_reshape_and_cache_fp4(cuda(key, dtype), cuda(value, dtype), kt, vt, st, KS, VS)
    rk, rv = torch.empty_like(cuda(key, dtype)), torch.empty_like(cuda(key, dtype))
    pa.pa_gather_cache_fp4(rk, rv, kt, vt, st, KS, VS)
    no_error()
    for got, rows, s in ((rk, k64, KS), (rv, v64, VS)):
        want = rounded(fp4.values(*fp4.quantise(rows, s), s), dtype)
        assert np.array_equal(oracle.widen(W.from_torch(got, dtype), dtype), want)


def test_write_reports_a_slot_beyond_the_pool_and_writes_the_others():
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("slot")
    NB, Hkv, D, bs = 4, 2, 64, 16
    key, k64 = store(rng.standard_normal((4, Hkv, D)), "f16")
    kt = torch.zeros(NB, Hkv, fp4.tile_bytes(D, bs), dtype=torch.uint8, device="cuda")
    vt = torch.zeros_like(kt)
    slots = np.array([5, NB * bs, 1 << 45, 63], np.int64)
    pa.pa_reshape_and_cache_fp4(cuda(key, "f16"), cuda(key, "f16"), kt, vt, cuda(slots), KS, KS)
    assert pa.pa_get_device_error() == 3
    for of, got in (("k", kt), ("v", vt)):
        logical = fp4.unpack(np.zeros((NB, Hkv, fp4.tile_bytes(D, bs)), np.uint8), D, bs, of)
        fp4.write(k64, logical, [5, -1, -1, 63], KS)
        assert np.array_equal(got.cpu().numpy(), fp4.pack(*logical, of))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rows_that_start_on_16_bytes(dtype):
    """Row arrays on a 16-byte boundary that is none of 32 bytes are read by narrower loads: same bytes."""
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("offset", dtype)
    T, Hkv, D, bs = 50, 3, 128, 16
    key, value = (store(rng.standard_normal((T, Hkv, D)), dtype)[0] for _ in range(2))
    slots = cuda(rng.permutation(64)[:T].astype(np.int64))
    got = []
    for off in (0, 16):
        rows = []
        for x in (key, value):
            t = cuda(x, dtype)
            n = off // t.element_size()
            flat = torch.empty(t.numel() + n, dtype=t.dtype, device="cuda")
            flat[n:] = t.view(-1)
            rows.append(flat[n:].view(T, Hkv, D))
            assert rows[-1].data_ptr() % 32 == off
        pools = [torch.zeros(4, Hkv, fp4.tile_bytes(D, bs), dtype=torch.uint8, device="cuda") for _ in range(2)]
        pa.pa_reshape_and_cache_fp4(*rows, *pools, slots, KS, VS)
        got.append(pools)
    no_error()
    for a, b in zip(*got):
        assert torch.equal(a, b)


# --- the reads back -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_gather_is_exact_and_leaves_padded_rows(dtype, D, bs):
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("gather", dtype, D, bs)
    NB, Hkv, T = 9, 3, 133
    tiles = rng.integers(0, 256, (2, NB, Hkv, fp4.tile_bytes(D, bs)), dtype=np.uint8)   # any codes, any scale bytes
    slots = rng.integers(0, NB * bs, T).astype(np.int64)                                # repeats among them
    slots[[0, 50, T - 1]] = [-1, NB * bs, -7]
    rows = torch.full((2, T + 2, Hkv, D), 7.0, device="cuda").to(torch.float32 if dtype == "f32" else
                                                                 torch.float16 if dtype == "f16" else torch.bfloat16)
    pa.pa_gather_cache_fp4(rows[0, 1:-1], rows[1, 1:-1], cuda(tiles[0]), cuda(tiles[1]), cuda(slots), KS, VS)
    assert pa.pa_get_device_error() == 3
    for got, of, t, s in ((rows[0], "k", tiles[0], KS), (rows[1], "v", tiles[1], VS)):
        want = np.full((T + 2, Hkv, D), 7.0)
        v = rounded(fp4.pool_values(t, D, bs, of, s), dtype)
        for i, slot in enumerate(slots):
            if 0 <= slot < NB * bs:
                want[i + 1] = v[slot // bs, :, slot % bs]
        assert np.array_equal(oracle.widen(W.from_torch(got, dtype), dtype), want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_expand_is_exact_and_touches_nothing_else(dtype, D, bs):
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("expand", dtype, D, bs)
    NB, NBO, Hkv = 11, 17, 3
    tiles = rng.integers(0, 256, (2, NB, Hkv, fp4.tile_bytes(D, bs)), dtype=np.uint8)
    pairs = np.stack([rng.integers(0, NB, 9), rng.permutation(NBO)[:9]], 1).astype(np.int64)
    pairs = np.concatenate([pairs, [[NB, 3], [-1, 3], [2, NBO], [2, -5]]])                # four refused on the device
    td = torch.float16 if dtype == "f16" else torch.bfloat16
    ko = torch.full((NBO, Hkv, D // 8, bs, 8), 7.0, dtype=td, device="cuda")
    vo = torch.full((NBO, Hkv, D, bs), 7.0, dtype=td, device="cuda")
    pa.pa_expand_blocks_fp4(ko, vo, cuda(tiles[0]), cuda(tiles[1]), cuda(pairs), KS, VS)
    assert pa.pa_get_device_error() == 5
    k, v = np.full(ko.shape, 7.0), np.full(vo.shape, 7.0)
    kx = rounded(fp4.pool_values(tiles[0], D, bs, "k", KS), dtype)
    vx = rounded(fp4.pool_values(tiles[1], D, bs, "v", VS), dtype)
    for s, d in pairs[:9]:
        k[d] = kx[s].reshape(Hkv, bs, D // 8, 8).transpose(0, 2, 1, 3)
        v[d] = vx[s].transpose(0, 2, 1)
    assert np.array_equal(oracle.widen(W.from_torch(ko, dtype), dtype), k, equal_nan=True)
    assert np.array_equal(oracle.widen(W.from_torch(vo, dtype), dtype), v, equal_nan=True)


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32)])
def test_copy_blocks_moves_tiles(D, bs):
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("copy", D, bs)
    before = rng.integers(0, 256, (2, 12, 5, fp4.tile_bytes(D, bs)), dtype=np.uint8)
    kt, vt = cuda(before[0]), cuda(before[1])
    pairs = np.array([[0, 7], [0, 8], [3, 11]], np.int64)
    pa.pa_copy_blocks_fp4(kt, vt, cuda(pairs), D)
    no_error()
    want = before.copy()
    for s, d in pairs:
        want[:, d] = before[:, s]
    assert np.array_equal(kt.cpu().numpy(), want[0]) and np.array_equal(vt.cpu().numpy(), want[1])


# --- decode ------------------------------------------------------------------------------------------

class Case:
    """Sequences over shuffled blocks of random FP4 pools; slots past a sequence's end hold NaN scales."""

    def __init__(self, lens, G, Hkv, D, bs, q_dtype, *key, q_std=1.0, extra=3, std=1.0):
        rng = rng_of("decode", tuple(lens[:4]), len(lens), G, Hkv, D, bs, q_dtype, *key)
        self.lens, self.D, self.bs, self.Hkv, self.q_dtype = list(lens), D, bs, Hkv, q_dtype
        n = [-(-L // bs) for L in lens]
        NB = sum(n) + extra
        perm = rng.permutation(NB).astype(np.int32)
        self.table = np.full((len(lens), max(n) + 1), -1, np.int32)
        at = 0
        self.pools = []
        for of, s in (("k", KS), ("v", VS)):
            _, c, f = random_pool(rng, NB, Hkv, D, bs, s, of, std)
            self.pools.append((c, f))
        for i, m in enumerate(n):
            self.table[i, :m] = perm[at:at + m]
            at += m
            if m and lens[i] % bs:
                for c, f in self.pools:
                    c[self.table[i, m - 1], :, lens[i] % bs:] = 7
                    f[self.table[i, m - 1], :, lens[i] % bs:] = fp4.NAN_SCALE
        self.k, self.v = (fp4.pack(c, f, of) for (c, f), of in zip(self.pools, "kv"))
        q = rng.standard_normal((len(lens), G * Hkv, D)).astype(np.float32) * q_std
        self.q, self.q64 = store(q, q_dtype)
        self.scale = 1 / math.sqrt(D)
        self.max_len = max(max(lens), 1)

    def upload(self):
        return dict(q=cuda(self.q, self.q_dtype), k=cuda(self.k), v=cuda(self.v), table=cuda(self.table),
                    lens=cuda(np.array(self.lens, np.int32)))

    def run(self, t=None, out=None, max_len=None, **kw):
        import paged_kv_cache_306_gb300 as pa
        t = self.upload() if t is None else t
        out = torch.full_like(t["q"], math.nan) if out is None else out
        pa.pa_decode_fp4(out, t["q"], t["k"], t["v"], t["table"], t["lens"], self.scale, max_len or self.max_len, KS,
                         VS, **kw)
        return out

    def reference(self, seqs=None):
        """(exact out, bound without the final rounding) [n, H, D]."""
        seqs = range(len(self.lens)) if seqs is None else seqs
        k64, v64 = fp4.f64_pools(self.k, self.v, self.D, self.bs, KS, VS)
        table, lens = self.table[list(seqs)], np.array(self.lens, np.int32)[list(seqs)]
        q = np.ascontiguousarray(self.q[list(seqs)])
        args = (table, lens, self.scale, "f64")
        out = oracle.decode(q, k64, v64, *args, q_dtype=self.q_dtype)
        mass = oracle.decode(q, k64, np.abs(v64), *args, q_dtype=self.q_dtype)
        kn = np.nanmax(np.sqrt((np.moveaxis(k64, 3, 2).reshape(*k64.shape[:2], self.bs, -1) ** 2).sum(-1)))
        qn = np.sqrt((self.q64[list(seqs)] ** 2).sum(-1, keepdims=True))
        d = (self.D + 8) * 2.0 ** -23 * abs(self.scale) * qn * kn + 2.0 ** -20
        L = lens.astype(np.float64)[:, None, None]
        rel = 2.0 ** -11 + 2 * d + (L / 8 + 64) * 2.0 ** -22
        return out, rel * mass + L * 2.0 ** -24 * np.nanmax(np.abs(v64))

    def check(self, out, seqs=None):
        got = as_f64(out)
        got = got if seqs is None else got[list(seqs)]
        ref, bound = self.reference(seqs)
        assert np.isfinite(got).all()
        excess = np.abs(got - ref) - bound - half_ulp(np.abs(ref) + bound, self.q_dtype)
        assert excess.max() <= 0, f"off by {np.abs(got - ref).max():.3e}, {excess.max():.3e} past the bound"


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 130, 300]


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 16, 17, 40])
def test_decode_lengths_and_groups(q_dtype, D, bs, G):
    c = Case(EDGES, G, 2, D, bs, q_dtype)
    out = c.run()
    no_error()
    c.check(out)


@pytest.mark.parametrize("q_dtype,D,bs,G,Hkv,lens", [
    ("f16", 128, 16, 7, 4, [4096, 512, 1000, 2047, 1]),
    ("bf16", 128, 16, 4, 8, [9001]),
    ("bf16", 64, 32, 10, 1, [20000, 3]),
    ("f16", 64, 16, 1, 5, [1, 1, 1, 7000, 1]),
    ("f16", 128, 32, 20, 1, [5000, 4999, 5001]),
    ("f16", 128, 16, 1, 32, [513, 600]),
    ("f16", 64, 16, 2, 1, [150001]),                  # one segment over every CTA
    ("bf16", 128, 16, 1, 1, [3, 60000, 1]),
])
def test_decode_long_and_ragged(q_dtype, D, bs, G, Hkv, lens):
    c = Case(lens, G, Hkv, D, bs, q_dtype)
    out = c.run()
    no_error()
    c.check(out)


@pytest.mark.parametrize("S,G,Hkv,D,bs", [(1, 4, 2, 128, 16), (1500, 2, 2, 64, 16), (2100, 1, 1, 128, 32),
                                         (1024, 8, 1, 64, 32), (1025, 16, 1, 64, 16)])
def test_decode_many_sequences(S, G, Hkv, D, bs):
    rng = rng_of("many", S)
    c = Case([int(x) for x in rng.integers(1, 90, S)], G, Hkv, D, bs, "f16")
    out = c.run()
    no_error()
    c.check(out)


@pytest.mark.parametrize("S", [1, 7, 30, 200])
@pytest.mark.parametrize("longest", [20, 60, 200, 500, 900])
@pytest.mark.parametrize("G,Hkv,D,bs", [(4, 2, 128, 16), (10, 3, 64, 32)])
def test_decode_batches_of_short_sequences(S, longest, G, Hkv, D, bs):
    """Segments from much shorter to much longer than a CTA's share: whole ones a CTA, or cut at CTAs' ends."""
    lens = [int(x) for x in rng_of("short", S, longest, G).integers(1, longest + 1, S)]
    c = Case(lens, G, Hkv, D, bs, "f16", longest)
    out = c.run()
    no_error()
    c.check(out)


def test_decode_with_a_loose_length_bound():
    """max_seq_len far above the lengths: the tables are wide, the sequences short."""
    c = Case([5, 40, 100], 4, 2, 128, 16, "f16")
    c.table = np.concatenate([c.table, np.full((3, 3000), -1, np.int32)], 1)
    out = c.run(max_len=16 * 2000)
    no_error()
    c.check(out)


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
def test_decode_heads_of_very_different_size(q_dtype):
    """bf16 heads from 2^-20 to 2^20 (fp16 from 2^-10 to 2^6), peaked softmaxes among them."""
    c = Case([1, 77, 200], 8, 2, 128, 16, q_dtype)
    span = np.linspace(-20, 20, 16) if q_dtype == "bf16" else np.linspace(-10, 6, 16)
    c.q, c.q64 = store(oracle.widen(c.q, q_dtype).astype(np.float32) * (2.0 ** np.round(span))[None, :, None], q_dtype)
    out = c.run()
    no_error()
    got = as_f64(out)
    ref, bound = c.reference()
    # a peaked head's weights move with the score's error: heads whose error exceeds 1/8 are held to the range of V
    fine = bound < 0.125 * np.abs(ref).max()
    excess = np.abs(got - ref) - bound - half_ulp(np.abs(ref) + bound, q_dtype)
    assert np.isfinite(got).all() and fine.mean() > 0.4 and excess[fine].max() <= 0


def test_lengths_outside_the_contract_give_zero_rows_and_an_error():
    import paged_kv_cache_306_gb300 as pa
    c = Case([40, 17, 90, 33], 4, 2, 64, 16, "f16")
    t = c.upload()
    t["lens"] = cuda(np.array([40, 0, -3, 91], np.int32))
    out = c.run(t)
    assert pa.pa_get_device_error() == 2
    assert not out[1:].any()
    c.check(out, [0])
    t["lens"].zero_()
    out = c.run(t)
    assert pa.pa_get_device_error() == 2 and not out.any()


def test_block_ids_outside_the_pool_are_reported():
    import paged_kv_cache_306_gb300 as pa
    for bad in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        c = Case([40, 90, 100], 4, 2, 64, 16, "f16")
        c.table[1, 3] = bad
        out = c.run()
        assert pa.pa_get_device_error() == 1
        c.check(out, [0, 2])


def test_placement_and_repetition_do_not_change_a_bit():
    c = Case([700, 33, 1, 4000], 7, 2, 128, 16, "bf16", extra=40)
    a = c.run()
    assert same_bytes(a, c.run())
    rng = rng_of("move")
    to = rng.permutation(len(c.k)).astype(np.int32)
    k, v = np.empty_like(c.k), np.empty_like(c.v)
    k[to], v[to] = c.k, c.v
    c.k, c.v, c.table = k, v, np.where(c.table >= 0, to[c.table], -1).astype(np.int32)
    assert same_bytes(a, c.run())
    no_error()


def test_decode_writes_only_its_rows_and_its_workspace():
    import paged_kv_cache_306_gb300 as pa
    c = Case([700, 33, 1, 1500], 10, 2, 128, 16, "f16")
    t = c.upload()
    big = torch.full((8,) + t["q"].shape[1:], math.nan, dtype=torch.float16, device="cuda")
    need = pa.pa_decode_fp4_workspace_size(4, 20, 2, 128, c.max_len, 16)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    before = {n: x.clone() for n, x in t.items()}
    c.run(t, out=big[2:6], workspace=ws[256:256 + need] if need else None)
    no_error()
    assert torch.isnan(big[:2]).all() and torch.isnan(big[6:]).all()
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + need:] == 0xA5).all())
    assert all(same_bytes(before[n], t[n]) for n in t)
    c.check(big[2:6])


def test_a_short_workspace_is_refused():
    import paged_kv_cache_306_gb300 as pa
    c = Case([1000, 800], 4, 2, 128, 16, "f16")
    t = c.upload()
    need = pa.pa_decode_fp4_workspace_size(2, 8, 2, 128, c.max_len, 16)
    if not need:
        return
    lib, B = pa.load(), pa._binding
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(t["q"])
    for ptr, n, status in ((ws.data_ptr(), need - 1, B.PA_ERR_WORKSPACE), (0, need, B.PA_ERR_WORKSPACE),
                           (ws.data_ptr() + 8, need, B.PA_ERR_ALIGNMENT)):
        st = lib.pa_decode_fp4(out.data_ptr(), t["q"].data_ptr(), t["k"].data_ptr(), t["v"].data_ptr(),
                               t["table"].data_ptr(), t["table"].shape[1], t["lens"].data_ptr(), 2, c.max_len, 8, 2,
                               128, 16, c.k.shape[0], c.scale, ptr, n, B.PA_F16, KS, VS, None)
        assert st == status


def test_a_captured_call_follows_its_inputs():
    """One captured call replayed over growing, shrinking and equal batches; the workspace and the pools
    keep what the last replay left."""
    import paged_kv_cache_306_gb300 as pa
    cases = [Case(lens, 4, 2, 128, 16, "f16", extra=0) for lens in
             ([3000, 1, 500, 2999], [1, 1, 1, 1], [2000, 2000, 2000, 2000], [17, 3000, 1, 64], [1, 1, 1, 3000])]
    blocks = max(len(c.k) for c in cases)
    width = max(c.table.shape[1] for c in cases)
    t = dict(q=torch.empty(4, 8, 128, dtype=torch.float16, device="cuda"),
             k=torch.empty((blocks,) + cases[0].k.shape[1:], dtype=torch.uint8, device="cuda"),
             table=torch.full((4, width), -1, dtype=torch.int32, device="cuda"),
             lens=torch.ones(4, dtype=torch.int32, device="cuda"))
    t["v"] = torch.empty_like(t["k"])

    def load(c):
        u = c.upload()
        for n in ("q", "lens"):
            t[n].copy_(u[n])
        t["table"].fill_(-1)
        t["table"][:, :c.table.shape[1]] = u["table"]
        for n in ("k", "v"):
            t[n][:len(c.k)] = u[n]

    out = torch.empty_like(t["q"])
    need = pa.pa_decode_fp4_workspace_size(4, 8, 2, 128, 3000, 16)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    load(cases[0])
    cases[0].run(t, out=out, max_len=3000, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cases[0].run(t, out=out, max_len=3000, workspace=ws)
    for c in cases + cases[::-1]:
        load(c)
        out.fill_(math.nan)
        g.replay()
        no_error()
        c.check(out)


def test_two_captured_steps_share_a_workspace_and_pools():
    """A step (write, block copy, decode, reads back) captured twice, for batches of different shapes, on one
    workspace and one pair of pools; replayed in turn on a side stream with new rows, slots and lengths."""
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("steps")
    Hkv, D, bs, NB = 2, 128, 16, 600
    kt = torch.full((NB, Hkv, fp4.tile_bytes(D, bs)), 0xFF, dtype=torch.uint8, device="cuda")
    vt = torch.full_like(kt, 0xFF)
    logical = [fp4.unpack(x.cpu().numpy(), D, bs, of) for x, of in ((kt, "k"), (vt, "v"))]
    first = [store(rng.standard_normal((NB * bs, Hkv, D)), "f16") for _ in range(2)]
    every = np.arange(NB * bs, dtype=np.int64)
    pa.pa_reshape_and_cache_fp4(cuda(first[0][0], "f16"), cuda(first[1][0], "f16"), kt, vt, cuda(every), KS, VS)
    for rows, lg, s in zip(first, logical, (KS, VS)):
        fp4.write(rows[1], lg, every, s)
    shapes = [(4, 8, 2100), (2, 2, 4000)]       # sequences, heads, longest
    ws = torch.empty(max(pa.pa_decode_fp4_workspace_size(S, H, Hkv, D, L, bs) for S, H, L in shapes), dtype=torch.uint8,
                     device="cuda")
    f16, i64 = dict(dtype=torch.float16, device="cuda"), dict(dtype=torch.int64, device="cuda")
    steps = []
    for S, H, L in shapes:
        t = dict(key=torch.zeros(S, Hkv, D, **f16), value=torch.zeros(S, Hkv, D, **f16), slots=torch.full((S,), -1, **i64),
                 pairs=torch.zeros(1, 2, **i64), q=torch.zeros(S, H, D, **f16), out=torch.zeros(S, H, D, **f16),
                 table=torch.zeros(S, L // bs + 1, dtype=torch.int32, device="cuda"),
                 lens=torch.ones(S, dtype=torch.int32, device="cuda"), rk=torch.zeros(S, Hkv, D, **f16),
                 rv=torch.zeros(S, Hkv, D, **f16), ko=torch.zeros(2, Hkv, D // 8, bs, 8, **f16),
                 vo=torch.zeros(2, Hkv, D, bs, **f16), expand=torch.zeros(1, 2, **i64))

        def step(t=t, L=L):
            pa.pa_copy_blocks_fp4(kt, vt, t["pairs"], D)
            pa.pa_reshape_and_cache_fp4(t["key"], t["value"], kt, vt, t["slots"], KS, VS)
            pa.pa_decode_fp4(t["out"], t["q"], kt, vt, t["table"], t["lens"], 0.09, L, KS, VS, ws)
            pa.pa_gather_cache_fp4(t["rk"], t["rv"], kt, vt, t["slots"], KS, VS)
            pa.pa_expand_blocks_fp4(t["ko"], t["vo"], kt, vt, t["expand"], KS, VS)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        steps.append((t, g))
    side = torch.cuda.Stream()
    for rep in range(6):
        i = rep % 2
        (S, H, L), (t, g) = shapes[i], steps[i]
        c = Case([int(x) for x in rng.integers(1, L, S - 1)] + [L - rep], H // Hkv, Hkv, D, bs, "f16", rep)
        need = [-(-x // bs) for x in c.lens]
        perm = rng.permutation(NB - 2)[:sum(need)].astype(np.int32) + 2
        c.table = np.zeros((S, L // bs + 1), np.int32)
        for s in range(S):
            c.table[s, :need[s]] = perm[sum(need[:s]):sum(need[:s + 1])]
        slots = np.array([c.table[s, (x - 1) // bs] * bs + (x - 1) % bs for s, x in enumerate(c.lens)], np.int64)
        new = [store(rng.standard_normal((S, Hkv, D)), "f16") for _ in range(2)]
        src = int(perm[0])
        for lg, rows, sc in zip(logical, new, (KS, VS)):
            for part in lg:
                part[rep % 2] = part[src]
            fp4.write(rows[1], lg, slots, sc)
        for n, v in (("key", cuda(new[0][0], "f16")), ("value", cuda(new[1][0], "f16")), ("slots", cuda(slots)),
                     ("pairs", cuda(np.array([[src, rep % 2]], np.int64))), ("q", cuda(c.q, "f16")),
                     ("table", cuda(c.table)), ("lens", cuda(np.array(c.lens, np.int32))),
                     ("expand", cuda(np.array([[src, 1]], np.int64)))):
            t[n].copy_(v)
        t["out"].fill_(math.nan)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        no_error()
        c.scale, c.max_len = 0.09, L
        c.k, c.v = fp4.pack(*logical[0], "k"), fp4.pack(*logical[1], "v")
        assert np.array_equal(kt.cpu().numpy(), c.k) and np.array_equal(vt.cpu().numpy(), c.v)
        c.check(t["out"])
        for got, rows, sc in ((t["rk"], new[0], KS), (t["rv"], new[1], VS)):
            assert np.array_equal(as_f64(got), rounded(fp4.values(*fp4.quantise(rows[1], sc), sc), "f16"))
        assert np.array_equal(as_f64(t["vo"][1]).transpose(0, 2, 1),
                              rounded(fp4.pool_values(c.v[src:src + 1], D, bs, "v", VS), "f16")[0])


def test_lengths_and_tables_written_right_before_the_call():
    """The kernel may look at both while the previous kernel still runs: what that one writes must count."""
    cases = [Case(lens, 4, 2, 128, 16, "f16", i, extra=0) for i, lens in
             enumerate(([3000, 1, 500, 2999], [1, 1, 1, 1], [17, 3000, 1, 64], [800, 790, 30, 2000]))]
    width = max(c.table.shape[1] for c in cases)
    ups = [c.upload() for c in cases]
    tables = []
    for u in ups:
        t = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
        t[:, :u["table"].shape[1]] = u["table"]
        tables.append(t)
    lens, table = torch.ones(4, dtype=torch.int32, device="cuda"), torch.zeros_like(tables[0])
    outs = []
    for rep in range(12):
        i = rep % 4
        u = ups[i]
        pad = torch.zeros(1 << 24, device="cuda").cumsum(0)     # a kernel before, so that the host runs ahead
        table.copy_(tables[i])
        lens.copy_(u["lens"])
        outs.append((i, cases[i].run(dict(u, table=table, lens=lens), max_len=3000)))
        if rep >= 8:                                            # a call of the library in between
            outs.append((i, cases[i].run(dict(u, table=table, lens=lens), max_len=3000)))
        del pad
    no_error()
    for i, out in outs:
        cases[i].check(out)


def test_calls_on_two_streams_with_their_own_workspaces():
    cases = [Case([2500, 100, 64], 4, 2, 128, 16, "f16"), Case([300, 2500], 4, 4, 128, 16, "f16", 2)]
    ts = [c.upload() for c in cases]
    outs = [torch.full_like(t["q"], math.nan) for t in ts]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, t, o, s in zip(cases, ts, outs, streams):
            c.run(t, out=o, stream=s)      # each takes a workspace of its own, on a stream that is not current
    torch.cuda.synchronize()
    no_error()
    for c, o in zip(cases, outs):
        c.check(o)


def test_two_host_threads_with_streams_of_their_own():
    """Writes, reads and decodes from two threads at once, each on its own stream, pools and workspaces."""
    import threading
    import paged_kv_cache_306_gb300 as pa
    cases = [Case([1200, 33, 700], 4, 2, 128, 16, "f16", "a"), Case([60, 2500], 4, 2, 64, 32, "bf16", "b")]
    ts = [c.upload() for c in cases]
    rows, failed = [], []
    for c, t in zip(cases, ts):     # every row read back and written again
        slots = cuda(np.arange(len(c.k) * c.bs, dtype=np.int64))
        rows.append((slots, *(torch.empty(len(slots), c.Hkv, c.D, device="cuda") for _ in range(2))))
    outs = [torch.full_like(t["q"], math.nan) for t in ts]
    torch.cuda.synchronize()

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                slots, k, v = rows[i]
                for _ in range(25):
                    pa.pa_gather_cache_fp4(k, v, ts[i]["k"], ts[i]["v"], slots, KS, VS)
                    pa.pa_reshape_and_cache_fp4(k, v, ts[i]["k"], ts[i]["v"], slots, KS, VS)
                    cases[i].run(ts[i], out=outs[i])
            stream.synchronize()
        except Exception as e:      # reported by the main thread
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    no_error()
    for c, o, t in zip(cases, outs, ts):
        c.k, c.v = t["k"].cpu().numpy(), t["v"].cpu().numpy()
        c.check(o)


def test_many_kv_heads():
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("heads")
    T, Hkv, D, bs, NB = 20, 1001, 64, 16, 3
    (key, k64), (value, v64) = (store(rng.standard_normal((T, Hkv, D)), "bf16") for _ in range(2))
    kt = torch.zeros(NB, Hkv, fp4.tile_bytes(D, bs), dtype=torch.uint8, device="cuda")
    vt = torch.zeros_like(kt)
    slots = np.concatenate([np.arange(32, 48), np.arange(4)]).astype(np.int64)    # blocks 2 and 0
    pa.pa_reshape_and_cache_fp4(cuda(key, "bf16"), cuda(value, "bf16"), kt, vt, cuda(slots), KS, VS)
    rk, rv = torch.empty(2, T, Hkv, D, device="cuda")
    pa.pa_gather_cache_fp4(rk, rv, kt, vt, cuda(slots), KS, VS)
    want = [rounded(fp4.values(*fp4.quantise(x, s), s), "f32") for x, s in ((k64, KS), (v64, VS))]
    assert np.array_equal(as_f64(rk), want[0]) and np.array_equal(as_f64(rv), want[1])
    ko = torch.zeros(2, Hkv, D // 8, bs, 8, dtype=torch.float16, device="cuda")
    vo = torch.zeros(2, Hkv, D, bs, dtype=torch.float16, device="cuda")
    pa.pa_expand_blocks_fp4(ko, vo, kt, vt, cuda(np.array([[2, 1]], np.int64)), KS, VS)
    assert np.array_equal(as_f64(vo[1]).transpose(2, 0, 1), rounded(want[1][:16], "f16"))
    c = Case([T], 1, Hkv, D, bs, "bf16", "heads", extra=1)
    c.table = np.array([[2, 0]], np.int32)
    c.k, c.v = kt.cpu().numpy(), vt.cpu().numpy()
    out = c.run()
    no_error()
    c.check(out)


def test_pools_past_32_bit_offsets():
    """Blocks at the end of pools of more than 4 GiB each: the write, both reads and decode."""
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("far")
    Hkv, D, bs, L = 8, 128, 32, 100
    NB = (1 << 32) // (Hkv * fp4.tile_bytes(D, bs)) + 5000
    kt = torch.empty(NB, Hkv, fp4.tile_bytes(D, bs), dtype=torch.uint8, device="cuda")
    vt = torch.empty_like(kt)
    blocks = np.array([NB - 1, NB - 3, 2, NB - 2])
    slots = np.array([int(blocks[t // bs]) * bs + t % bs for t in range(L)], np.int64)
    (key, k64), (value, v64) = (store(rng.standard_normal((L, Hkv, D)), "f16") for _ in range(2))
    pa.pa_reshape_and_cache_fp4(cuda(key, "f16"), cuda(value, "f16"), kt, vt, cuda(slots), KS, VS)
    rk, rv = torch.empty(2, L, Hkv, D, dtype=torch.float16, device="cuda")
    pa.pa_gather_cache_fp4(rk, rv, kt, vt, cuda(slots), KS, VS)
    no_error()
    want = fp4.values(*fp4.quantise(k64, KS), KS), fp4.values(*fp4.quantise(v64, VS), VS)
    assert np.array_equal(as_f64(rk), rounded(want[0], "f16")) and np.array_equal(as_f64(rv), rounded(want[1], "f16"))
    ko = torch.zeros(5, Hkv, D // 8, bs, 8, dtype=torch.float16, device="cuda")
    vo = torch.zeros(5, Hkv, D, bs, dtype=torch.float16, device="cuda")
    pa.pa_expand_blocks_fp4(ko, vo, kt, vt, cuda(np.array([[NB - 3, 4]], np.int64)), KS, VS)
    no_error()
    assert np.array_equal(as_f64(vo[4]).transpose(2, 0, 1), rounded(want[1][32:64], "f16"))
    c = Case([L], 2, Hkv, D, bs, "f16", "far", extra=0)
    c.table = np.arange(4, dtype=np.int32)[None]
    small = [torch.stack([p[int(b)] for b in blocks]) for p in (kt, vt)]
    c.k, c.v = (p.cpu().numpy() for p in small)
    for p, of in ((c.k, "k"), (c.v, "v")):   # what lies past the sequence was never written: give it values for the bound
        codes, f = fp4.unpack(p, D, bs, of)
        f[3, :, L - 96:] = 0
        p[...] = fp4.pack(codes, f, of)
    t = c.upload()
    t.update(k=kt, v=vt, table=cuda(blocks.astype(np.int32)[None]))
    out = c.run(t)
    no_error()
    c.check(out)


@pytest.mark.parametrize("lens,G,D", [([1, 17, 300, 2500, 40, 900], 7, 128), ([6000, 5000], 12, 64), ([40000], 1, 128)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_correct(lens, G, D):
    """Every CTA that waits for pieces of other CTAs waits for a tag nobody writes, for 2 ms: the wait runs
    out, the call returns."""
    import paged_kv_cache_306_gb300 as pa
    c = Case(lens, G, 2, D, 16, "f16")
    t = c.upload()
    need = pa.pa_decode_fp4_workspace_size(len(lens), 2 * G, 2, D, c.max_len, 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    try:
        pa.pa_set_test_wait_limit(2_000_000)
        c.run(t, workspace=ws)
    finally:
        pa.pa_set_test_wait_limit(0)
    assert pa.pa_get_device_error() == 4 and pa.pa_get_device_error() == 0
    out = c.run(t, workspace=ws)
    no_error()
    c.check(out)


@pytest.mark.parametrize("fill", [0x00, 0xFF, 0xA5])
def test_a_workspace_may_hold_anything(fill):
    import paged_kv_cache_306_gb300 as pa
    c = Case([5000, 1, 900, 3000], 4, 2, 128, 16, "f16")
    t = c.upload()
    ws = torch.full((pa.pa_decode_fp4_workspace_size(4, 8, 2, 128, 5000, 16),), fill, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        out = c.run(t, workspace=ws)
    no_error()
    c.check(out)
    short = Case([70, 2000], 8, 2, 64, 32, "bf16")       # another shape on the same workspace, and back
    short.check(short.run(workspace=ws))
    c.check(c.run(t, workspace=ws))
    no_error()


def test_a_nan_in_the_cache_reaches_its_own_rows_only():
    """A NaN scale of one token of one kv head: in K every query head of it, in V the 16 dims of its group."""
    import paged_kv_cache_306_gb300 as pa
    c = Case([300, 40, 700], 3, 2, 128, 16, "f16")
    clean = c.run()
    t = c.upload()
    (kc, kf), (vc, vf) = ((x.copy(), f.copy()) for x, f in c.pools)
    kf[c.table[0, 4], 1, 7, 2] = fp4.NAN_SCALE
    vf[c.table[2, 30], 0, 3, 5] = fp4.NAN_SCALE
    t["k"], t["v"] = cuda(fp4.pack(kc, kf, "k")), cuda(fp4.pack(vc, vf, "v"))
    out = c.run(t)
    no_error()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 3:] = True                      # query heads 3 .. 5 read kv head 1
    bad[2, :3, 80:96] = True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("wrong", [math.nan, math.inf])
def test_a_query_that_is_no_number_spoils_its_own_rows_only(q_dtype, wrong):
    c = Case([300, 40, 9000], 3, 2, 128, 16, q_dtype)
    t = c.upload()
    t["q"][0, 1, 77] = t["q"][2, 5, 0] = wrong
    out = c.run(t)
    no_error()
    assert not math.isnan(wrong) or (torch.isnan(out[0, 1]).all() and torch.isnan(out[2, 5]).all())
    ref = cuda(c.reference()[0]).to(out.dtype)
    out[0, 1], out[2, 5] = ref[0, 1], ref[2, 5]
    c.check(out)


@pytest.mark.parametrize("scale", [0.0, -0.09, 3.0e-5])
def test_decode_scales_of_any_sign(scale):
    c = Case([1, 40, 333], 3, 2, 64, 16, "bf16")
    c.scale = scale
    out = c.run()
    no_error()
    c.check(out)


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [2.0 ** 10, -2.0 ** 24, 2.0 ** 40, 2.0 ** 63])
def test_scores_of_any_size_leave_the_largest(q_dtype, scale):
    """q of -1, 0 and 1 and scales sf of 1: every score is a sum of at most 128 codes, exact in fp32, and
    two that differ do so by 1/2 at least, 2^9 and more after the softmax's scale.  So the answer is the mean of the
    V rows whose score is the largest (the smallest for a negative scale), wherever their pieces are."""
    c = Case([1, 65, 3000, 20000], 2, 2, 128, 16, q_dtype, scale)
    (kc, kf), vp = c.pools
    kf[...] = 0x38                                            # sf = 1
    rng = rng_of("largest", scale)
    c.q = store(rng.integers(-1, 2, size=c.q.shape).astype(np.float64), q_dtype)[0]
    c.k = fp4.pack(kc, kf, "k")
    c.scale = scale / KS
    out = c.run()
    no_error()
    k64, v64 = fp4.f64_pools(c.k, c.v, 128, 16, KS, VS)
    args = (c.table, np.array(c.lens, np.int32), c.scale, "f64")
    ref, mass = (oracle.decode(c.q, k64, v, *args, q_dtype=q_dtype) for v in (v64, np.abs(np.nan_to_num(v64))))
    bound = (np.array(c.lens)[:, None, None] / 8 + 64) * 2.0 ** -22 * mass     # sums in fp32
    assert (np.abs(as_f64(out) - ref) - bound - half_ulp(np.abs(ref) + bound, q_dtype)).max() <= 0


# --- as they are used together ------------------------------------------------------------------------

def test_a_serving_run_over_an_fp4_cache():
    """Prompts in two chunks (quantising write; the context expanded for pa_prefill), then a fork and steps
    of copy-on-write, write and decode, the block manager handing out the blocks."""
    import paged_kv_cache_306_gb300 as pa
    rng = rng_of("serve")
    Hkv, G, D, bs, NB = 2, 4, 128, 16, 64
    H, scale = Hkv * G, 1 / math.sqrt(D)
    bm = pa.BlockManager(NB, bs)
    kt = torch.full((NB, Hkv, fp4.tile_bytes(D, bs)), 0xFF, dtype=torch.uint8, device="cuda")
    vt = torch.full_like(kt, 0xFF)
    logical = [fp4.unpack(kt.cpu().numpy(), D, bs, "k"), fp4.unpack(vt.cpu().numpy(), D, bs, "v")]
    rows = {}

    def write(slots):
        (key, k64), (value, v64) = (store(rng.standard_normal((len(slots), Hkv, D)), "f16") for _ in range(2))
        pa.pa_reshape_and_cache_fp4(cuda(key, "f16"), cuda(value, "f16"), kt, vt, cuda(slots), KS, VS)
        fp4.write(k64, logical[0], slots, KS)
        fp4.write(v64, logical[1], slots, VS)

    def pools64():
        return fp4.f64_pools(fp4.pack(*logical[0], "k"), fp4.pack(*logical[1], "v"), D, bs, KS, VS)

    # prompts: the second chunk attends to everything through 16-bit copies of the blocks
    for sid, n in ((0, 100), (1, 37)):
        rows[sid] = bm.add_sequence(sid, n)
    first = {0: 60, 1: 5}
    write(np.concatenate([rows[s][:first[s]] for s in (0, 1)]))
    write(np.concatenate([rows[s][first[s]:] for s in (0, 1)]))
    table, lens = bm.block_tables([0, 1], 8)
    used = np.unique(table[table >= 0]).astype(np.int64)
    ko = torch.zeros(NB, Hkv, D // 8, bs, 8, dtype=torch.float16, device="cuda")
    vo = torch.zeros(NB, Hkv, D, bs, dtype=torch.float16, device="cuda")
    pa.pa_expand_blocks_fp4(ko, vo, kt, vt, cuda(np.stack([used, used], 1)), KS, VS)
    qsl = np.array([0, 40, 72], np.int32)
    q = store(rng.standard_normal((72, H, D)), "f16")[0]
    out = torch.empty(72, H, D, dtype=torch.float16, device="cuda")
    pa.pa_prefill(out, cuda(q, "f16"), ko, vo, cuda(table), cuda(lens), cuda(qsl), scale, int(lens.max()))
    no_error()
    k16 = W.from_torch(ko, "f16")
    v16 = W.from_torch(vo, "f16")
    ref = oracle.prefill(q, k16, v16, table, lens, qsl, scale, "f16")
    assert (np.abs(as_f64(out) - ref) - half_ulp(ref, "f16")).max() <= TOL["f16"]
    x = rounded(fp4.values(*logical[0], KS), "f16")[used].reshape(len(used), Hkv, bs, D // 8, 8).transpose(0, 1, 3, 2, 4)
    assert np.array_equal(oracle.widen(k16, "f16")[used], x, equal_nan=True)
    # steps
    bm.fork(0, 2)
    for step in range(20):
        slots, copies = bm.append_tokens([0, 1, 2])
        if len(copies):
            pa.pa_copy_blocks_fp4(kt, vt, cuda(copies), D)
            for codes, f in logical:
                for s, d in copies:
                    codes[d], f[d] = codes[s], f[s]
        write(slots)
        table, lens = bm.block_tables([0, 1, 2], 8)
        q = store(rng.standard_normal((3, H, D)), "f16")[0]
        got = torch.empty(3, H, D, dtype=torch.float16, device="cuda")
        pa.pa_decode_fp4(got, cuda(q, "f16"), kt, vt, cuda(table), cuda(lens), scale, 8 * bs, KS, VS)
        if step % 5 == 0:
            no_error()
            ref = oracle.decode(q, *pools64(), table, lens, scale, "f64", q_dtype="f16")
            assert (np.abs(as_f64(got) - ref) - half_ulp(ref, "f16")).max() <= TOL["f16"]
    bm.close()


# --- the binding ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("path", ["extension", "ctypes"])
def test_both_marshalling_paths_check_and_compute_alike(path, monkeypatch):
    """The compiled marshalling and the Python one: the same results, the same refusals."""
    import paged_kv_cache_306_gb300 as pa
    from paged_kv_cache_306_gb300 import _binding as B
    if path == "extension":
        assert B._fp4_calls() is not None, "the extension was not built"
    else:
        monkeypatch.setattr(B, "_fp4_calls", lambda: None)
    rng = rng_of("paths")
    NB, Hkv, D, bs, T = 12, 2, 128, 16, 30
    key, k64 = store(rng.standard_normal((T, Hkv, D)), "bf16")
    rows = cuda(key, "bf16")
    kt = torch.zeros(NB, Hkv, fp4.tile_bytes(D, bs), dtype=torch.uint8, device="cuda")
    vt = torch.zeros_like(kt)
    slots = cuda(np.arange(T, dtype=np.int64))
    back = torch.zeros_like(rows), torch.zeros_like(rows)
    pa.pa_reshape_and_cache_fp4(rows, rows, kt, vt, slots, KS, VS)
    pa.pa_gather_cache_fp4(*back, kt, vt, slots, KS, VS)
    for got, s in zip(back, (KS, VS)):
        assert np.array_equal(as_f64(got), rounded(fp4.values(*fp4.quantise(k64, s), s), "bf16"))
    ko = torch.zeros(NB, Hkv, D // 8, bs, 8, dtype=torch.bfloat16, device="cuda")
    vo = torch.zeros(NB, Hkv, D, bs, dtype=torch.bfloat16, device="cuda")
    pairs = cuda(np.array([[0, 3], [1, 4]], np.int64))
    pa.pa_expand_blocks_fp4(ko, vo, kt, vt, pairs, KS, VS)
    assert torch.equal(vo[3].permute(2, 0, 1), back[1][:16])
    q = cuda(store(rng.standard_normal((1, 4, D)), "f16")[0], "f16")
    table, lens, out = cuda(np.array([[0, 1]], np.int32)), cuda(np.array([T], np.int32)), torch.empty_like(q)
    ws = pa.pa_decode_fp4(out, q, kt, vt, table, lens, 0.1, 32, KS, VS)
    again = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert pa.pa_decode_fp4(again, q, kt, vt, table, lens, 0.1, 32, KS, VS, ws, side) is ws
    side.synchronize()
    assert same_bytes(out, again)
    long = torch.zeros(1, 2000, dtype=torch.int32, device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    grown = pa.pa_decode_fp4(again, q, kt, vt, long, lens, 0.1, 32000, KS, VS, small)   # too small a workspace
    assert grown is not small and grown.numel() >= pa.pa_decode_fp4_workspace_size(1, 4, 2, D, 32000, 16) > 16
    no_error()

    def refused(status, f, *a):
        with pytest.raises(pa.PAError) as e:
            f(*a)
        assert e.value.status == status, str(e.value)
    bad, unsupported = B.PA_ERR_INVALID_ARG, B.PA_ERR_UNSUPPORTED
    for f in (pa.pa_reshape_and_cache_fp4, pa.pa_gather_cache_fp4):
        refused(bad, f, rows.cpu(), rows, kt, vt, slots, KS, VS)
        refused(bad, f, rows, rows.half(), kt, vt, slots, KS, VS)                     # two row types
        refused(bad, f, rows, rows[:, :, ::2], kt, vt, slots, KS, VS)                 # not contiguous
        refused(bad, f, rows, rows, kt, vt, slots[:-1].contiguous(), KS, VS)          # a slot short
        refused(bad, f, rows, rows, kt, vt, slots.int(), KS, VS)
        refused(bad, f, rows, rows, kt, vt[:-1].contiguous(), slots, KS, VS)          # pools of two sizes
        refused(bad, f, rows, rows, kt.float(), vt, slots, KS, VS)
        refused(bad, f, rows[:, :1].contiguous(), rows[:, :1].contiguous(), kt, vt, slots, KS, VS)   # heads
        refused(bad, f, rows[..., :64].contiguous(), rows[..., :64].contiguous(), kt[..., :1000].contiguous(),
                vt[..., :1000].contiguous(), slots, KS, VS)
        refused(bad, f, rows, rows, kt, vt, slots, 0.0, VS)
        refused(unsupported, f, rows.to(torch.float64), rows.to(torch.float64), kt, vt, slots, KS, VS)
    refused(bad, pa.pa_expand_blocks_fp4, ko, vo.half(), kt, vt, pairs, KS, VS)
    refused(bad, pa.pa_expand_blocks_fp4, ko, vo, kt, vt, pairs.view(-1), KS, VS)                    # no pairs
    refused(bad, pa.pa_copy_blocks_fp4, kt, vt, pairs.view(-1), D)
    refused(bad, pa.pa_expand_blocks_fp4, ko[:, :, :, :8].contiguous(), vo, kt, vt, pairs, KS, VS)
    refused(unsupported, pa.pa_expand_blocks_fp4, ko.float(), vo.float(), kt, vt, pairs, KS, VS)
    refused(bad, pa.pa_decode_fp4, out, q.bfloat16(), kt, vt, table, lens, 0.1, 32, KS, VS)
    refused(bad, pa.pa_decode_fp4, out, q, kt, vt, table, lens, 0.1, 33, KS, VS)      # longer than the table
    refused(bad, pa.pa_decode_fp4, out, q, kt, vt, table.long(), lens, 0.1, 32, KS, VS)
    refused(bad, pa.pa_decode_fp4, out, q, kt, vt, table, lens, float("nan"), 32, KS, VS)
    refused(bad, pa.pa_decode_fp4, out[:, :2].contiguous(), q, kt, vt, table, lens, 0.1, 32, KS, VS)
    refused(unsupported, pa.pa_decode_fp4, out.float(), q.float(), kt, vt, table, lens, 0.1, 32, KS, VS)
    no_error()

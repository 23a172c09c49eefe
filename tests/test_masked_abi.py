"""Refusals of the rotary and masked calls on the host, and the rotary frequencies (no GPU)."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_306_gb300 as pa
from paged_kv_cache_306_gb300 import _binding as B
from paged_kv_cache_306_gb300 import build as pa_build
from oracle import masked

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return B.load()


_BUF = {}


@pytest.fixture(scope="module", autouse=True)
def _owned_buffer():
    """Every pointer lies inside a buffer the test owns, so that a check that stopped refusing would
    launch on memory that exists (as in the other tests of the C ABI)."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        t = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        _BUF["base"], _BUF["keep"] = t.data_ptr(), t
    else:
        raw = (ctypes.c_ubyte * ((1 << 20) + 256))()
        _BUF["base"], _BUF["keep"] = (ctypes.addressof(raw) + 255) // 256 * 256, raw
    yield
    _BUF.clear()


def A(off):
    assert 0 <= off < (1 << 20)
    return ctypes.c_void_p(_BUF["base"] + off) if off else ctypes.c_void_p(0)


def decode(lib, **kw):
    a = dict(out=8192, q=8192, k=8192, v=8192, bt=8192, mb=4, sl=8192, S=1, msl=16, H=4, Hkv=4, D=128, bs=16, nb=8,
             scale=0.1, cap=0.0, slopes=0, window=0, ws=0, wsb=0, qt=B.PA_F16, ct=B.PA_F16, ks=1.0, vs=1.0)
    a.update(kw)
    return lib.pa_decode_masked(A(a["out"]), A(a["q"]), A(a["k"]), A(a["v"]), A(a["bt"]), a["mb"], A(a["sl"]), a["S"],
                                a["msl"], a["H"], a["Hkv"], a["D"], a["bs"], a["nb"], a["scale"], a["cap"],
                                A(a["slopes"]), a["window"], A(a["ws"]), a["wsb"], a["qt"], a["ct"], a["ks"], a["vs"],
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(cap=-1.0), B.PA_ERR_INVALID_ARG),
    (dict(cap=NAN), B.PA_ERR_INVALID_ARG),
    (dict(cap=INF), B.PA_ERR_INVALID_ARG),
    (dict(cap=2.0 ** -65), B.PA_ERR_INVALID_ARG),
    (dict(cap=2.0 ** 65), B.PA_ERR_INVALID_ARG),
    (dict(window=-1), B.PA_ERR_INVALID_ARG),
    (dict(slopes=8194), B.PA_ERR_ALIGNMENT),
    (dict(scale=NAN), B.PA_ERR_INVALID_ARG),
    (dict(D=96), B.PA_ERR_UNSUPPORTED),
    (dict(bs=8), B.PA_ERR_UNSUPPORTED),
    (dict(H=6), B.PA_ERR_INVALID_ARG),
    (dict(msl=65), B.PA_ERR_INVALID_ARG),
    (dict(qt=7), B.PA_ERR_INVALID_ARG),
    (dict(qt=B.PA_BF16), B.PA_ERR_INVALID_ARG),          # queries of another type than a 16-bit pool
    (dict(ks=2.0), B.PA_ERR_INVALID_ARG),
    (dict(ct=B.PA_FP8_E4M3, ks=0.0), B.PA_ERR_INVALID_ARG),
    (dict(ct=B.PA_FP8_E4M3, qt=B.PA_F32), B.PA_ERR_UNSUPPORTED),
    (dict(q=8200), B.PA_ERR_ALIGNMENT),
    (dict(q=0), B.PA_ERR_INVALID_ARG),
])
def test_decode_masked_refuses(lib, kw, status):
    assert decode(lib, **kw) == status
    assert lib.pa_last_error_message()


def test_decode_masked_with_no_sequences_is_a_no_op(lib):
    assert decode(lib, S=0, q=0, out=0) == B.PA_OK


def test_masked_workspace_is_zero_for_refused_arguments(lib):
    size = lib.pa_decode_masked_workspace_size
    assert size(2, 8, 2, 96, 70, 16, 0, B.PA_F16) == 0
    assert size(2, 8, 3, 128, 70, 16, 0, B.PA_F16) == 0
    assert size(2, 8, 2, 128, 70, 16, -1, B.PA_F16) == 0
    assert size(0, 8, 2, 128, 70, 16, 0, B.PA_F16) == 0
    with pytest.raises(pa.PAError):
        pa.pa_decode_masked_workspace_size(2, 8, 2, 128, 1 << 31, 16, 0, B.PA_F16)
    with pytest.raises(pa.PAError):
        pa.pa_decode_masked_workspace_size(2, 8, 2, 128, 70, 16, 1 << 32, B.PA_F16)


def prefill(lib, **kw):
    a = dict(out=8192, q=8192, k=8192, v=8192, bt=8192, mb=4, sl=8192, qsl=8192, pre=0, S=1, T=4, msl=16, H=4, Hkv=4,
             D=128, bs=16, nb=8, scale=0.1, cap=0.0, slopes=0, window=0, dt=B.PA_F16)
    a.update(kw)
    return lib.pa_prefill_masked(A(a["out"]), A(a["q"]), A(a["k"]), A(a["v"]), A(a["bt"]), a["mb"], A(a["sl"]),
                                 A(a["qsl"]), A(a["pre"]), a["S"], a["T"], a["msl"], a["H"], a["Hkv"], a["D"], a["bs"],
                                 a["nb"], a["scale"], a["cap"], A(a["slopes"]), a["window"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(cap=-1.0), B.PA_ERR_INVALID_ARG),
    (dict(cap=NAN), B.PA_ERR_INVALID_ARG),
    (dict(window=-5), B.PA_ERR_INVALID_ARG),
    (dict(slopes=8193), B.PA_ERR_ALIGNMENT),
    (dict(pre=8193), B.PA_ERR_ALIGNMENT),
    (dict(scale=0.0), B.PA_ERR_INVALID_ARG),
    (dict(scale=-0.1), B.PA_ERR_INVALID_ARG),
    (dict(scale=NAN), B.PA_ERR_INVALID_ARG),
    (dict(scale=INF), B.PA_ERR_INVALID_ARG),
    (dict(dt=B.PA_F32), B.PA_ERR_UNSUPPORTED),
    (dict(dt=B.PA_FP8_E4M3), B.PA_ERR_UNSUPPORTED),
    (dict(D=96), B.PA_ERR_UNSUPPORTED),
    (dict(T=-1), B.PA_ERR_INVALID_ARG),
    (dict(nb=1 << 25), B.PA_ERR_UNSUPPORTED),
    (dict(qsl=0), B.PA_ERR_INVALID_ARG),
    (dict(out=8200), B.PA_ERR_ALIGNMENT),
])
def test_prefill_masked_refuses(lib, kw, status):
    assert prefill(lib, **kw) == status


def test_prefill_masked_with_no_tokens_is_a_no_op(lib):
    assert prefill(lib, T=0, q=0, out=0) == B.PA_OK


def rope(lib, **kw):
    a = dict(qo=4096, ko=8192, q=12288, k=16384, sq=512, sk=128, pos=8192, f=8192, T=2, H=4, Hkv=1, D=128, r=128,
             layout=0, amp=1.0, dt=B.PA_F16)
    a.update(kw)
    return lib.pa_rope(A(a["qo"]), A(a["ko"]), A(a["q"]), A(a["k"]), a["sq"], a["sk"], A(a["pos"]), A(a["f"]), a["T"],
                       a["H"], a["Hkv"], a["D"], a["r"], a["layout"], a["amp"], a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), B.PA_ERR_UNSUPPORTED),
    (dict(r=0), B.PA_ERR_INVALID_ARG),
    (dict(r=15), B.PA_ERR_INVALID_ARG),
    (dict(r=144), B.PA_ERR_INVALID_ARG),
    (dict(r=24), B.PA_ERR_UNSUPPORTED),
    (dict(layout=2), B.PA_ERR_INVALID_ARG),
    (dict(amp=NAN), B.PA_ERR_INVALID_ARG),
    (dict(amp=INF), B.PA_ERR_INVALID_ARG),
    (dict(dt=B.PA_FP8_E4M3), B.PA_ERR_UNSUPPORTED),
    (dict(dt=9), B.PA_ERR_UNSUPPORTED),
    (dict(T=-1), B.PA_ERR_INVALID_ARG),
    (dict(T=1 << 31), B.PA_ERR_INVALID_ARG),
    (dict(H=0), B.PA_ERR_INVALID_ARG),
    (dict(Hkv=70000), B.PA_ERR_UNSUPPORTED),
    (dict(sq=504), B.PA_ERR_INVALID_ARG),
    (dict(sq=516), B.PA_ERR_ALIGNMENT),
    (dict(sk=0), B.PA_ERR_INVALID_ARG),
    (dict(sk=(1 << 31) + 8), B.PA_ERR_UNSUPPORTED),
    (dict(q=0), B.PA_ERR_INVALID_ARG),
    (dict(ko=0), B.PA_ERR_INVALID_ARG),
    (dict(pos=0), B.PA_ERR_INVALID_ARG),
    (dict(f=0), B.PA_ERR_INVALID_ARG),
    (dict(q=12296), B.PA_ERR_ALIGNMENT),
    (dict(f=8196), B.PA_ERR_ALIGNMENT),
])
def test_rope_refuses(lib, kw, status):
    assert rope(lib, **kw) == status


def test_rope_with_no_tokens_is_a_no_op(lib):
    assert rope(lib, T=0, q=0, qo=0) == B.PA_OK


def rope_and_cache(lib, **kw):
    a = dict(qo=4096, q=12288, k=16384, v=16384, sq=512, sk=128, sv=128, kc=32768, vc=65536, pos=8192, slots=8192,
             f=8192, T=2, H=4, Hkv=1, D=128, r=128, bs=16, nb=2, layout=0, amp=1.0, dt=B.PA_F16, ct=B.PA_F16, ks=1.0,
             vs=1.0)
    a.update(kw)
    return lib.pa_rope_and_cache(A(a["qo"]), A(a["q"]), A(a["k"]), A(a["v"]), a["sq"], a["sk"], a["sv"], A(a["kc"]),
                                 A(a["vc"]), A(a["pos"]), A(a["slots"]), A(a["f"]), a["T"], a["H"], a["Hkv"], a["D"],
                                 a["r"], a["bs"], a["nb"], a["layout"], a["amp"], a["dt"], a["ct"], a["ks"], a["vs"],
                                 None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=32), B.PA_ERR_UNSUPPORTED),
    (dict(r=40), B.PA_ERR_UNSUPPORTED),
    (dict(bs=0), B.PA_ERR_INVALID_ARG),
    (dict(nb=0), B.PA_ERR_INVALID_ARG),
    (dict(ct=B.PA_BF16), B.PA_ERR_INVALID_ARG),
    (dict(ks=0.5), B.PA_ERR_INVALID_ARG),
    (dict(ct=B.PA_FP8_E4M3, vs=0.0), B.PA_ERR_INVALID_ARG),
    (dict(ct=B.PA_FP8_E4M3, ks=INF), B.PA_ERR_INVALID_ARG),
    (dict(dt=B.PA_FP8_E4M3, ct=B.PA_FP8_E4M3), B.PA_ERR_UNSUPPORTED),
    (dict(sv=120), B.PA_ERR_INVALID_ARG),
    (dict(sv=132), B.PA_ERR_ALIGNMENT),
    (dict(slots=0), B.PA_ERR_INVALID_ARG),
    (dict(vc=0), B.PA_ERR_INVALID_ARG),
    (dict(slots=8196), B.PA_ERR_ALIGNMENT),
    (dict(kc=32776), B.PA_ERR_ALIGNMENT),
])
def test_rope_and_cache_refuses(lib, kw, status):
    assert rope_and_cache(lib, **kw) == status


@pytest.mark.parametrize("kw", [                # rows: q 2 x 1024 bytes, k 2 x 256
    dict(qo=12288, sq=640),                      # in place, but not the same rows
    dict(qo=12288 + 1024), dict(qo=12288 - 16), dict(qo=12288 + 2032),
    dict(qo=12288 + 2048 + 240, sq=640),         # q's second row ends 256 bytes later
    dict(ko=12288), dict(ko=16384 + 256), dict(ko=16384, sk=136), dict(ko=4096 + 2032), dict(ko=4096 - 496),
    dict(qo=16384 - 2032), dict(qo=16384 + 496),
])
def test_rope_refuses_outputs_over_other_rows(lib, kw):
    assert rope(lib, **kw) == B.PA_ERR_INVALID_ARG
    assert b"overlap" in lib.pa_last_error_message()


@pytest.mark.parametrize("kw", [dict(qo=12288, sq=640), dict(qo=16384 + 240), dict(qo=24576 - 2032, v=24576)])
def test_rope_and_cache_refuses_outputs_over_other_rows(lib, kw):
    assert rope_and_cache(lib, **kw) == B.PA_ERR_INVALID_ARG
    assert b"overlap" in lib.pa_last_error_message()


def test_rope_and_cache_with_no_tokens_is_a_no_op(lib):
    assert rope_and_cache(lib, T=0, q=0, kc=0) == B.PA_OK


@pytest.mark.parametrize("kw", [
    dict(), dict(rotary_dim=64, base=500000.0), dict(scaling="linear", factor=4.0),
    dict(scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0, base=500000.0),
    dict(scaling="yarn", factor=4.0, original_len=4096), dict(scaling="yarn", factor=1.0, original_len=1),
    dict(scaling="yarn", factor=40.0, original_len=4096, rotary_dim=64, low=1.0, high=1.0001),
])
def test_frequencies(lib, kw):
    kw = dict(dict(rotary_dim=128, base=10000.0), **kw)
    f, amp = pa.pa_rope_frequencies(**kw)
    ref, ref_amp = masked.frequencies(**kw)
    assert np.allclose(f.numpy(), ref, rtol=1e-14, atol=0)
    assert amp == pytest.approx(ref_amp, rel=1e-7)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=-4), dict(base=1.0), dict(base=NAN), dict(scaling="other"),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=NAN), dict(scaling="bands", factor=2.0),
    dict(scaling="yarn", factor=2.0, original_len=4096, low=4.0, high=4.0),
    dict(scaling="bands", factor=2.0, original_len=4096, low=0.0), dict(rotary_dim=1 << 32),
])
def test_frequencies_refused(lib, kw):
    with pytest.raises(pa.PAError):
        pa.pa_rope_frequencies(**dict(dict(rotary_dim=128, base=10000.0), **kw))


def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(1, 4, 128, dtype=torch.float16), torch.zeros(1, 2, 128, dtype=torch.float16)
    kc, vc = torch.zeros(1, 2, 16, 16, 8, dtype=torch.float16), torch.zeros(1, 2, 128, 16, dtype=torch.float16)
    i32, i64 = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    f = torch.zeros(64, dtype=torch.float64)
    with pytest.raises(pa.PAError):
        pa.pa_decode_masked(q, q, kc, vc, i32, i32[0], 0.1, 16)
    with pytest.raises(pa.PAError):
        pa.pa_prefill_masked(q, q, kc, vc, i32, i32[0], i32[0], 0.1, 16)
    with pytest.raises(pa.PAError):
        pa.pa_rope(q, k, q, k, i64, f)
    with pytest.raises(pa.PAError):
        pa.pa_rope_and_cache(q, q, k, k, kc, vc, i64, i64, f)

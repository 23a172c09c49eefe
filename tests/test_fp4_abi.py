"""Host-side refusals of the FP4 calls (no GPU: each call returns before any launch)."""
import ctypes

import pytest

import paged_kv_cache_306_gb300 as pa
from paged_kv_cache_306_gb300 import _binding as B
from paged_kv_cache_306_gb300 import build as pa_build

_BUF = {}


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return B.load()


@pytest.fixture(scope="module", autouse=True)
def _owned_buffer():
    """Every pointer lies in a buffer of the test: a check that failed to refuse would launch on memory that exists."""
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
    return ctypes.c_void_p(_BUF["base"] + off) if off else ctypes.c_void_p(0)


def test_tile_bytes(lib):
    assert lib.pa_fp4_tile_bytes(128, 16) == 1152 and lib.pa_fp4_tile_bytes(64, 32) == 1152
    assert lib.pa_fp4_tile_bytes(64, 16) == 576 and lib.pa_fp4_tile_bytes(128, 32) == 2304
    for d, bs in ((96, 16), (128, 8), (0, 0), (-64, 16), (256, 16)):
        assert lib.pa_fp4_tile_bytes(d, bs) == 0


ROWS = [
    (dict(D=96), B.PA_ERR_UNSUPPORTED), (dict(bs=8), B.PA_ERR_UNSUPPORTED), (dict(Hkv=65536), B.PA_ERR_UNSUPPORTED),
    (dict(Hkv=0), B.PA_ERR_INVALID_ARG), (dict(nb=0), B.PA_ERR_INVALID_ARG), (dict(T=-1), B.PA_ERR_INVALID_ARG),
    (dict(T=1 << 31), B.PA_ERR_INVALID_ARG), (dict(T=(1 << 31) - 1, Hkv=4096), B.PA_ERR_UNSUPPORTED),
    (dict(dt=B.PA_FP8_E4M3), B.PA_ERR_UNSUPPORTED), (dict(dt=9), B.PA_ERR_UNSUPPORTED),
    (dict(ks=0.0), B.PA_ERR_INVALID_ARG), (dict(vs=-1.0), B.PA_ERR_INVALID_ARG),
    (dict(ks=float("nan")), B.PA_ERR_INVALID_ARG), (dict(vs=float("inf")), B.PA_ERR_INVALID_ARG),
    (dict(ks=2.0 ** -65), B.PA_ERR_INVALID_ARG), (dict(ks=2.0 ** 65), B.PA_ERR_INVALID_ARG),
    (dict(key=24), B.PA_ERR_ALIGNMENT), (dict(k=8), B.PA_ERR_ALIGNMENT), (dict(slots=20), B.PA_ERR_ALIGNMENT),
    (dict(key=0), B.PA_ERR_INVALID_ARG), (dict(slots=0), B.PA_ERR_INVALID_ARG), (dict(T=0, key=0), B.PA_OK),
]


@pytest.mark.parametrize("call", ["pa_reshape_and_cache_fp4", "pa_gather_cache_fp4"])
@pytest.mark.parametrize("kw,status", ROWS)
def test_row_calls_reject_bad_arguments(lib, call, kw, status):
    a = dict(key=16, value=16, k=16, v=16, slots=16, T=2, Hkv=2, D=64, bs=16, nb=8, dt=B.PA_F16, ks=0.5, vs=0.5)
    a.update(kw)
    st = getattr(lib, call)(A(a["key"]), A(a["value"]), A(a["k"]), A(a["v"]), A(a["slots"]), a["T"], a["Hkv"], a["D"],
                            a["bs"], a["nb"], a["dt"], a["ks"], a["vs"], None)
    assert st == status


@pytest.mark.parametrize("kw,status", [
    (dict(D=72), B.PA_ERR_UNSUPPORTED), (dict(bs=64), B.PA_ERR_UNSUPPORTED), (dict(dt=B.PA_F32), B.PA_ERR_UNSUPPORTED),
    (dict(n=-1), B.PA_ERR_INVALID_ARG), (dict(nbo=0), B.PA_ERR_INVALID_ARG), (dict(nb=0), B.PA_ERR_INVALID_ARG),
    (dict(ks=0.0), B.PA_ERR_INVALID_ARG), (dict(ko=8), B.PA_ERR_ALIGNMENT), (dict(sd=20), B.PA_ERR_ALIGNMENT),
    (dict(ko=0), B.PA_ERR_INVALID_ARG), (dict(n=0, ko=0), B.PA_OK),
])
def test_expand_rejects_bad_arguments(lib, kw, status):
    a = dict(ko=16, vo=16, k=16, v=16, sd=16, n=2, Hkv=2, D=64, bs=16, nbo=8, nb=8, dt=B.PA_F16, ks=0.5, vs=0.5)
    a.update(kw)
    assert lib.pa_expand_blocks_fp4(A(a["ko"]), A(a["vo"]), A(a["k"]), A(a["v"]), A(a["sd"]), a["n"], a["Hkv"], a["D"],
                                    a["bs"], a["nbo"], a["nb"], a["dt"], a["ks"], a["vs"], None) == status


def test_copy_blocks_rejects_bad_arguments(lib):
    def c(k=16, sd=16, n=2, D=64, bs=16, nb=8):
        return lib.pa_copy_blocks_fp4(A(k), A(16), A(sd), n, 2, D, bs, nb, None)
    assert c(D=80) == B.PA_ERR_UNSUPPORTED and c(bs=4) == B.PA_ERR_UNSUPPORTED
    assert c(k=24) == B.PA_ERR_ALIGNMENT and c(sd=12) == B.PA_ERR_ALIGNMENT
    assert c(n=-1) == B.PA_ERR_INVALID_ARG and c(k=0) == B.PA_ERR_INVALID_ARG and c(nb=0) == B.PA_ERR_INVALID_ARG
    assert c(n=0, k=0) == B.PA_OK


@pytest.mark.parametrize("kw,status", [
    (dict(H=6, Hkv=4), B.PA_ERR_INVALID_ARG), (dict(D=96), B.PA_ERR_UNSUPPORTED), (dict(bs=8), B.PA_ERR_UNSUPPORTED),
    (dict(msl=65), B.PA_ERR_INVALID_ARG), (dict(msl=0), B.PA_ERR_INVALID_ARG), (dict(dt=B.PA_F32), B.PA_ERR_UNSUPPORTED),
    (dict(dt=B.PA_FP8_E4M3), B.PA_ERR_UNSUPPORTED), (dict(nb=0), B.PA_ERR_INVALID_ARG),
    (dict(S=-1), B.PA_ERR_INVALID_ARG), (dict(S=65536), B.PA_ERR_INVALID_ARG), (dict(mb=0), B.PA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), B.PA_ERR_INVALID_ARG), (dict(scale=3e38, ks=2.0 ** 60), B.PA_ERR_INVALID_ARG),
    (dict(ks=0.0), B.PA_ERR_INVALID_ARG), (dict(vs=float("inf")), B.PA_ERR_INVALID_ARG),
    (dict(q=8200), B.PA_ERR_ALIGNMENT), (dict(bt=8194), B.PA_ERR_ALIGNMENT), (dict(q=0), B.PA_ERR_INVALID_ARG),
    (dict(S=0, q=0, out=0), B.PA_OK),
])
def test_decode_rejects_bad_arguments(lib, kw, status):
    a = dict(out=8192, q=8192, k=8192, v=8192, bt=8192, mb=4, sl=8192, S=1, msl=16, H=4, Hkv=2, D=128, bs=16, nb=8,
             scale=0.1, ws=0, wsb=0, dt=B.PA_F16, ks=0.5, vs=0.25)
    a.update(kw)
    st = lib.pa_decode_fp4(A(a["out"]), A(a["q"]), A(a["k"]), A(a["v"]), A(a["bt"]), a["mb"], A(a["sl"]), a["S"],
                           a["msl"], a["H"], a["Hkv"], a["D"], a["bs"], a["nb"], a["scale"], A(a["ws"]), a["wsb"],
                           a["dt"], a["ks"], a["vs"], None)
    assert st == status


def test_workspace_size_is_zero_for_arguments_decode_rejects(lib):
    assert lib.pa_decode_fp4_workspace_size(2, 8, 2, 96, 70, 16) == 0
    assert lib.pa_decode_fp4_workspace_size(2, 8, 3, 128, 70, 16) == 0
    assert lib.pa_decode_fp4_workspace_size(0, 8, 2, 128, 70, 16) == 0


def test_binding_refuses_cpu_tensors_and_shapes_that_disagree(lib):
    torch = pytest.importorskip("torch")
    pool = torch.zeros(4, 2, 1152, dtype=torch.uint8)
    rows = torch.zeros(3, 2, 128, dtype=torch.float16)
    slots = torch.zeros(3, dtype=torch.int64)
    for call in (pa.pa_reshape_and_cache_fp4, pa.pa_gather_cache_fp4):
        with pytest.raises(pa.PAError):
            call(rows, rows, pool, pool, slots, 0.5, 0.5)
    with pytest.raises(pa.PAError):
        pa.pa_decode_fp4(rows, rows, pool, pool, torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32),
                         0.1, 16, 0.5, 0.5)
    with pytest.raises(pa.PAError):
        pa.pa_copy_blocks_fp4(pool, pool, torch.zeros(1, 2, dtype=torch.int64), 128)
    with pytest.raises(pa.PAError):
        pa.pa_expand_blocks_fp4(torch.zeros(4, 2, 16, 16, 8, dtype=torch.float16),
                                torch.zeros(4, 2, 128, 16, dtype=torch.float16), pool, pool,
                                torch.zeros(1, 2, dtype=torch.int64), 0.5, 0.5)

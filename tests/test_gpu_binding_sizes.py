"""Sizes past 32 bits, which C's int cannot hold: refused, not cut to their lower bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(params=["extension", "ctypes"])
def pa(request, monkeypatch):
    import paged_kv_cache_306_gb300 as m
    from paged_kv_cache_306_gb300 import _binding as B
    if request.param == "extension":
        assert B._fp4_calls() is not None, "the extension was not built"
    else:
        monkeypatch.setattr(B, "_fp4_calls", lambda: None)
    return m


def empty(*shape, dtype=torch.float16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def test_rope(pa):
    pos, f = torch.zeros(1, dtype=torch.int64, device="cuda"), empty(32, dtype=torch.float64)
    q, k = empty(1, 2, 64), empty(1, 1, 64)
    many = empty(2 ** 31 + 32, dtype=torch.float64)              # 2^32 + 64 rotary dims
    kc, vc = empty(1, 1, 8, 16, 8), empty(1, 1, 64, 16)
    with pytest.raises(pa.PAError, match="32 bits"):
        pa.pa_rope(torch.empty_like(q), torch.empty_like(k), q, k, pos, many)
    with pytest.raises(pa.PAError, match="32 bits"):
        pa.pa_rope_and_cache(torch.empty_like(q), q, k, k, kc, vc, pos, pos, many)
    del many
    wide = empty(1, 1, 2 ** 32 + 64)
    with pytest.raises(pa.PAError, match="32 bits"):
        pa.pa_rope(torch.empty_like(wide), torch.empty_like(wide), wide, wide, pos, f)
    assert pa.pa_get_device_error() in pa.DEVICE_ERRORS


def test_tables(pa):
    kc, vc = empty(1, 1, 8, 16, 8), empty(1, 1, 64, 16)
    q, lens = empty(1, 1, 64), torch.ones(1, dtype=torch.int32, device="cuda")
    table = empty(1, 2 ** 32 + 4, dtype=torch.int32)
    with pytest.raises(pa.PAError, match="32 bits"):
        pa.pa_decode_masked(torch.empty_like(q), q, kc, vc, table, lens, 0.1, 16)
    with pytest.raises(pa.PAError, match="32 bits"):
        pa.pa_prefill_masked(torch.empty_like(q), q, kc, vc, table, lens, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                             0.1, 16)

"""pa_decode_fp4's schedule at the ends of its arguments' ranges."""
import math

import numpy as np
import pytest

from helpers import as_f64
from oracle import fp4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_306_gb300 as pa
    pa.load()


@pytest.mark.parametrize("bound", [INT_MAX, INT_MAX - 30, INT_MAX - 31, INT_MAX - 32])
def test_the_longest_length_bounds_use_the_whole_gpu(bound):
    import paged_kv_cache_306_gb300 as pa
    assert pa.pa_decode_fp4_workspace_size(1, 2, 1, 64, bound, 32) == \
        pa.pa_decode_fp4_workspace_size(1, 2, 1, 64, 1 << 30, 32) > 0


@pytest.mark.parametrize("L,bound", [(100, INT_MAX), (9001, INT_MAX - 1), (INT_MAX, INT_MAX), (INT_MAX - 31, INT_MAX)])
def test_a_sequence_under_the_longest_bound(L, bound):
    """Tables as wide as the longest sequence, every entry the same block of 32 tokens: token t is the block's token
    t mod 32, with the weight 2^-(t mod 4) (fp4_checks has the construction) and a V row of its own, 6 in the dims
    2 (t mod 32) and 2 (t mod 32) + 1.  A token of the block counts L // 32 or one more times.  Up to 2^-4 for the
    long sums: of 2^26 chunks a warp of 152 x 12 adds 36793, two additions each, off by 2^-22 at most: 2^-5.8."""
    import paged_kv_cache_306_gb300 as pa
    D, bs, ks, vs = 64, 32, 0.0173, 0.0214
    t = np.arange(bs)
    k, v = np.zeros((2, 1, 1, bs, D), np.uint8)
    k[0, 0, t, 0] = np.array([0, 10, 12, 13], np.uint8)[t % 4]        # 0, -1, -2, -3
    v[0, 0, t, 2 * t] = v[0, 0, t, 2 * t + 1] = 7                     # 6
    one = np.full((1, 1, bs, D // 16), 0x38, np.uint8)
    tiles = [torch.from_numpy(fp4.pack(x, one, of)).cuda() for x, of in ((k, "k"), (v, "v"))]
    q = torch.zeros(1, 2, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 1
    table = torch.zeros(1, -(-bound // bs), dtype=torch.int32, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, math.nan)
    pa.pa_decode_fp4(out, q, *tiles, table, lens, 1 / (ks * math.log2(math.e)), bound, ks, vs)
    assert pa.pa_get_device_error() == 0
    c = (L // bs + (t < L % bs)) * 2.0 ** -(t % 4)
    want = np.repeat(6 * vs * c / c.sum(), 2)
    got = as_f64(out)
    assert np.isfinite(got).all()
    # one more rounding: fp16, half a step of 2^-11
    assert (np.abs(got - want) <= want * (2.0 ** -11 + (2.0 ** -4 if L > 1 << 20 else 2.0 ** -18))).all()


def test_the_grid_counts_the_warps_of_the_kernel_that_runs():
    """Head size 64 has 12 warps a CTA whatever the group: one long segment of 1200 chunks is 100 CTAs, for 8 query
    heads a kv head and for 16 (head size 128: 8 warps with 9 and more heads)."""
    import paged_kv_cache_306_gb300 as pa
    size = pa.pa_decode_fp4_workspace_size
    assert size(1, 16, 1, 64, 38400, 16) == size(1, 8, 1, 64, 38400, 16)
    assert size(1, 16, 1, 128, 25600, 16) == size(1, 8, 1, 128, 38400, 16)


@pytest.mark.parametrize("path", ["extension", "ctypes"])
@pytest.mark.parametrize("bound", [(1 << 32) + 40, 1 << 31, -(1 << 31) - 1, (1 << 32) + 40000])
def test_a_length_bound_past_32_bits_is_refused(path, bound, monkeypatch):
    """2^32 + 40 is not 40."""
    import paged_kv_cache_306_gb300 as pa
    from paged_kv_cache_306_gb300 import _binding as B
    if path == "ctypes":
        monkeypatch.setattr(B, "_fp4_calls", lambda: None)
    q = torch.zeros(1, 2, 64, dtype=torch.float16, device="cuda")
    pool = torch.zeros(4, 1, pa.pa_fp4_tile_bytes(64, 16), dtype=torch.uint8, device="cuda")
    table, lens = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(pa.PAError) as e:
        pa.pa_decode_fp4(torch.empty_like(q), q, pool, pool, table, lens, 0.1, bound, 0.5, 0.5)
    assert e.value.status == B.PA_ERR_INVALID_ARG
    with pytest.raises(pa.PAError):
        pa.pa_decode_fp4_workspace_size(1, 2, 1, 64, bound, 16)
    assert pa.pa_get_device_error() == 0

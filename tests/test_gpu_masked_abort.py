"""A masked decode of few blocks, one of whose warps gave up waiting: the pieces that the others left make no row."""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, f64, queries
from masked_rows import check_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

TIMEOUT = 4             # PA_DEVERR_TIMEOUT
LIMIT_NS = 2_000_001    # odd: the wait of the warp with the first block alone runs out (as elsewhere, it neither faults nor hangs)


@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "fp8"), ("f32", "f32")], ids="/".join)
@pytest.mark.parametrize("lens", [[100], [40, 60], [250]], ids=str)
def test_rows_with_a_missing_piece_are_left_alone(types, lens):
    import paged_kv_cache_306_gb300 as pa
    pools = Pools(lens, 1, 64, 16, types[1], 1)
    kc, vc, bt = pools.on("cuda")
    q = queries(len(lens), 4 if types[1] != "f32" else 1, 64, types[0], 2)
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert pa.pa_get_device_error() in pa.DEVICE_ERRORS     # (and cleared)
    n0 = pa.pa_launch_count()

    def call():
        out = torch.full_like(q, 99.0).cuda()
        pa.pa_decode_masked(out, q.cuda(), kc, vc, bt, sl, 0.125, max(lens), 9.0)
        return out
    try:
        pa.pa_set_test_wait_limit(LIMIT_NS)
        out = call()
    finally:
        pa.pa_set_test_wait_limit(0)
    assert pa.pa_launch_count() == n0 + 1                   # (a launch of one CTA, which merges by itself)
    assert pa.pa_get_device_error() == TIMEOUT
    ref = masked.decode(f64(q), *pools.exact(), pools.table, lens, 0.125, 16, softcap=9.0)
    left = (out.float() == 99.0).all(-1).cpu().numpy()      # [sequence, head]
    assert left[0].all(), "the first sequence lacks its first piece"
    for s in np.flatnonzero(~left.all(1)):                  # a row that was written is right
        check_rows(out[s:s + 1], ref[s:s + 1], q[s:s + 1], pools, 0.125, 9.0, 0.0, types[0])
    out = call()
    assert pa.pa_get_device_error() == 0
    check_rows(out, ref, q, pools, 0.125, 9.0, 0.0, types[0])

"""Decode over FP4 pools where the merge of pieces decides: marked sequences, and random rows within the
sharp bound (fp4_checks; what both can tell apart is tested in test_fp4_checks.py)."""
import math

import numpy as np
import pytest

from fp4_checks import LONG, RANDOM, Markers, sharp_bound_of
from helpers import as_f64, half_ulp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_306_gb300 as pa
    pa.load()


def run(m, max_len=None, workspace=None):
    import paged_kv_cache_306_gb300 as pa
    import workloads as W
    q = W.to_torch(m.q, m.q_dtype, "cuda")
    k, v, table = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (m.k, m.v, m.table))
    out = torch.full_like(q, math.nan)
    pa.pa_decode_fp4(out, q, k, v, table, torch.tensor(m.lens, dtype=torch.int32, device="cuda"), m.scale,
                     max_len or m.max_len, m.k_scale, m.v_scale, workspace)
    return out


def check(m, out):
    import paged_kv_cache_306_gb300 as pa
    assert pa.pa_get_device_error() == 0
    got = as_f64(out)
    assert np.isfinite(got).all()
    for i, L in enumerate(m.lens):
        assert m.excess(i, got[i]) <= 0, f"sequence {i} of {L} tokens"


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("case", LONG, ids=["-".join(map(str, c[0])) for c in LONG])
def test_every_token_counts_once(case, seed):
    m = Markers(*case, seed=seed)
    check(m, run(m))


@pytest.mark.parametrize("longest", [100, 900, 4000])
@pytest.mark.parametrize("S,G,Hkv,D,bs", [(3, 4, 2, 128, 16), (40, 9, 2, 64, 32), (150, 1, 3, 64, 16)])
def test_every_token_of_a_batch_counts_once(S, G, Hkv, D, bs, longest):
    lens = [int(x) for x in np.random.default_rng([S, longest]).integers(1, longest + 1, S)]
    m = Markers(lens, G, Hkv, D, bs, "f16")
    check(m, run(m))


@pytest.mark.parametrize("q_dtype,D,bs,G,Hkv,lens", RANDOM)
def test_random_rows_within_the_sharp_bound(q_dtype, D, bs, G, Hkv, lens):
    from test_gpu_fp4 import KS, VS, Case, no_error
    c = Case(lens, G, Hkv, D, bs, q_dtype)
    out = c.run()
    no_error()
    ref, bound = sharp_bound_of(c, KS, VS)
    got = as_f64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) - bound - half_ulp(np.abs(ref) + bound, q_dtype)).max() <= 0


@pytest.mark.parametrize("case", [LONG[5], LONG[6]], ids=["40000", "ragged"])
def test_every_token_counts_once_after_a_wait_that_ran_out(case):
    import paged_kv_cache_306_gb300 as pa
    m = Markers(*case)
    need = pa.pa_decode_fp4_workspace_size(len(m.lens), m.G * m.Hkv, m.Hkv, m.D, m.max_len, m.bs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    try:
        pa.pa_set_test_wait_limit(2_000_000)
        run(m, workspace=ws)
    finally:
        pa.pa_set_test_wait_limit(0)
    assert pa.pa_get_device_error() == 4
    check(m, run(m, workspace=ws))

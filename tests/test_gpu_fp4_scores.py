"""Decode over FP4 pools at the end of the range of the softmax's scale: scores times the scale are past
fp32's largest number, their differences decide all the same, whole in one warp or cut into pieces."""
import numpy as np
import pytest

import oracle
from helpers import as_f64, half_ulp
from oracle import fp4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_306_gb300 as pa
    pa.load()


@pytest.mark.parametrize("q_dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,D,G", [([1, 65, 3000, 20000], 128, 2), ([9000, 40], 64, 11)])
@pytest.mark.parametrize("scale", [2.0 ** 100, -2.0 ** 118, 2.0 ** 121, 2.0 ** 122])
def test_the_largest_scale_leaves_the_largest_score(q_dtype, lens, D, G, scale):
    """q of -1, 0 and 1 and group scales of 1: every score is a sum of at most 128 codes, exact in fp32, and two
    that differ do so by 1/2 at least, 2^99 and more after the scale.  So the answer is the mean of the V rows
    whose score is the largest (the smallest for a negative scale)."""
    from test_gpu_fp4 import KS, VS, Case, no_error, rng_of, store
    c = Case(lens, G, 2, D, 16, q_dtype, scale)
    (kc, kf), _ = c.pools
    kf[...] = 0x38
    c.q = store(rng_of("largest", scale).integers(-1, 2, size=c.q.shape).astype(np.float64), q_dtype)[0]
    c.k = fp4.pack(kc, kf, "k")
    c.scale = scale / KS
    assert np.isfinite(np.float32(c.scale)) and np.isfinite(np.float32(scale * 1.4427))
    out = c.run()
    no_error()
    k64, v64 = fp4.f64_pools(c.k, c.v, D, 16, KS, VS)
    args = (c.table, np.array(c.lens, np.int32), c.scale, "f64")
    ref, mass = (oracle.decode(c.q, k64, v, *args, q_dtype=q_dtype) for v in (v64, np.abs(np.nan_to_num(v64))))
    bound = (np.array(c.lens)[:, None, None] / 8 + 64) * 2.0 ** -22 * mass     # sums in fp32
    got = as_f64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) - bound - half_ulp(np.abs(ref) + bound, q_dtype)).max() <= 0

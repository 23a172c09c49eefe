"""Where pa_decode_fp4 keeps what its CTAs tell one another, and its refusals of workspaces."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_306_gb300 as pa
    pa.load()


@pytest.mark.parametrize("lens,G,Hkv,D", [([9000, 5000], 4, 2, 128), ([30000], 1, 1, 64), ([700, 2500, 3], 16, 1, 64)])
@pytest.mark.parametrize("more", [0, 64, 1 << 20])
def test_the_tags_are_the_workspaces_first_bytes(lens, G, Hkv, D, more):
    """The first num_SMs * 8 bytes hold nothing but tags, in a workspace of any size and for every shape: each is
    as it was or, where a piece was passed on, cleared."""
    import paged_kv_cache_306_gb300 as pa
    from test_gpu_fp4 import Case, no_error
    c = Case(lens, G, Hkv, D, 16, "f16")
    need = pa.pa_decode_fp4_workspace_size(len(lens), G * Hkv, Hkv, D, c.max_len, 16)
    assert need > 0
    ws = torch.full((need + more,), 0xA5, dtype=torch.uint8, device="cuda")
    out = c.run(workspace=ws)
    no_error()
    c.check(out)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert need >= 8 * sms
    tags = ws[:8 * sms].view(-1, 8)
    kept, cleared = (tags == 0xA5).all(1), (tags == 0).all(1)
    assert bool((kept | cleared).all()) and bool(cleared.any())

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


@pytest.mark.parametrize("S,H,Hkv,D,L", [(2, 8, 2, 128, 1000), (1, 16, 1, 64, 30000), (300, 4, 4, 64, 200)])
def test_a_workspace_a_byte_short_or_askew_is_refused(S, H, Hkv, D, L):
    import paged_kv_cache_306_gb300 as pa
    B = pa._binding
    lib = pa.load()
    need = pa.pa_decode_fp4_workspace_size(S, H, Hkv, D, L, 16)
    assert need > 0                                     # these shapes take more than one CTA
    ws = torch.full((need + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    q = torch.zeros(S, H, D, dtype=torch.float16, device="cuda")
    out = torch.full_like(q, 7)
    pool = torch.zeros(4, Hkv, pa.pa_fp4_tile_bytes(D, 16), dtype=torch.uint8, device="cuda")
    table = torch.zeros(S, -(-L // 16), dtype=torch.int32, device="cuda")
    lens = torch.full((S,), L, dtype=torch.int32, device="cuda")

    def call(ptr, size):
        return lib.pa_decode_fp4(out.data_ptr(), q.data_ptr(), pool.data_ptr(), pool.data_ptr(), table.data_ptr(),
                                 table.shape[1], lens.data_ptr(), S, L, H, Hkv, D, 16, 4, 0.1, ptr, size, B.PA_F16, 0.5,
                                 0.5, None)
    assert call(ws.data_ptr(), need - 1) == B.PA_ERR_WORKSPACE
    assert call(0, need) == B.PA_ERR_WORKSPACE
    assert call(ws.data_ptr() + 8, need) == B.PA_ERR_ALIGNMENT
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((ws == 0xA5).all())          # nothing ran
    assert call(ws.data_ptr(), need) == B.PA_OK
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0 and bool((out == 0).all())

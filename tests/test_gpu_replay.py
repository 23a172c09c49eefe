"""Captured decode calls replayed over other lengths on one workspace.

A captured call keeps its arguments, the launch's own number among them, while its lengths and tables
change between replays, and the workspace holds what the last replay left.  Every replay has to give the
bits that an eager call with a fresh workspace gives for the same inputs.  The bound on the lengths is loose
(a program captures with the longest context it serves), so that short batches leave warps without work.
"""
import numpy as np
import pytest

import oracle
import workloads as W
from helpers import as_f64, assert_close, same_bytes, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LONGEST = 6000
LENS = [[6000, 6000, 6000], [300, 41, 700], [6000, 1, 3000], [17, 2000, 16], [1, 1, 1], [300, 41, 700], [90, 6000, 512]]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_306_gb300 as pa
    pa.load()


def _call(pa, kind, wl, t, groups, workspace):
    """One call into t["out"]; returns the workspace it used."""
    head = (t["out"], t["q"])
    tail = (wl.scale, LONGEST)
    pools, tables = (t["k_cache"], t["v_cache"]), (t["block_tables"], t["seq_lens"])
    if kind == "plain":
        return pa.pa_decode(*head, *pools, *tables, *tail, workspace=workspace)
    if kind == "partitions":
        return pa.pa_decode(*head, *pools, *tables, *tail, 64, workspace=workspace)
    if kind == "scaled":
        return pa.pa_decode_scaled(*head, *pools, *tables, *tail, wl.k_scale, wl.v_scale, workspace=workspace)
    if kind == "step":
        return pa.pa_decode_step(*head, t["key"], t["value"], *pools, None, *tables, *tail, workspace=workspace)
    return pa.pa_decode_shared(*head, None, None, *pools, None, *tables, *groups, *tail, workspace=workspace)


@pytest.mark.parametrize("kind,dtype,H,Hkv,D,bs", [
    ("plain", "f16", 8, 2, 128, 16), ("plain", "f32", 4, 4, 64, 16), ("plain", "bf16", 2, 2, 128, 32),
    ("plain", "bf16", 32, 2, 64, 16), ("partitions", "f16", 4, 2, 64, 32), ("scaled", "fp8", 4, 4, 128, 16),
    ("scaled", "fp8", 20, 2, 64, 32), ("step", "f16", 8, 2, 128, 16), ("shared", "bf16", 8, 2, 128, 16),
])
def test_a_captured_decode_follows_its_lengths(kind, dtype, H, Hkv, D, bs):
    import paged_kv_cache_306_gb300 as pa
    q_dtype = "f16" if dtype == "fp8" else None
    wl = W.make_private(f"replay-{kind}", dtype, [LONGEST] * 3, H, Hkv, D, bs, seed=17, q_dtype=q_dtype,
                        partition_size=-1, poison=False)
    groups = None
    if kind == "shared":
        wl.block_tables[1:, :40] = wl.block_tables[0, :40]
        groups = (torch.zeros(3, dtype=torch.int32, device="cuda"), torch.full((3,), 40, dtype=torch.int32, device="cuda"))
    t = upload(wl)
    t["out"] = torch.empty_like(t["q"])
    clean = t["k_cache"].clone(), t["v_cache"].clone()
    ws = _call(pa, kind, wl, t, groups, None)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert _call(pa, kind, wl, t, groups, ws) is ws
    k64, v64 = wl.clone_pools()
    for lens in LENS:
        t["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        outs = []
        for captured in (False, True):
            t["k_cache"].copy_(clean[0])
            t["v_cache"].copy_(clean[1])
            t["out"].zero_()
            if captured:
                g.replay()
            else:
                _call(pa, kind, wl, t, groups, None)
            outs.append(t["out"].clone())
        assert pa.pa_get_device_error() == 0
        assert same_bytes(*outs), f"lengths {lens}: off by {(outs[0] - outs[1]).abs().max().item():.3e}"
        if kind != "step":
            ref = oracle.decode(wl.q, k64, v64, wl.block_tables, np.array(lens, np.int32), wl.scale, dtype,
                                q_dtype=wl.q_dtype, k_scale=wl.k_scale, v_scale=wl.v_scale)
            assert_close(as_f64(outs[1]), ref, dtype, out_dtype=wl.q_dtype)


def test_a_captured_decode_on_the_built_in_scratch_follows_its_lengths():
    import paged_kv_cache_306_gb300 as pa
    lib = pa.load()
    wl = W.make_private("replay-noalloc", "f16", [2000], 8, 2, 64, 16, seed=18, partition_size=-1, poison=False)
    t = upload(wl)
    out = torch.empty_like(t["q"])

    def call():
        st = lib.pa_decode_noalloc(out.data_ptr(), t["q"].data_ptr(), t["k_cache"].data_ptr(), t["v_cache"].data_ptr(),
                                   t["block_tables"].data_ptr(), wl.max_blocks_per_seq, t["seq_lens"].data_ptr(), 1,
                                   2000, 8, 2, 64, 16, wl.num_blocks, wl.scale, -1, 1,
                                   torch.cuda.current_stream().cuda_stream)
        assert st == 0
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for L in (2000, 150, 1, 1999, 333):
        t["seq_lens"].fill_(L)
        want = torch.empty_like(out)
        pa.pa_decode(want, t["q"], t["k_cache"], t["v_cache"], t["block_tables"], t["seq_lens"], wl.scale, 2000)
        out.zero_()
        g.replay()
        assert pa.pa_get_device_error() == 0
        assert same_bytes(out, want), f"length {L}"

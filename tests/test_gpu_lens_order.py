"""Lengths and prefix groups that the kernel right before a decode call writes: the call may start while that kernel still
runs, and what it writes must count all the same.  (Here a kernel of this library, which lets the next one start early:
pa_rope copies the bits of the dims that it does not turn, and they are the lengths.)"""
import numpy as np
import pytest

from oracle import masked
from masked_checks import Pools, f64, queries
from masked_rows import check_rows

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
S, LONGEST = 24, 1500


@pytest.fixture(scope="module")
def pa():
    import paged_kv_cache_306_gb300 as m
    m.load()
    assert m.pa_get_device_error() in m.DEVICE_ERRORS     # (and cleared)
    return m


class Courier:
    """int32 arrays in device memory that a rope kernel brings there."""

    def __init__(self, pa):
        self.pa, self.freq = pa, pa.pa_rope_frequencies(16)[0].cuda()
        self.pos = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.rows, self.key = torch.zeros(1, 3, 64, device="cuda"), torch.zeros(1, 1, 64, device="cuda")
        self.key_out = torch.empty_like(self.key)
        ints = self.rows.view(torch.int32)
        self.lens, self.group, self.blocks = (ints[0, i, 16:16 + S] for i in range(3))

    def parcel(self, *arrays):
        x = torch.zeros(1, 3, 64, dtype=torch.int32)
        for i, a in enumerate(arrays):
            x[0, i, 16:16 + S] = torch.from_numpy(np.asarray(a, np.int32))
        return x.cuda().view(torch.float32)

    def bring(self, parcel):
        self.pa.pa_rope(self.rows, self.key_out, parcel, self.key, self.pos, self.freq)


def lengths(seed):
    n = np.random.default_rng(seed).integers(1, LONGEST + 1, S)
    n[:3] = [1, LONGEST, 17]
    return np.random.default_rng(seed + 50).permutation(n)


@pytest.mark.parametrize("call", ["decode", "masked", "step"])
@pytest.mark.parametrize("dtype,group", [("f16", 4), ("f16", 1), ("bf16", 12)])
def test_lengths_from_the_kernel_before(pa, call, dtype, group):
    pools = Pools([LONGEST] * S, 2, 64, 16, dtype, 3)
    kc, vc, bt = pools.on("cuda")
    q = queries(S, 2 * group, 64, dtype, 4)
    qg, c = q.cuda(), Courier(pa)
    sets = [lengths(i) for i in range(4)]
    parcels, outs, ws = [c.parcel(n) for n in sets], [], None
    # (the step writes each sequence's newest row: the one that is there, so that no call changes the pools)
    news = [[torch.stack([(kc[bt[s, (n - 1) // 16].long(), :, :, (n - 1) % 16].reshape(2, 64) if x is kc else
                           vc[bt[s, (n - 1) // 16].long(), :, :, (n - 1) % 16]) for s, n in enumerate(ns)])
             for x in (kc, vc)] for ns in sets]
    c.bring(parcels[3])
    torch.cuda.synchronize()
    for rep in range(24):
        out = torch.empty_like(qg)
        c.bring(parcels[rep % 4])
        if call == "masked":
            ws = pa.pa_decode_masked(out, qg, kc, vc, bt, c.lens, 0.125, LONGEST, 9.0, None, 700, workspace=ws)
        elif call == "decode":
            ws = pa.pa_decode(out, qg, kc, vc, bt, c.lens, 0.125, LONGEST, workspace=ws)
        else:
            ws = pa.pa_decode_step(out, qg, *news[rep % 4], kc, vc, None, bt, c.lens, 0.125, LONGEST, workspace=ws)
        outs.append(out)
    assert pa.pa_get_device_error() == 0
    kw = dict(softcap=9.0, window=700) if call == "masked" else {}
    refs = [masked.decode(f64(q), *pools.exact(), pools.table, n, 0.125, 16, **kw) for n in sets]
    for rep, out in enumerate(outs):
        check_rows(out, refs[rep % 4], q, pools, 0.125, kw.get("softcap", 0.0), 0.0, dtype, f"call {rep}")


def test_prefix_groups_from_the_kernel_before(pa):
    """Sequences of one prompt: the same first blocks in their tables, said to be shared, by more or less of them."""
    pools = Pools([LONGEST] * S, 2, 64, 16, "f16", 5)
    pools.table[:, :60] = pools.table[0, :60]
    kc, vc, bt = pools.on("cuda")
    q = queries(S, 8, 64, "f16", 6)
    qg, c = q.cuda(), Courier(pa)
    rng = np.random.default_rng(7)
    sets = []
    for i in range(4):
        n = np.maximum(lengths(10 + i), 20)
        sets.append((n, np.sort(rng.integers(0, 1 + 3 * i, S)), np.minimum(rng.integers(0, 61, S), n // 16)))
    parcels, outs, ws = [c.parcel(*x) for x in sets], [], None
    c.bring(parcels[3])
    torch.cuda.synchronize()
    for rep in range(24):
        out = torch.empty_like(qg)
        c.bring(parcels[rep % 4])
        ws = pa.pa_decode_shared(out, qg, None, None, kc, vc, None, bt, c.lens, c.group, c.blocks, 0.125, LONGEST,
                                 workspace=ws)
        outs.append(out)
    assert pa.pa_get_device_error() == 0
    refs = [masked.decode(f64(q), *pools.exact(), pools.table, x[0], 0.125, 16) for x in sets]
    for rep, out in enumerate(outs):
        check_rows(out, refs[rep % 4], q, pools, 0.125, what=f"call {rep}")

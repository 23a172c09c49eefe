"""What the marked sequences and the sharp bound of the FP4 decode tests can tell apart (on the CPU).

Mistakes are planted in the expected output; each has to fall outside what a right kernel may give.
"""
import numpy as np
import pytest

import oracle
from fp4_checks import LONG, RANDOM, Markers, sharp_bound_of
from helpers import half_ulp
from oracle import fp4

IDS = ["-".join(map(str, c[0])) for c in LONG]


@pytest.mark.parametrize("case", LONG, ids=IDS)
def test_the_expected_output_is_the_oracles(case):
    m = Markers(*case)
    k64, v64 = fp4.f64_pools(m.k, m.v, m.D, m.bs, m.k_scale, m.v_scale)
    ref = oracle.decode(m.q, k64, v64, m.table, np.array(m.lens, np.int32), m.scale, "f64", q_dtype=m.q_dtype)
    for i in range(len(m.lens)):
        assert np.abs(m.expected(i) - ref[i]).max() <= 2.0 ** -18 * np.abs(ref[i]).max()
        assert m.excess(i, m.rounded(ref[i])) <= 0


@pytest.mark.parametrize("case", LONG, ids=IDS)
def test_a_lost_doubled_or_misweighted_chunk_is_rejected(case):
    m = Markers(*case)
    for i, L in enumerate(m.lens):
        if L < 2:
            continue
        assert m.excess(i, np.zeros_like(m.expected(i))) > 0
        for at in {0, 32, L // 2 // 32 * 32, (L - 1) // 32 * 32}:           # a chunk of 32 tokens, the last one too
            if at >= L or L <= 32:
                continue
            # (a weight of a quarter more or less: a maximum that is off by a third in log2 units)
            for factor in (0.0, 2.0, 1.25, 0.75):
                w = np.ones(L)
                w[at:at + 32] = factor
                assert m.excess(i, m.rounded(m.expected(i, w))) > 0, (L, at, factor)
        w = np.ones(L)                                                        # a CTA's share: 1 / 152 of the launch
        w[L // 3:L // 3 + max(1, L // 152)] = 0
        assert m.excess(i, m.rounded(m.expected(i, w))) > 0


@pytest.mark.parametrize("q_dtype,D,bs,G,Hkv,lens", RANDOM)
def test_the_sharp_bound_rejects_no_output_and_a_lost_tenth(q_dtype, D, bs, G, Hkv, lens):
    pytest.importorskip("torch")
    from test_gpu_fp4 import KS, VS, Case
    c = Case(lens, G, Hkv, D, bs, q_dtype)
    ref, bound = sharp_bound_of(c, KS, VS)
    assert np.isfinite(bound).all()
    limit = bound + half_ulp(np.abs(ref) + bound, q_dtype)
    k64, v64 = fp4.f64_pools(c.k, c.v, D, bs, KS, VS)
    short = np.array([L - L // 10 for L in lens], np.int32)
    lost = oracle.decode(c.q, k64, v64, c.table, short, c.scale, "f64", q_dtype=q_dtype)
    for i, L in enumerate(lens):
        assert np.median(limit[i]) < 0.5 * np.sqrt((ref[i] ** 2).mean())
        assert (np.abs(ref[i]) > limit[i]).mean() > 0.5                       # an all-zero output
        if L >= 10:
            assert (np.abs(lost[i] - ref[i]) > limit[i]).any()

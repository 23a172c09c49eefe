"""What the marked sequences of the masked calls' GPU tests can tell apart (no GPU): mistakes are planted in the expected
rows, and each has to fall outside what a right kernel may give."""
import numpy as np
import pytest

from masked_checks import slopes_of
from masked_marks import LN2, Marked, rounded
from oracle import masked

pytest.importorskip("torch")
TYPES = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "fp8"), ("bf16", "fp8")]
KINDS = [dict(), dict(softcap=3.0), dict(slopes=True), dict(softcap=5.0, slopes=True)]


def small_slopes(h):
    return slopes_of(h) * 2.0 ** -8


@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="/".join)
def test_the_expected_row_is_the_oracles(types, kw):
    kw = dict(kw, window=50)
    if kw.pop("slopes", False):
        kw["slopes"] = small_slopes(4)
    m = Marked([1, 50, 200], 2, 64, 16, types[1], 1)
    q = m.queries(3, 4, types[0]).double().numpy()
    ref = masked.decode(q, *m.exact(), m.table, m.lens, LN2, 16, **kw)
    for s, n in enumerate(m.lens):
        row = m.row(s, n - 1, 4, **kw)
        assert np.abs(row - ref[s]).max() <= 1e-12
        assert m.excess(rounded(row, types[0]), row, types[0]).max() <= 0
    k, v = masked.rows_of(*m.exact(), m.table[2], 200, 16)
    for p, prefix in ((0, 130), (60, 130), (199, 500)):
        row = masked.attend(q[0], p, k, v, LN2, prefix=prefix, **kw)
        assert np.abs(row - m.row(2, p, 4, prefix=prefix, **kw)).max() <= 1e-12


@pytest.mark.parametrize("kw", KINDS, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("n,window,d", [(17, 0, 64), (700, 0, 64), (700, 129, 64), (2000, 1024, 128), (300, 1, 64), (300, 2, 64)])
def test_one_position_lost_doubled_or_too_many(types, n, window, d, kw):
    kw = dict(kw, window=window)
    if kw.pop("slopes", False):
        kw["slopes"] = small_slopes(4)
    m = Marked([n], 2, d, 16, types[1], n)
    for p in {n - 1, n // 2}:
        ref = m.row(0, p, 4, **kw)
        lo = max(0, p - window + 1) if window else 0

        def rejected(row):          # in every head
            return (m.excess(rounded(row, types[0]), ref, types[0], bias=8.0).max(1) > 0).all()
        for at in {lo, lo + 1, (lo + p) // 2, p - 1, p}:
            if not lo <= at <= p or p == lo:
                continue
            for factor in (0.0, 2.0):
                w = np.ones(n)
                w[at] = factor
                assert rejected(m.row(0, p, 4, weight=w, **kw)), (p, at, factor)
        for shift in ((-1, 0), (1, 0), (0, 1), (0, -1)):
            if lo + shift[0] < 0 or p + shift[1] >= n or lo + shift[0] > p + shift[1]:
                continue
            assert rejected(m.row(0, p, 4, shift=shift, **kw)), (p, shift)


@pytest.mark.parametrize("types", TYPES, ids="/".join)
@pytest.mark.parametrize("n,run", [(20011, 16), (40000, 16), (150001, 64), (9000, 8)])
def test_a_run_of_a_long_sequence_lost_or_misweighted(types, n, run):
    m = Marked([n], 1, 64, 16, types[1], n, marks="stretch")
    ref = m.row(0, n - 1, 2)
    for at in {0, n // 3 // 16 * 16, n - run}:
        for factor in (0.0, 2.0):
            w = np.ones(n)
            w[at:at + run] = factor
            assert (m.excess(rounded(m.row(0, n - 1, 2, weight=w), types[0]), ref, types[0]).max(1) > 0).all(), (at, factor)
    w = np.ones(n)                 # a piece's weight off by an eighth (its maximum by a sixth in log2 units)
    w[n // 4:n // 4 + n // 100] = 1.125
    assert (m.excess(rounded(m.row(0, n - 1, 2, weight=w), types[0]), ref, types[0]).max(1) > 0).all()

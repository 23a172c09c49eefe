"""Checks of capped, biased and masked attention row by row (a sequence's head, or a query row's): every element
against a bound from that row's own scores, and the row's norm, so that no row hides behind another."""
import numpy as np

from masked_checks import EPS, P_ROUNDING, TINY, f64


def row_bounds(q, k, v, ref, scale, softcap, bias, dtype, p_rounding):
    """(per element, per row relative) for rows [.., D] of q and ref, with the errors of masked_checks' attention_bound
    but for the tanh, which is off by 2^-20 of its result: at most of the cap, and of the row's largest score (and
    what a score is off by, it is off by less after the tanh, and by no more than its range)."""
    d = q.shape[-1]
    reach = abs(scale) * np.abs(q).sum(-1, keepdims=True) * np.abs(np.nan_to_num(k)).max()
    capped = np.minimum(reach, softcap) if softcap else 0.0
    dot = (d + 4) * 2.0 ** -24 * reach
    arg = (np.minimum(dot, 2 * softcap) if softcap else dot) + capped * 2.0 ** -20 + bias * 2.0 ** -22
    own = EPS[dtype] * (1 + 2.0 ** -6)
    each = 2 * (arg + 2.0 ** -20 + p_rounding) * np.abs(np.nan_to_num(v)).max() + own * np.abs(ref) + TINY[dtype]
    # as a whole: the weights' roundings are independent, so that a row of any number of keys is off by their size
    # (4: the norm of a few keys' worth may fall together); its own rounding is at most `own` of each element
    return each, own + 4 * (p_rounding + 2.0 ** -20 + np.minimum(arg, 1.0))


def check_rows(out, ref, q, pools, scale, softcap=0.0, bias=0.0, dtype="f16", what=""):
    got = f64(out)
    assert np.isfinite(got).all(), f"{what}: {np.isnan(got).sum()} NaN of {got.size}"
    each, whole = row_bounds(f64(q), *pools.exact(), ref, scale, softcap, bias, dtype, P_ROUNDING[pools.dtype])
    worst = np.max(np.abs(got - ref) / each)
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound (error {np.abs(got - ref).max():.2e})"
    rel = np.linalg.norm(got - ref, axis=-1, keepdims=True) / np.maximum(np.linalg.norm(ref, axis=-1, keepdims=True), 1e-30)
    worst = np.max(rel / whole)
    assert worst <= 1.0, f"{what}: a row {worst:.2f} times the relative bound (relative error {rel.max():.2e})"

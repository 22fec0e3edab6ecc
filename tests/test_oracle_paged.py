"""Pins of the paged cache's plain restatement: bounds bound, scores bound the
logits, joined bounds equal fresh ones, and the page tables keep their counts."""
import numpy as np
import pytest

from oracle import paged as P


def rows(seed, n, scale=1.0):
    x = np.random.default_rng(seed).standard_normal((n, 128)) * scale
    return x.astype(np.float32).view(np.uint32).__and__(0xFFFF0000).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("scale", [1e-20, 1e-6, 0.01, 1.0, 300.0, 60000.0])
def test_bounds_hold_and_use_the_finest_step(scale):
    x = rows(1, 37, scale)
    lo, hi, e = P.bounds(x)
    assert np.all(lo * 2.0 ** e <= x.min(0)) and np.all(hi * 2.0 ** e >= x.max(0))
    assert np.all((lo + 1) * 2.0 ** e > x.min(0)) and np.all((hi - 1) * 2.0 ** e < x.max(0))
    assert np.abs(lo).max() <= 127 and np.abs(hi).max() <= 127
    assert e == P.EXP_MIN or np.abs(x).max() > 127 * 2.0 ** (e - 1)


def test_step_exponent_at_its_borders():
    assert P.step_exponent(0.0) == P.EXP_MIN
    assert P.step_exponent(127.0) == 0 and P.step_exponent(127.5) == 1 and P.step_exponent(63.5) == -1
    assert P.step_exponent(127 * 2.0 ** P.EXP_MIN) == P.EXP_MIN


def test_bounds_do_not_depend_on_how_rows_are_divided():
    x = np.concatenate([rows(2, 9, 0.1), rows(3, 20, 5.0), rows(4, 7, 40.0)])
    lo, hi, e = P.bounds(x)
    a = P.bounds(x[:9])
    for part in (x[9:29], x[29:]):
        b = P.bounds(part)
        ee = max(a[2], b[2])
        a = (np.minimum(*(np.floor(r[0] * 2.0 ** (r[2] - ee)) for r in (a, b))),
             np.maximum(*(np.ceil(r[1] * 2.0 ** (r[2] - ee)) for r in (a, b))), ee)
    assert a[2] == e and np.array_equal(a[0], lo) and np.array_equal(a[1], hi)


def test_the_score_bounds_the_summed_code_logits_of_every_row():
    k, q = rows(5, 64), rows(6, 4, 2.0)
    c = P.query_codes(q)
    s = P.block_score(c, *P.bounds(k))
    assert s >= (c @ k.T).sum(0).max()
    assert abs(c).max() <= 127


def test_choice_by_hand():
    assert P.choose_blocks([5, 1, 9, 9, 2, 7], 4, 1, 1) == [0, 2, 3, 5]
    assert P.choose_blocks([5, 9, 9, 9, 2, 7], 3, 1, 1) == [0, 1, 5]      # the tie goes to the lower block
    assert P.choose_blocks([1, 2, 3], 3, 0, 0) == [0, 1, 2]
    assert P.choose_blocks([1, 2, 3, 0], 2, 0, 2) == [2, 3]


def test_tables_by_hand():
    t = P.Tables(8, 4, 4)
    assert t.reserve([0], [70]) == [] and t.pages[0] == [0, 1]
    assert t.fork([0, 0], [1, 2]) == [] and t.refs() == [3, 3, 0, 0, 0, 0, 0, 0]
    # all three extend the shared last page: the first two copy it, the last one keeps it
    assert t.reserve([2, 0, 1], [1, 1, 1]) == [(1, 2, 1), (1, 3, 1)]
    assert t.pages == [[0, 3], [0, 1], [0, 2], []]
    assert t.truncate([2, 2, 0], [0, 0, 64]) == [1] and t.refs() == [2, 1, 0, 0, 0, 0, 0, 0]
    assert t.reserve([3, 0], [200, 1]) is not None and t.pages[3] == [2, 3, 4, 5] and t.pages[0] == [0, 6]
    assert t.reserve([3], [57]) is None and t.reserve([2], [129]) is None     # past its table row; no pages left
    t.truncate([3], [0])
    assert t.compact() == [(6, 2)] and t.pages[:2] == [[0, 2], [0, 1]]


def test_the_attention_bound_shrinks_with_the_values():
    """Values times a power of two have the same codes while their steps (here from 0.003 on) stay normal in fp16, above
    2^-14, and a bound times that power; the older bound keeps an absolute part."""
    k, v, q, vis = rows(7, 50), rows(8, 50, 0.3), rows(9, 1, 2.0)[0], np.arange(50) < 43
    found = []
    for f in (1.0, 2.0 ** -4):
        kd, kp, _ = P.dequantised(k, 4)
        vd, vp, vc = P.dequantised(v * f, 8)
        want = P.attend(q, kd, vd, vis)
        found.append((want, P.attend_bound(q, kd, kp, vp, vc, P.quantize(v * f, 8)[1], vis, want),
                      P.attend_error(q, kd, kp, vp, vc, vis, want)))
    (w0, b0, e0), (w1, b1, e1) = found
    assert np.array_equal(w0 * 2.0 ** -4, w1) and np.allclose(b0 * 2.0 ** -4, b1, rtol=1e-12)
    assert (b0 <= e0).all() and (e1 > e0 * 2.0 ** -4).all()
    assert not P.attend_bound(q, kd, kp, vp, vc, P.quantize(v, 8)[1], vis & False, 0 * want).any()


def test_weights_of_whole_softmaxes_sum_to_the_number_of_rows():
    k, q = rows(5, 40), rows(6, 6)
    lims = [40, 39, 17, 1, 0, -3]
    lse = [np.log(np.exp(k[:n] @ r / 128 ** 0.5).sum()) if n > 0 else -np.inf for r, n in zip(q, lims)]
    w = P.weights(q, k, lse, lims)
    assert np.isclose(w.sum(), 4.0) and w[39] < w.sum() and (w >= 0).all()
    assert np.isclose(P.weights(q[3:4], k, lse[3:4], [1])[0], 1.0)


@pytest.mark.parametrize("n, k, first, last", [(10, 7, 2, 3), (200, 64, 4, 32), (70, 69, 0, 69), (65, 1, 0, 0), (9, 5, 5, 0),
                                               (30, 0, 0, 0), (12, 12, 1, 1), (5, 9, 0, 2)])
def test_eviction_keeps_the_largest_and_moves_no_more_than_it_must(n, k, first, last):
    mass = np.random.default_rng(n).integers(0, 5, n).astype(float)
    src = P.keep_positions(mass, n, k, first, last)
    m = min(n, k)
    assert len(src) == m and len(set(src)) == m and all(0 <= s < n for s in src)
    if n <= k:
        assert src == list(range(n))
        return
    assert set(range(first)) | set(range(n - last, n)) <= set(src)
    assert src[k - last:] == list(range(n - last, n))
    out = [j for j in range(first, n - last) if j not in src]
    chosen = [j for j in src if first <= j < n - last]
    for a in out:
        assert all(mass[b] > mass[a] or (mass[b] == mass[a] and b < a) for b in chosen)
    w = k - last
    assert all(src[j] == j for j in range(w) if j in src)          # below w a kept position keeps its place
    moved = [src[j] for j in range(w) if src[j] != j]
    assert moved == sorted(moved) and all(s >= w for s in moved)


def test_eviction_takes_nan_for_the_largest():
    mass = np.array([1.0, np.nan, 3.0, np.inf, np.nan, 2.0])
    assert P.keep_positions(mass, 6, 2, 0, 0) == [4, 1]
    assert sorted(P.keep_positions(mass, 6, 3, 0, 0)) == [1, 3, 4]

"""Pins of the bounded cache's oracle functions on tiny cases, by other means than their own."""
import itertools
import math

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("L,window,sinks", [(7, 3, 2), (7, 0, 2), (7, 3, 0), (7, 9, 1), (3, 1, 2), (5, 0, 0), (1, 1, 0)])
def test_visible_tokens_counted_one_by_one(L, window, sinks):
    got = oracle.window_visible(L, window, sinks)
    want = [i for i in range(L) if i in range(sinks) or i in range(max(0, L - window), L)]
    assert list(np.flatnonzero(got)) == want


def test_window_rows_is_attention_over_the_visible_rows_alone():
    rng = np.random.default_rng(3)
    qf, rows = rng.standard_normal((2, 6)), rng.standard_normal((9, 6))
    r = oracle.window_rows(qf, rows, 3, 2, 0.5, 4)
    seen = [0, 1, 6, 7, 8]
    for h in range(2):
        e = [math.exp(0.5 * sum(a * b for a, b in zip(qf[h], rows[t]))) for t in seen]
        assert np.allclose(r["lse"][h], math.log(sum(e)), rtol=1e-13)
        for k in range(4):
            assert np.isclose(r["out_lat"][h, k], sum(x * rows[t, k] for x, t in zip(e, seen)) / sum(e), rtol=1e-12)
    empty = oracle.window_rows(qf, rows, 0, 0, 0.5, 4)
    assert np.all(empty["out_lat"] == 0) and np.all(np.isneginf(empty["lse"]))


def test_hidden_rows_do_not_enter():
    rng = np.random.default_rng(4)
    qf, rows = rng.standard_normal((2, 6)), rng.standard_normal((9, 6))
    a = oracle.window_rows(qf, rows, 3, 2, 0.5, 4)
    rows[2:6] = np.nan
    b = oracle.window_rows(qf, rows, 3, 2, 0.5, 4)
    assert np.array_equal(a["out_lat"], b["out_lat"])


def test_weight_sums_add_to_the_number_of_heads():
    """With the row's own log-sum-exps, the weights of all tokens of all heads add to the heads."""
    rng = np.random.default_rng(5)
    qf, rows = rng.standard_normal((3, 6)), rng.standard_normal((8, 6))
    lse = oracle.attend_rows(qf, rows, 0.7, 4)["lse"]
    w, _ = oracle.attn_weight_sums(qf, rows, lse, 0.7)
    assert w.shape == (8,) and np.isclose(w.sum(), 3.0, rtol=1e-13)
    p = oracle.attend_rows(qf, rows, 0.7, 4)["p"]
    assert np.allclose(w, p.sum(axis=0), rtol=1e-12)


def test_evict_keeps_the_heaviest_set_by_brute_force():
    rng = np.random.default_rng(6)
    for trial in range(40):
        L = int(rng.integers(5, 9))
        keep = int(rng.integers(3, L))
        sinks = int(rng.integers(0, 2))
        recent = int(rng.integers(0, keep - sinks))
        w = rng.integers(0, 4, L).astype(float)
        got = oracle.evict_keep(w, L, keep, sinks, recent)
        assert len(got) == keep and np.all(np.diff(got) > 0)
        sure = set(range(sinks)) | set(range(L - recent, L))
        sets = [c for c in itertools.combinations(range(L), keep) if sure <= set(c)]
        best = max(sum(w[list(c)]) for c in sets)
        assert sum(w[got]) == best
        # among the heaviest sets the lowest tokens: the first in lexicographic order
        assert tuple(got) == min(c for c in sets if sum(w[list(c)]) == best)


def test_evict_orders_nan_zero_and_infinities():
    w = np.array([np.nan, -np.inf, -0.0, 0.0, np.inf, -1.0, np.nan])
    assert list(oracle.evict_keep(w, 7, 1, 0, 0)) == [4]
    assert list(oracle.evict_keep(w, 7, 2, 0, 0)) == [2, 4]      # -0 and 0 are equal: the lower token
    assert list(oracle.evict_keep(w, 7, 4, 0, 0)) == [2, 3, 4, 5]
    assert list(oracle.evict_keep(w, 7, 5, 0, 0)) == [1, 2, 3, 4, 5]
    assert list(oracle.evict_keep(w, 7, 6, 0, 0)) == [0, 1, 2, 3, 4, 5]
    assert list(oracle.evict_keep(w, 7, 7, 0, 0)) == list(range(7))
    assert list(oracle.evict_keep(w, 7, 3, 1, 1)) == [0, 4, 6]

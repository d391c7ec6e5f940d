"""CPU pins of the paged-cache oracle (oracle/paged.py): facts that do not come
from its own code, and planted mistakes that some pin must catch."""

from __future__ import annotations

import types

import numpy as np
import pytest

import oracle
import oracle.paged as paged_mod


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def _paged(k, P, seed):
    """(B, Hkv, L, D) keys as a pool in random page order, and the table."""
    B, Hkv, L, D = k.shape
    n = -(-L // P)
    order = np.random.default_rng(seed).permutation(B * n)
    pool = _rand(seed + 1, B * n, Hkv, P, D)
    table = order.reshape(B, n)
    for b in range(B):
        for p in range(L):
            pool[table[b, p // P], :, p % P] = k[b, :, p]
    return pool, table


def pin_rows_of_full_attention(m):
    """each request is the last rows of causal attention over its sequence,
    every query head with its group's keys"""
    B, H, Hkv, L, D, P, Tq = 2, 4, 2, 23, 8, 5, 3
    q, k, v = _rand(1, B, H, L, D), _rand(2, B, Hkv, L, D), _rand(3, B, Hkv, L, D)
    pk, table = _paged(k, P, 7)
    pv, _ = _paged(v, P, 7)
    full, lse = oracle.attention_forward(q, k.repeat(2, 1), v.repeat(2, 1), 0.4)
    o, l, a, _ = m.decode(q[:, :, L - Tq:], pk, pv, table, [L] * B, 0.4)
    assert np.allclose(o, full[:, :, L - Tq:], atol=1e-12) and np.allclose(l, lse[:, :, L - Tq:])
    assert (a >= np.abs(o) - 1e-12).all()
    # a shorter length is another sequence
    o2, _, _, _ = m.decode(q[:, :, 9:12], pk, pv, table, [12, 12], 0.4)
    assert np.allclose(o2, full[:, :, 9:12], atol=1e-12)


def pin_rows_without_keys(m):
    k = _rand(4, 2, 1, 4, 8)
    o, l, _, _ = m.decode(_rand(5, 3, 1, 2, 8), k, k, np.array([[0], [1], [-1]]), [0, 1, 4], 1.0)
    assert (o[0] == 0).all() and np.isneginf(l[0]).all()
    assert (o[1, 0, 0] == 0).all() and np.allclose(o[1, 0, 1], k[1, 0, 0])
    assert (o[2] == 0).all() and np.isneginf(l[2]).all()


def pin_listed_pages(m):
    """all pages listed is dense; one page listed is that page alone"""
    k, table = _paged(_rand(6, 1, 2, 17, 8), 4, 3)
    q = _rand(8, 1, 2, 1, 8)
    dense = m.decode(q, k, k, table, [17], 0.3)
    every = np.array([[[0, 1, 2, 3, 4]] * 2])
    assert np.allclose(m.decode(q, k, k, table, [17], 0.3, every)[0], dense[0])
    one = m.decode(q, k, k, table, [17], 0.3, np.array([[[4, -1, -1, -1, -1]] * 2]))
    assert np.allclose(one[0][0, :, 0], k[table[0, 4], :, 0])


def pin_select_bounds_the_scores(m):
    """with all keys of a page equal its score is q . k; the order follows"""
    B, L, P, D, K = 1, 40, 4, 8, 4
    keys = _rand(9, 10, 1, 1, D)
    bounds = keys.repeat(2, 2)
    q = _rand(10, B, 1, 1, D)
    table = np.arange(10)[None]
    got = m.select(q, bounds, table, [L], P, K, 0, 0)[0, 0]
    want = np.sort(np.argsort(-(keys[:, 0, 0] @ q[0, 0, 0]))[:K])
    assert np.array_equal(got, want)
    assert np.array_equal(m.select(q, bounds, table, [9], P, K, 0, 0)[0, 0], [0, 1, 2, -1])
    forced = m.select(-q, bounds, table, [L], P, 3, 1, 2)[0, 0]
    assert np.array_equal(forced, [0, 8, 9])
    same = np.broadcast_to(bounds[:1], bounds.shape)
    assert np.array_equal(m.select(q, same, table, [L], P, K, 0, 1)[0, 0], [0, 1, 2, 9])


def pin_append_keeps_lowest_and_highest(m):
    kn = np.array([3.0, -1.0, 2.0, 7.0]).reshape(4, 1, 1)
    k = np.zeros((2, 1, 2, 1))
    b = np.stack([np.full((2, 1, 1), -5.0), np.full((2, 1, 1), 5.0)], 2)
    k2, _, b2 = m.append(kn, kn, [1, 2, 3, -1], k, k, b)
    assert k2.ravel().tolist() == [0, 3, -1, 2] and k.ravel().tolist() == [0] * 4
    assert b2[0].ravel().tolist() == [-5, 5] and b2[1].ravel().tolist() == [-1, 2]


def pin_plan_by_hand(m):
    table = np.array([[4, 0, -1], [2, -1, -1], [-1, -1, -1], [3, -1, -1]])
    got = m.plan([3, -1, 2, 0], [5, 2, 0, 1], table, np.array([9, 1, 5, 6, 7, 8]), [1, 4], 3, 6)
    assert got["status"] == m.OK
    # request 0: positions 5 in page 0, 6 and 7 in a new page (ring entry 1)
    assert got["slots"].tolist() == [0 * 3 + 2, 1 * 3, 1 * 3 + 1, 5 * 3, 5 * 3 + 1, -1]
    assert got["positions"].tolist() == [5, 6, 7, 0, 1, -1]
    assert got["cu"].tolist() == [0, 3, 3, 5, 5] and got["lengths"].tolist() == [8, 0, 2, 1]
    assert got["state"].tolist() == [3, 5] and got["ring"].tolist() == [9, 1, 5, 6, 2, 8]
    assert got["table"][0].tolist() == [4, 0, 1] and got["table"][2].tolist() == [5, -1, -1]
    few = m.plan([3, -1, 2, 0], [5, 2, 0, 1], table, np.array([9, 1, 5, 6, 7, 8]), [1, 2], 3, 6)
    assert few["status"] == m.TOO_LARGE and few["lengths"].tolist() == [5, 2, 0, 1]


def pin_plan_frees_held_pages_only(m):
    holed = np.array([[4, 0, -1], [6, 2, -1], [-1, -1, -1], [3, -1, -1]])
    got = m.plan([0, -1, 0, 0], [5, 6, 0, 1], holed, np.array([9, 1, 5, 4, 3, 8]), [1, 4], 3, 6)
    assert got["status"] == m.OK and got["state"].tolist() == [1, 5]
    assert got["ring"].tolist() == [9, 1, 5, 4, 2, 8] and got["lengths"].tolist() == [5, 0, 0, 1]


ALL_PINS = [pin_rows_of_full_attention, pin_rows_without_keys, pin_listed_pages,
            pin_select_bounds_the_scores, pin_append_keeps_lowest_and_highest, pin_plan_by_hand,
            pin_plan_frees_held_pages_only]


@pytest.mark.parametrize("pin", ALL_PINS, ids=lambda p: p.__name__)
def test_pin_holds(pin):
    pin(paged_mod)


MUTANTS = [
    ("new position off by one", "x = int(lengths[b]) - Tq + t", "x = int(lengths[b]) - Tq + t - 1"),
    ("heads of another group", "row_q = q[b, h * G + g, t]", "row_q = q[b, g, t]"),
    ("own key not seen", "if pos <= x]", "if pos < x]"),
    ("scale dropped", "s = scale * (keys @ row_q)", "s = keys @ row_q"),
    ("lists ignored", "if pages is None:", "if True:"),
    ("bounds swapped", "lo, hi = bounds[pg, h]", "hi, lo = -bounds[pg, h]"),
    ("ties to the higher index", "key=lambda i: (-score[i], i)", "key=lambda i: (-score[i], -i)"),
    ("last pages not forced", "set(range(n - n_last, n))", "set()"),
    ("old bounds kept", "if row == 0:", "if row < 0:"),
    ("ring's entries in reverse", "ring[(head + taken) % n_pool]", "ring[(tail - 1 - taken) % n_pool]"),
    ("pages that are not held freed", "if 0 <= table[b, i] < n_pool:       # a page that is held",
     "if True:"),
    ("freed to the head", "new_ring[(tail + freed) % n_pool]", "new_ring[(head + freed) % n_pool]"),
]


@pytest.mark.parametrize("desc,old,new", MUTANTS, ids=[m[0] for m in MUTANTS])
def test_planted_mistake_is_caught(desc, old, new):
    with open(paged_mod.__file__) as f:
        src = f.read()
    assert src.count(old) == 1, old
    mod = types.ModuleType("paged_mutant")
    exec(compile(src.replace(old, new), "paged_mutant", "exec"), mod.__dict__)
    for pin in ALL_PINS:
        try:
            with np.errstate(all="ignore"):
                pin(mod)
        except (AssertionError, ValueError, IndexError):
            return
    pytest.fail(f"no pin catches: {desc}")

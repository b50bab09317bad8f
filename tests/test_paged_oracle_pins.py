"""The definitions of the paged cache and of the beams' steps against hand-worked values and invariants."""
import math

import numpy as np
import pytest

import oracle as O
from oracle import paged_oracle as P


def test_scaled_frequencies():
    inv = np.array([1.0, 0.01, 1e-4])
    assert np.allclose(P.scaled_inv(inv, 4.0, 0, 0, 0), inv / 4)                     # all divided
    # 2 pi * 100 positions: 100, 1 and 0.01 turns; low 1, high 4: kept, divided, divided
    got = P.scaled_inv(inv, 4.0, 200 * math.pi, 1.0, 4.0)
    assert np.allclose(got, [1.0, 0.0025, 2.5e-5])
    # half way between: turns 2.5 -> keep 0.5 -> 0.5 + 0.5 / 4
    assert np.allclose(P.scaled_inv([1.0], 4.0, 5 * math.pi, 1.0, 4.0), [0.625])


def test_scaled_rotation_by_hand():
    x = np.array([[[1.0, 0.0, 0.0, 0.0]]])                                           # D = 4, base 100: w = 1, 0.1
    y = P.rope_scaled(x, [[2]], O.Rope("1d", 100.0), (2.0, 0, 0, 0, 3.0))            # position 2, halved, times 3
    assert np.allclose(y, [[[3 * math.cos(1), 0, 3 * math.sin(1), 0]]])
    x = np.array([[[0.0, 0.0, 0.0, 5.0, 1.0, 0.0]]])                                 # last 2 dims, one interleaved pair
    y = P.rope_scaled(x, [[2]], O.Rope("interleaved", 100.0, rot_offset=4, rot_dim=2), (2.0, 0, 0, 0, 1.0))
    assert np.allclose(y, [[[0, 0, 0, 5, math.cos(1), math.sin(1)]]])


@pytest.mark.parametrize("kind,secs,n_axes", [("1d", None, 1), ("sections", (2, 3, 2, 1), 4), ("2d", None, 2), ("interleaved", None, 1)])
def test_factor_one_is_the_plain_rotation(kind, secs, n_axes):
    r = np.random.default_rng(1)
    x, pos = r.standard_normal((3, 2, 16)), r.integers(0, 1000, (3, n_axes))
    rope = O.Rope(kind, 1e4, secs)
    assert np.allclose(P.rope_scaled(x, pos, rope, (1.0, 0, 0, 0, 1.0)), O.rope_apply(x, pos, rope), atol=1e-12)


def test_pages_hold_what_a_window_holds():
    """Chunks appended through shuffled pages attend as the same tokens in one fixed window."""
    r = np.random.default_rng(2)
    Hkv, G, D, page, T = 2, 3, 8, 4, 11
    k, v, q = r.standard_normal((T, Hkv, D)), r.standard_normal((T, Hkv, D)), r.standard_normal((T, Hkv * G, D))
    pk, pv = np.full((6, Hkv, page, D), np.nan), np.full((6, Hkv, page, D), np.nan)
    table = [[4, 0, 5]]
    got = []
    for a, b in ((0, 5), (5, 6), (6, 11)):
        P.paged_append(k[a:b], v[a:b], pk, pv, table, [b], [0, b - a], "f32")
        got.append(P.paged_attention(q[a:b], pk, pv, table, [b], [0, b - a])[0])
    ck, cv = (O.store(x, "f32").transpose(1, 0, 2) for x in (k, v))
    assert np.allclose(np.concatenate(got), O.prefill(q, ck, cv, T, "causal"), atol=1e-12)
    assert np.isnan(pk[5, :, 3]).all() and np.isnan(pk[[1, 2, 3]]).all()             # nothing else written


def test_tokens_that_see_nothing():
    pk = pv = np.ones((1, 1, 4, 8))
    o, _ = P.paged_attention(np.ones((3, 1, 8)), pk, pv, [[0]], [2], [0, 3])         # 3 new tokens, 2 slots
    assert (o[0] == 0).all() and np.allclose(o[1:], 1)


def test_beam_step_by_hand():
    z = np.log(np.array([[[0.5, 0.25, 0.25], [0.1, 0.6, 0.3]]]))
    s = np.log(np.array([[0.4, 0.5]]))
    got = P.beam_step(z, s, 3)[0]                                                    # .3 (1,1), .2 (0,0), .15 (1,2)
    assert [g[:2] for g in got] == [(1, 1), (0, 0), (1, 2)]
    assert np.allclose([g[2] for g in got], np.log([0.3, 0.2, 0.15]))
    got = P.beam_step(z, s, 3, finished=np.array([[0, 1]]), end_id=2)[0]             # .5 (1, end), .2 (0,0), then a tie
    assert [g[:2] for g in got] == [(1, 2), (0, 0), (0, 1)]
    got = P.beam_step(z, np.array([[0.0, -math.inf]]), 5)[0]
    assert [g[:2] for g in got] == [(0, 0), (0, 1), (0, 2), (-1, -1), (-1, -1)]
    bad = z.copy()
    bad[0, 0, 1] = math.nan
    assert all(g[0] == 1 for g in P.beam_step(bad, s, 3)[0])


def test_reorder_by_hand():
    page, layers = 4, 2
    pool = np.arange(layers * 8 * page, dtype=float).reshape(layers, 8, 1, page, 1)
    was = pool.copy()
    # three beams of 6 slots: shared page 0, tails 1, 2, 3, spares 5, 6, 7; beams 0 and 2 go on from beam 2, beam 1 from itself
    rows, lens, spares = P.reorder([[2, 1, 2]], [[[0, 1], [0, 2], [0, 3]]], [[6, 6, 6]], [[5, 6, 7]], [pool], 8)
    assert rows == [[[0, 3], [0, 2], [0, 7]]] and lens == [[6, 6, 6]] and spares == [[5, 6, 1]]   # page 1 is free again
    assert (pool[:, 7, 0, :2] == was[:, 3, 0, :2]).all() and (pool[:, 7, 0, 2:] == was[:, 7, 0, 2:]).all()
    same = [i for i in range(8) if i != 7]
    assert (pool[:, same] == was[:, same]).all()
    # beams that share a partly filled page (after a prompt): the first keeps it, no page is freed
    rows, lens, spares = P.reorder([[0, 0, 1]], [[[0, 1]] * 3], [[6, 6, 6]], [[5, 6, 7]], [pool], 8)
    assert rows == [[[0, 1], [0, 6], [0, 7]]] and spares == [[5, -1, -1]]
    # full pages are shared; no parent: nothing left; no spare: length -1
    assert P.reorder([[0, 0, 0]], [[[0, 1]] * 3], [[8, 8, 8]], [[5, 6, 7]], [pool], 8)[0] == [[[0, 1]] * 3]
    rows, lens, spares = P.reorder([[0, -1, 0]], [[[0, 1], [0, 2], [0, 3]]], [[6, 6, 6]], [[5, 6, 8]], [pool], 8)
    assert lens == [[6, 0, -1]] and spares == [[5, 6, 8]]

"""Pins of the sampling oracle: over a fine grid of random numbers the kept
tokens and the drawn one reproduce the target's distribution."""
import itertools

import numpy as np
import pytest

from oracle import sample as osm


def test_probabilities_of_special_rows():
    f = np.float32
    assert np.allclose(osm.probabilities(np.array([0, np.log(3), -np.inf, np.nan], f), 1.0), [0.25, 0.75, 0, 0])
    assert np.allclose(osm.probabilities(np.array([1, np.inf, np.inf, 0], f), 0.7), [0, 0.5, 0.5, 0])
    assert np.allclose(osm.probabilities(np.array([1, 3, 3, 2], f), 0.0), [0, 0.5, 0.5, 0])
    assert np.allclose(osm.probabilities(np.array([1, 3, -np.inf, 2], f), np.inf), [1 / 3, 1 / 3, 0, 1 / 3])
    assert not osm.probabilities(np.array([np.nan, -np.inf], f), 1.0).any()
    z = np.array([0.5, -1, 2], f)
    assert np.allclose(osm.probabilities(z, 2.0), np.exp(z / 2) / np.exp(z / 2).sum())


def test_draw_borders():
    w = np.array([0.0, 1.0, 0.0, 3.0, 0.0])
    assert [osm.draw(w, u)[0] for u in (0.0, 0.2, 0.25, 0.999, 1.0)] == [1, 1, 3, 3, 3]


def _mid(n):
    return (np.arange(n) + 0.5) / n


def test_one_draft_reproduces_the_target():
    p = np.array([0.125, 0.5, 0.25, 0.125])
    q = np.array([0.5, 0.25, 0.125, 0.125], dtype=np.float32)
    logits = np.log(np.stack([p, [0.25] * 4])).astype(np.float32)
    got = np.zeros(4)
    n = 64
    for x in range(4):
        for u1, u0 in itertools.product(_mid(n), _mid(n)):
            r = osm.accept(logits, [0, x], [u0, u1], draft=np.stack([q, q]))
            first = x if r.accept_len == 1 else r.bonus
            got[first] += q[x] / n ** 2
    assert np.allclose(got, p, atol=1.5 / n)


@pytest.mark.parametrize("kids", [[2], [1, 2], [3, 0, 1], [1, 1, 2]])
def test_picked_children_reproduce_the_target(kids):
    p = np.array([0.125, 0.5, 0.25, 0.125])
    T = 1 + len(kids)
    logits = np.log(np.stack([p] + [[0.25] * 4] * len(kids))).astype(np.float32)
    got = np.zeros(4)
    n = 16
    for us in itertools.product(_mid(n), repeat=T):
        r = osm.accept(logits, [0] + kids, us, parent=np.array([-1] + [0] * len(kids)))
        got[kids[r.accept_node - 1] if r.accept_len else r.bonus] += 1 / n ** T
    assert np.allclose(got, p, atol=2.0 / n)


def test_nothing_left_and_empty_rows():
    logits = np.array([[0, -np.inf], [0, 0]], dtype=np.float32)
    r = osm.accept(logits, [0, 0], [0.3, 1.0])       # u = 1: token 0, which has everything, is not accepted
    assert (r.accept_len, r.bonus) == (0, 0)
    r = osm.accept(np.full((2, 2), np.nan, dtype=np.float32), [0, 1], [0.3, 0.0])
    assert (r.accept_len, r.bonus) == (0, 0) and r.token_prob.tolist() == [1.0, 0.0]

"""Pins of oracle/filter.py."""
import numpy as np
import pytest

from oracle.filter import filtered
from oracle.sample import probabilities

ROW = np.log(np.array([0.1, 0.4, 0.05, 0.3, 0.15], np.float64)).astype(np.float32)


def kept(row, **kw):
    return np.flatnonzero(filtered(row, 1.0, **kw)[0]).tolist()


def test_hand_worked():
    assert kept(ROW) == [0, 1, 2, 3, 4] == kept(ROW, k=5) == kept(ROW, k=9) == kept(ROW, k=-1)
    assert kept(ROW, k=2) == [1, 3] and kept(ROW, k=1) == [1]
    assert kept(ROW, p=0.39) == [1] == kept(ROW, p=0.0) == kept(ROW, p=-3.0)
    assert kept(ROW, p=0.41) == [1, 3] == kept(ROW, p=0.69) and kept(ROW, p=0.71) == [1, 3, 4]
    assert kept(ROW, p=1.0) == kept(ROW, p=float("nan")) == [0, 1, 2, 3, 4]
    assert kept(ROW, m=0.3) == [1, 3, 4] and kept(ROW, m=2.0) == [1] and kept(ROW, m=float("nan")) == [0, 1, 2, 3, 4]
    # of the first two (0.4 and 0.3) 0.56 of 0.7 is 0.392: one stays; without top-k two would
    assert kept(ROW, k=2, p=0.56) == [1] and kept(ROW, p=0.56) == [1, 3]
    assert np.allclose(filtered(ROW, 1.0, k=2)[0], [0, 4 / 7, 0, 3 / 7, 0])


def test_ties_go_by_index():
    row = np.array([1, 2, 2, 2, 0, np.nan], np.float32)
    assert kept(row, k=2) == [1, 2] and kept(row, p=0.01) == [1] and kept(row, m=1.0) == [1, 2, 3]
    assert kept(np.array([0.0, -0.0, 0.0], np.float32), k=2) == [0, 1]
    assert filtered(row, 0.0, k=2)[0].tolist() == [0, 0.5, 0.5, 0, 0, 0]
    assert filtered(np.array([0, np.inf, np.inf], np.float32), 1.0, p=0.5)[0].tolist() == [0, 1, 0]
    assert not filtered(np.full(3, np.nan, np.float32), 1.0, k=1)[0].any()


@pytest.mark.parametrize("seed", range(10))
def test_limits_one_by_one(seed):
    rng = np.random.default_rng(seed)
    row = (rng.standard_normal(200) * 2).astype(np.float32)
    p = probabilities(row, 0.7)
    by = np.argsort(-p)
    k = int(rng.integers(1, 200))
    assert set(np.flatnonzero(filtered(row, 0.7, k=k)[0])) == set(by[:k])
    share = float(rng.uniform(0.05, 0.99))
    n = filtered(row, 0.7, p=share)[1]
    assert np.sum(p[by[:n]]) >= share > np.sum(p[by[:n - 1]])
    m = float(rng.uniform(0.01, 0.9))
    assert set(np.flatnonzero(filtered(row, 0.7, m=m)[0])) == set(np.flatnonzero(p >= m * p.max()))

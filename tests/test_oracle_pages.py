"""Pins of oracle/pages.py: hand-worked lists and what must hold of any."""
import numpy as np
import pytest

from oracle import pages as op


def i32(*x):
    return np.array(x, dtype=np.int32)


def test_hand_worked():
    # pages of 16; request 0 holds page 5 with 10 slots, request 1 nothing.
    table, held, free = i32([5, -1, -1], [-1, -1, -1]), i32(1, 0), i32(3, 1, 4, 0, -1, -1)
    n, slots, missed = op.reserve(i32(10, 0), i32(8, 17), table, held, free, 4, 16, 17)
    # needs 1 and 2: the list's last three, 1 4 0, in request order
    assert n == 1 and missed == 0 and table.tolist() == [[5, 1, -1], [4, 0, -1]] and held.tolist() == [2, 2]
    assert slots[0, :8].tolist() == [90, 91, 92, 93, 94, 95, 16, 17] and (slots[0, 8:] == -1).all()
    assert slots[1].tolist() == list(range(64, 80)) + [0]
    n, bad = op.release(i32(10, 0), table, held, free, n, 16)
    assert n == 4 and bad == 0 and free.tolist() == [3, 1, 4, 0, -1, -1] and table.tolist() == [[5, -1, -1], [-1, -1, -1]]
    assert held.tolist() == [1, 0]


def test_short_list_serves_in_order():
    table, held, free = np.full((4, 4), -1, np.int32), i32(0, 0, 0, 1), i32(7, 8, 9)
    table[3, 0] = 2
    n, slots, missed = op.reserve(i32(0, 0, 0, 3), i32(16, 48, 16, 4), table, held, free, 3, 16, 48, n_pages=10)
    # needs 1, 3, 1, 0: the second does not fit, so neither does the third; the last needs nothing
    assert n == 2 and missed == 2 and table[:, 0].tolist() == [9, -1, -1, 2] and held.tolist() == [1, 0, 0, 1]
    assert slots[3, :4].tolist() == [35, 36, 37, 38] and (slots[1] == -1).all()


def test_refused_requests_and_prefix():
    table, held, free = np.full((5, 3), -1, np.int32), i32(0, 0, 4, 1, 0), i32(6, 5, 4, 0, 0, 0, 0)
    n, slots, missed = op.reserve(i32(-1, 40, 0, 33, 32), i32(1, 9, 1, 1, 0), table, held, free, 3, 16, 8, prefix=(1, 2))
    # negative; n_new past n_pos; holds more than the table; holds 1 of the prefix's 2; needs only the prefix
    assert missed == 3 and n == 2 and table.tolist() == [[-1] * 3, [-1] * 3, [-1] * 3, [-1, 2, 4], [1, 2, -1]]
    assert held.tolist() == [0, 0, 4, 3, 2] and slots[3, 0] == 4 * 16 + 1
    n, bad = op.release(i32(-1, 0, 0, 0, 0), table, held, free, n, 16, n_prefix=2)
    assert n == 3 and bad == 2 and table[3].tolist() == [-1, 2, -1] and held.tolist() == [0, 0, 4, 2, 2]


@pytest.mark.parametrize("seed", range(20))
def test_every_page_in_one_place(seed):
    rng = np.random.default_rng(seed)
    R, P, N, S = int(rng.integers(1, 9)), 12, 40, 16
    table, held, free, n = np.full((R, P), -1, np.int32), np.zeros(R, np.int32), rng.permutation(N).astype(np.int32), N
    lens = np.zeros(R, np.int32)
    for _ in range(30):
        new = rng.integers(0, 40, R).astype(np.int32)
        before = free[:n].tolist()
        n, slots, _ = op.reserve(lens, new, table, held, free, n, S, 40)
        if rng.random() < 0.5:
            n, _ = op.release(lens, table, held, free, n, S)
            assert free[:n].tolist() == before
        else:
            lens = np.where(held * S >= lens + new, lens + new, lens).astype(np.int32)
        if rng.random() < 0.2:
            lens[rng.integers(R)] = 0
            n, _ = op.release(lens, table, held, free, n, S)
        used = [int(p) for r in range(R) for p in table[r, :held[r]]] + free[:n].tolist()
        assert sorted(used) == list(range(N))
        assert all((table[r, held[r]:] == -1).all() and held[r] * S >= lens[r] for r in range(R))

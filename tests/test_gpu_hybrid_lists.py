"""Verify steps with a page list where requests end, wait or start over: one
that runs to its table's last slot, a held one in front of others, one whose
slots do not reach behind the shared prefix."""
import numpy as np
import pytest

from tests.test_gpu_attn import dev, host
from tests.test_gpu_hybrid import refill
from tests.test_gpu_hybrid_pages import P, R, S, WORKLOADS, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_a_request_goes_on_to_its_tables_last_slot(w, graph):
    """As with fixed tables: held where its accepted rows do not fit, not where the span would not."""
    lens = [464, 459, 330, 463]                          # of 30 * 16; in the list the pages of these slots only
    full = np.concatenate([np.tile(np.arange(18), (R, 1)), 19 + np.arange(R * 12).reshape(R, 12)], 1).astype(np.int32)
    held = [-(-n // S) for n in lens]
    x_bufs, xa, x, loaded = make(w, n_pages=70)
    y_bufs, ya, y, _ = make(w, n_pages=70, listed=False)
    ya.page_table.copy_(dev(full))
    table = np.where(np.arange(30) < np.array(held)[:, None], full, -1).astype(np.int32)
    free = np.setdiff1d(np.arange(19, 70), table).astype(np.int32)
    xa.page_table.copy_(dev(table))
    xa.n_held.copy_(dev(np.array(held, np.int32)))
    xa.free_pages[:len(free)] = dev(free)
    xa.n_free.fill_(len(free))
    for a in (xa, ya):
        a.seq_len.copy_(dev(np.array(lens, np.int32)))
    if graph:
        x.capture_graph()
    ended = 0
    for i in range(12):
        refill(x_bufs, xa, i, True, loaded.parent)
        refill(y_bufs, ya, i, True, loaded.parent)
        p, q = x.replay() if graph else x.run(), y.run()
        assert all(np.array_equal(u, v) for u, v in zip(p, q)), (i, p, q)
        assert xa.seq_len.tolist() == ya.seq_len.tolist() and xa.held.tolist() == ya.held.tolist()
        on = [r for r in range(R) if not int(xa.held[r])]
        assert np.array_equal(host(xa.out)[:, on], host(ya.out)[:, on]), i
        assert int(xa.page_status[0, 0]) == 0
        ended = R - len(on)
    assert ended >= 3 and max(xa.seq_len.tolist()) > 464


@pytest.mark.parametrize("graph", [False, True])
def test_a_held_request_takes_no_pages_from_those_behind_it(graph):
    """Pages for exactly the requests that go on, a held one in front of them."""
    w = WORKLOADS[0]
    bufs, a, step, loaded = make(w)
    if graph:
        step.capture_graph()
    go = step.replay if graph else step.run
    a.temperature[0] = float("nan")
    refill(bufs, a, 0, True, loaded.parent)
    acc, _ = go()
    assert acc[0] == -1 and min(acc[1:]) >= 0
    taken = 0
    for i in range(1, 5):
        own = int(a.n_held[0])
        need = sum(max(0, -(-(int(a.seq_len[r]) + w.n_pos) // S) - int(a.n_held[r])) for r in range(1, R))
        a.n_free.fill_(need)                             # (the list below that stays as it is)
        refill(bufs, a, i, True, loaded.parent)
        acc, _ = go()
        assert int(a.page_status[0, 0]) == 0 and int(a.n_held[0]) == own
        assert acc[0] == -1 and min(acc[1:]) >= 0, i
        taken += need
    assert taken > 0 and a.held.tolist() == [1, 0, 0, 0]


@pytest.mark.parametrize("listed", [True, False])
@pytest.mark.parametrize("short", [0, 160, P - 1])
def test_a_request_that_ends_inside_the_prefix_leaves_it_alone(listed, short):
    """Its rows would go into pages that all requests read, or behind slots that are read through the prefix."""
    w = WORKLOADS[0]
    x_bufs, xa, x, loaded = make(w, listed=listed)
    y_bufs, ya, y, _ = make(w, listed=listed)
    if not listed:
        for a in (xa, ya):
            a.page_table.copy_(dev(np.concatenate([np.tile(np.arange(18), (R, 1)), 19 + np.arange(R * 10).reshape(R, 10),
                                                   np.full((R, 2), -1)], 1).astype(np.int32)))
    before = [host(c[:, :19]).copy() for c in (xa.k_cache, xa.v_cache)]
    xa.seq_len[2] = short
    for i in range(3):
        refill(x_bufs, xa, i, True, loaded.parent)
        refill(y_bufs, ya, i, True, loaded.parent)
        p, q = x.run(), y.run()
        assert p[0][2] == p[1][2] == -1 and int(xa.seq_len[2]) == short
        for r in (0, 1, 3):
            assert (p[0][r], p[1][r]) == (q[0][r], q[1][r]), (i, r)
        for c, b in zip((xa.k_cache, xa.v_cache), before):
            assert np.array_equal(host(c[:, :19]), b)


def test_lengths_start_behind_the_prefix():
    w = WORKLOADS[0]
    _, a, _, _ = make(w)
    from hybrid_recurrent_state_amd.step import AttnBuffers
    from synth.device import step_shape
    assert AttnBuffers(a.shape, step_shape(w)).seq_len.tolist() == [P] * R

"""Verify steps with a page list where a request runs to its table's last
slot."""
import numpy as np
import pytest

from tests.test_gpu_attn import dev, host
from tests.test_gpu_hybrid import refill
from tests.test_gpu_hybrid_pages import R, S, WORKLOADS, make

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

"""kv_pages_reserve_step (up to the end of a request's table, without some of
the requests) against the oracle: whole numbers, equal."""
import numpy as np
import pytest

from oracle import pages as op
from tests.test_gpu_attn import dev, host, hrs  # noqa: F401
from tests.test_gpu_pages import SIZES, Lists

pytestmark = pytest.mark.gpu


class Limited(Lists):
    def reserve(self, lens, new, skip=None):
        import torch
        out = torch.full((len(lens), self.n_pos), -5, dtype=torch.int64, device="cuda")
        d = lambda x: None if x is None else dev(np.asarray(x, np.int32))
        self.hrs.kv_pages_reserve_step(d(lens), *self.d, self.ws, page_size=self.S, n_pos=self.n_pos, n_new=d(new),
                                       prefix_table=dev(self.prefix) if self.pre else None, slot_map=out, status=self.status,
                                       skip=d(skip))
        self.n, want, missed = op.reserve(lens, np.full(len(lens), self.n_pos) if new is None else new, self.table, self.held,
                                          self.free, self.n, self.S, self.n_pos, self.prefix, clip=True, skip=skip)
        self.same(missed)
        assert np.array_equal(host(out), want)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "R{}P{}N{}S{}p{}T{}".format(*s))
def test_up_to_the_tables_end(hrs, size):
    R, P, N, S, prefix, n_pos = size
    x = Limited(hrs, R, P, N, S, seed=R + P, prefix=prefix, n_pos=n_pos)
    for step in range(4):
        lens = np.minimum(x.held.astype(np.int64) * S, x.rng.integers(0, P * S + 1, R)).astype(np.int32)
        if step > 1:
            lens = np.where(x.rng.random(R) < 0.2, x.rng.choice([P * S, P * S - 1, P * S + 1, -1], R), lens).astype(np.int32)
        x.reserve(lens, None if step == 1 else x.rng.integers(-1, n_pos + 2, R).astype(np.int32))
        x.release(np.maximum(lens, 0))


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "R{}P{}N{}S{}p{}T{}".format(*s))
def test_without_some_of_the_requests(hrs, size):
    """What they would take is for those behind them; refused ones among them are not counted."""
    R, P, N, S, prefix, n_pos = size
    x = Limited(hrs, R, P, N, S, seed=R + P + 1, prefix=prefix, n_pos=n_pos)
    for step in range(4):
        skip = np.where(x.rng.random(R) < 0.3, x.rng.choice([1, -1, 256, 1 << 31 - 1], R), 0).astype(np.int32)
        lens = np.minimum(x.held.astype(np.int64) * S, x.rng.integers(0, P * S + 1, R)).astype(np.int32)
        lens[x.rng.random(R) < 0.1] = -1
        before = x.held.copy()
        x.reserve(lens, x.rng.integers(0, n_pos + 1, R).astype(np.int32), skip)
        assert np.array_equal(x.held[skip != 0], before[skip != 0])
        x.release(np.maximum(lens, 0))


def test_large_lengths(hrs):
    x = Limited(hrs, 3, 4, 12, 16, seed=2, n_pos=20)
    x.reserve(np.array([2 ** 31 - 1, 63, 50], np.int32), None)
    assert x.held.tolist() == [0, 4, 4] and x.n == 4

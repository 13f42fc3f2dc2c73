"""kv_pages_reserve and kv_pages_release on the GPU against the oracle: whole
numbers, equal."""
import numpy as np
import pytest

from oracle import pages as op
from tests.test_gpu_attn import dev, hrs  # noqa: F401

pytestmark = pytest.mark.gpu


class Lists:
    """Tables, list and lengths on both sides."""

    def __init__(self, hrs, R, P, N, S, seed, prefix=0, n_pos=40, spare=None):
        import torch
        rng = np.random.default_rng(seed)
        self.hrs, self.rng, self.S, self.n_pos, self.pre = hrs, rng, S, n_pos, prefix
        order = rng.permutation(N).astype(np.int32)
        self.prefix = order[:prefix]
        spare = N - prefix if spare is None else spare
        self.free = np.full(N, -1, np.int32)
        self.free[:spare] = order[prefix:prefix + spare]
        self.n = spare
        self.table, self.held = np.full((R, P), -1, np.int32), np.zeros(R, np.int32)
        self.d = [dev(x) for x in (self.table, self.held, self.free, np.array([spare], np.int32))]
        self.ws = torch.full((hrs.kv_pages_workspace_bytes(R),), 0xA5, dtype=torch.uint8, device="cuda")
        self.status = torch.full((4,), -9, dtype=torch.int32, device="cuda")

    def reserve(self, lens, new, n_pos=None, slots=True):
        import torch
        n_pos = self.n_pos if n_pos is None else n_pos
        out = torch.full((len(lens), n_pos), -5, dtype=torch.int64, device="cuda") if slots else None
        n_new = None if new is None else dev(np.asarray(new, np.int32))
        self.hrs.kv_pages_reserve(dev(np.asarray(lens, np.int32)), *self.d, self.ws, page_size=self.S, n_pos=n_pos,
                                  n_new=n_new, prefix_table=dev(self.prefix) if self.pre else None, slot_map=out,
                                  status=self.status)
        self.n, want, missed = op.reserve(lens, np.full(len(lens), n_pos) if new is None else new, self.table, self.held,
                                          self.free, self.n, self.S, n_pos, self.prefix)
        self.same(missed)
        if slots:
            assert np.array_equal(out.cpu().numpy(), want)
        return want

    def release(self, keep):
        self.hrs.kv_pages_release(dev(np.asarray(keep, np.int32)), *self.d, self.ws, page_size=self.S, n_prefix=self.pre,
                                  status=self.status)
        self.n, bad = op.release(keep, self.table, self.held, self.free, self.n, self.S, self.pre)
        self.same(bad)

    def same(self, status):
        table, held, free, n = (x.cpu().numpy() for x in self.d)
        assert np.array_equal(table, self.table) and np.array_equal(held, self.held)
        assert int(n[0]) == self.n and np.array_equal(free, self.free)
        assert self.status.cpu().tolist() == [status, -9, -9, -9]


# R, entries of a table, pages, page size, prefix pages, most new positions: one block, and two launches of either call
SIZES = [(1, 1, 1, 16, 0, 1), (3, 12, 30, 16, 2, 40), (16, 194, 900, 64, 64, 17), (17, 9, 100, 128, 0, 1),
         (300, 5, 700, 32, 1, 64), (1024, 3, 2500, 16, 0, 17), (1025, 4, 3000, 16, 1, 9), (4096, 3, 9000, 16, 0, 2),
         (5, 700, 3000, 16, 0, 9000), (70, 1000, 30000, 16, 5, 700), (2000, 40, 60000, 1024, 3, 33)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "R{}P{}N{}S{}p{}T{}".format(*s))
def test_steps(hrs, size):
    """Steps of requests that grow, are cut back, end and start again, while the list runs short."""
    R, P, N, S, prefix, n_pos = size
    x = Lists(hrs, R, P, N, S, seed=R + P, prefix=prefix, n_pos=n_pos)
    lens = np.full(R, prefix * S, np.int32)
    for step in range(6):
        new = x.rng.integers(0, n_pos + 1, R).astype(np.int32)
        if step == 1:
            new[:] = n_pos
        x.reserve(lens, None if step == 1 else new, slots=step != 2)
        took = np.where(x.held * S >= lens + new, x.rng.integers(0, n_pos + 1, R).clip(0, new), 0)
        lens = (lens + took).astype(np.int32)
        lens[x.rng.random(R) < 0.2] = 0
        x.release(lens)
        lens = np.maximum(lens, prefix * S).astype(np.int32)


def test_refused_requests_stay(hrs):
    x = Lists(hrs, 8, 4, 40, 16, seed=5, n_pos=20, prefix=1)
    x.reserve(np.full(8, 16), np.full(8, 5))
    lens = np.array([-1, 16, 60, 16, 2 ** 31 - 1, 16, 16, 30], np.int32)
    x.held[3], x.held[5] = -2, 5
    x.d[1].copy_(dev(x.held))
    x.reserve(lens, np.array([1, 21, 5, 1, 20, 1, -1, 20], np.int32))
    x.release(np.array([-1, 0, 0, 0, 2 ** 31 - 1, 0, -5, 0], np.int32))


@pytest.mark.parametrize("P", [30, 40000])
def test_entries_that_name_no_page_and_a_full_list(hrs, P):
    x = Lists(hrs, 3, P, 50, 16, seed=P, spare=45)
    x.table[:, :20] = x.rng.integers(-3, 60, (3, 20))
    x.held[:] = (20, 7, 15)
    x.d[0].copy_(dev(x.table))
    x.d[1].copy_(dev(x.held))
    x.release(np.array([0, 0, 33], np.int32))
    assert x.n == 50


@pytest.mark.parametrize("n", [-4, 99])
def test_list_length_out_of_range(hrs, n):
    x = Lists(hrs, 2, 3, 6, 16, seed=1, spare=6)
    x.d[3].fill_(n)
    x.n = max(0, min(6, n))
    x.reserve(np.zeros(2, np.int32), np.array([16, 33], np.int32))


def test_large_numbers(hrs):
    """Slots past 2^31: a page number times the page size needs 64 bits."""
    import torch
    N = 1 << 22
    free = torch.arange(N, dtype=torch.int32, device="cuda")
    n = torch.tensor([N], dtype=torch.int32, device="cuda")
    table, held = torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(1, 2, dtype=torch.int64, device="cuda")
    ws = torch.empty(hrs.kv_pages_workspace_bytes(1), dtype=torch.uint8, device="cuda")
    hrs.kv_pages_reserve(torch.tensor([1023], dtype=torch.int32, device="cuda"), table, held, free, n, ws, page_size=1024,
                         slot_map=out)
    assert out.tolist() == [[(N - 2) * 1024 + 1023, (N - 1) * 1024]] and n.item() == N - 2


def test_captured_steps_carry_on(hrs):
    """Two captured graphs that share a workspace, replayed in turn with eager work between."""
    import torch
    x = Lists(hrs, 16, 20, 200, 16, seed=9, n_pos=17)
    lens = torch.zeros(16, dtype=torch.int32, device="cuda")
    slots = torch.zeros(16, 17, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    grow, cut = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(grow):
        hrs.kv_pages_reserve(lens, *x.d, x.ws, page_size=16, slot_map=slots, status=x.status)
    with torch.cuda.graph(cut):
        hrs.kv_pages_release(lens, *x.d, x.ws, page_size=16, status=x.status)
    now = np.zeros(16, np.int32)
    for _ in range(8):
        grow.replay()
        x.n, want, missed = op.reserve(now, np.full(16, 17), x.table, x.held, x.free, x.n, 16, 17)
        x.same(missed)
        assert np.array_equal(slots.cpu().numpy(), want)
        now = now + x.rng.integers(1, 18, 16).astype(np.int32)
        lens.copy_(dev(now))
        cut.replay()
        x.n, bad = op.release(now, x.table, x.held, x.free, x.n, 16)
        x.same(bad)

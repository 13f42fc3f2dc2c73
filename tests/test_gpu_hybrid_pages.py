"""Verify steps of requests behind a shared prefix whose page tables grow from
a free list and that sample after top-k, top-p and min-p: pages, attention,
acceptance and the appended rows of every step against the oracle on the same
history; replays of the captured step equal eager steps bit for bit; a request
that finds no page is held, and gets one when another one gives its back."""
import numpy as np
import pytest

from oracle import attn as oa
from oracle import pages as op
from oracle import sample as osm
from oracle.filter import filtered
from synth import QWEN_STACK_CHAIN, QWEN_STACK_TREE, scaled
from tests.gpu_util import say
from tests.test_gpu_attn import dev, host
from tests.test_gpu_hybrid import refill
from tests.test_gpu_shared import Shared

pytestmark = pytest.mark.gpu

R = 4
SMALL = dict(n_layers=3, n_req=R, vocab=512, n_kheads=2, n_vheads=4, conv_channels=2 * 2 * 128 + 4 * 128)
WORKLOADS = [scaled(QWEN_STACK_CHAIN, ring_slots=0, ring_width=0, **SMALL), scaled(QWEN_STACK_TREE, **SMALL)]
P, S = 300, 16                       # slots of the prefix (18 pages and 12 slots), slots of a page


def make(w, n_pages=60, f8=False, listed=True, filtered=True, prefix=P):
    import torch
    from hybrid_recurrent_state_amd.step import AttnBuffers, AttnShape, HybridVerifyStep, StepBuffers
    from synth.device import fill_step, step_shape
    bufs = StepBuffers(step_shape(w))
    loaded = fill_step(bufs, w)
    shape = AttnShape(2, 4, 2, 64, 32, n_pages=n_pages, page_size=S, table_len=30, theta=100.0, f8_cache=f8, prefix_len=prefix,
                      page_list=listed)
    a = AttnBuffers(shape, bufs.shape)
    rng = np.random.default_rng(5)
    for c in (a.k_cache, a.v_cache):                   # the prefix's slots, and what pages of the list hold from before
        x = rng.standard_normal(tuple(c.shape)).astype(np.float32) * (50 if f8 else 1)
        c.copy_(torch.from_numpy(x).to(c.dtype))
    if f8:
        a.k_scale.fill_(0.02)
        a.v_scale.fill_(0.015)
    a.seq_len.fill_(prefix)
    a.temperature.copy_(torch.tensor([0.7, 1.3, 1.0, 0.5]))
    a.top_k.copy_(torch.tensor([5, 0, 40, 0]))
    a.top_p.copy_(torch.tensor([1.0, 0.9, 0.8, 1.0]))
    a.min_p.copy_(torch.tensor([0.0, 0.02, 0.01, 0.0]))
    return bufs, a, HybridVerifyStep(bufs, a, parent=loaded.parent, filtered=filtered, sample=filtered), loaded


class Pages:
    """The page list and tables on the oracle's side."""

    def __init__(self, n_pages):
        self.table, self.held = np.full((R, 30), -1, np.int32), np.zeros(R, np.int32)
        self.free = np.concatenate([np.arange(19, n_pages), np.arange(19)]).astype(np.int32)
        self.n = n_pages - 19

    def reserve(self, lens, T):
        self.n, _, missed = op.reserve(lens, [T] * R, self.table, self.held, self.free, self.n, S, T, range(18))
        return missed

    def release(self, lens):
        self.n, _ = op.release(lens, self.table, self.held, self.free, self.n, S, 18)

    def same(self, a):
        assert np.array_equal(host(a.page_table), self.table) and np.array_equal(host(a.n_held), self.held)
        assert int(a.n_free) == self.n and np.array_equal(host(a.free_pages), self.free)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_steps_with_a_prefix_a_page_list_and_limits(w, f8):
    bufs, a, step, loaded = make(w, f8=f8)
    par, T = loaded.parent, w.n_pos
    pages, cache = Pages(60), "f8" if f8 else "bf16"
    for i in range(4):
        refill(bufs, a, i, True, par)
        lens = a.seq_len.tolist()
        before = [host(c).copy() for c in (a.k_cache, a.v_cache)]
        acc, bonus = step.run()
        assert pages.reserve(lens, T) == 0
        tables = pages.table.copy()
        path = host(bufs.path)
        for r in range(R):
            logits = host(bufs.logits)[r]
            rows = [filtered(logits[t], float(a.temperature[r]), int(a.top_k[r]), float(a.top_p[r]), float(a.min_p[r]))[0]
                    for t in range(T)]
            ref = osm.accept_from(np.stack(rows), host(bufs.tokens)[r], host(a.uniforms)[r],
                                  parent=None if par is None else par[r])
            assert np.array_equal(path[r], ref.path) and (int(acc[r]), int(bonus[r])) == (ref.accept_len, ref.bonus), (i, r)
        qh, kh, vh = host(a.q_out), host(a.k_out), host(a.v.contiguous())
        for l in range(2):
            c = Shared(R, T, 4, 2, 64, S, P, lens, "bf16", cache)
            c.q, c.k, c.v, c.kc, c.vc = qh[l], kh[l], vh[l], before[0][l], before[1][l]
            c.N, c.ptable, c.pages, c.parent = 60, np.arange(19, dtype=np.int32), tables, par
            c.ks, c.vs = (host(s)[l] if f8 else None for s in (a.k_scale, a.v_scale))
            c.check(a.out[l], what=f"step {i}")
            for r in range(R):
                for rows, b, s in ((kh, before[0], c.ks), (vh, before[1], c.vs)):
                    src = oa.quantize_e4m3(oa.widen(rows[l, r]), s) if f8 else rows[l, r]
                    oa.append(src, b[l], tables[r], lens[r], path[r], int(acc[r]) + 1)
        for c, b in zip((a.k_cache, a.v_cache), before):
            assert np.array_equal(host(c), b)
        lens = [n + int(x) + 1 for n, x in zip(lens, acc)]
        assert a.seq_len.tolist() == lens
        pages.release(lens)
        pages.same(a)
        assert int(a.status[:, 0].abs().sum()) == 0 and int(a.page_status[:, 0].abs().sum()) == 0
        say(f"step {i}: accepted {list(map(int, acc))}, {pages.n} pages left")


@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_graph_replays(w):
    import torch
    e_bufs, ea, eager, _ = make(w)
    g_bufs, ga, graphed, loaded = make(w)
    graphed.capture_graph()
    for i in range(5):
        refill(e_bufs, ea, i, True, loaded.parent)
        refill(g_bufs, ga, i, True, loaded.parent)
        assert all(np.array_equal(x, y) for x, y in zip(eager.run(), graphed.replay())), i
        for x, y in ((e_bufs.path, g_bufs.path), (e_bufs.out, g_bufs.out), (ea.out, ga.out), (ea.k_cache, ga.k_cache),
                     (ea.v_cache, ga.v_cache), (ea.seq_len, ga.seq_len), (ea.page_table, ga.page_table),
                     (ea.free_pages, ga.free_pages), (ea.n_free, ga.n_free), (ea.n_held, ga.n_held)):
            assert np.array_equal(host(x), host(y)), i
        torch.cuda.synchronize()


def test_a_page_list_gives_what_full_tables_give():
    """The same model with fixed tables of its own: results do not depend on which pages a request gets."""
    w = WORKLOADS[0]
    x_bufs, xa, x, loaded = make(w)
    y_bufs, ya, y, _ = make(w, listed=False)
    ya.page_table.copy_(dev(np.concatenate([np.tile(np.arange(18), (R, 1)), 19 + np.arange(R * 12).reshape(R, 12)], 1)
                            .astype(np.int32)))
    for i in range(4):
        refill(x_bufs, xa, i, True, loaded.parent)
        refill(y_bufs, ya, i, True, loaded.parent)
        assert all(np.array_equal(p, q) for p, q in zip(x.run(), y.run())), i
        assert np.array_equal(host(xa.out), host(ya.out)), i


@pytest.mark.parametrize("graph", [False, True])
def test_a_request_without_pages_is_held_and_others_go_on(graph):
    """A list for two requests' spans: the others are held as accept_hold does it once their accepted rows have no page,
    those two go on; a request that ends gives its pages back."""
    import torch
    import hybrid_recurrent_state_amd as hrs
    w = WORKLOADS[0]
    bufs, a, step, loaded = make(w, n_pages=19 + 5)     # 300 + 17 slots: two pages each
    if graph:
        step.capture_graph()
    go = step.replay if graph else step.run
    refill(bufs, a, 0, True, loaded.parent)
    acc, bonus = go()
    assert int(a.page_status[0, 0]) == 2 and acc[2:].tolist() == bonus[2:].tolist() == [-1, -1] and min(acc[:2]) >= 0
    assert a.seq_len.tolist()[2:] == [P, P] and a.n_held.tolist()[2:] == [18, 18] and a.held.tolist() == [0, 0, 1, 1]
    left = int(a.n_free)
    ended = torch.tensor([0] + [2 ** 31 - 1] * 3, dtype=torch.int32, device="cuda")
    hrs.kv_pages_release(ended, a.page_table, a.n_held, a.free_pages, a.n_free, a.workspace, page_size=S, n_prefix=18)
    assert int(a.n_free) > left and int(a.n_held[0]) == 18
    a.seq_len[0] = P                                    # another request starts behind the prefix in its place
    refill(bufs, a, 1, True, loaded.parent)
    acc, _ = go()
    assert acc[2:].tolist() == [-1, -1] and min(acc[:2]) >= 0       # held until a new speculation


def test_plain_step_behind_a_prefix():
    """Greedy acceptance, fixed tables and a prefix of whole pages: as the same slots in every request's own table."""
    w = WORKLOADS[1]
    x_bufs, xa, x, loaded = make(w, listed=False, filtered=False, prefix=288)
    y_bufs, ya, y, _ = make(w, listed=False, filtered=False, prefix=0)
    table = np.concatenate([np.tile(np.arange(18), (R, 1)), 19 + np.arange(R * 12).reshape(R, 12)], 1).astype(np.int32)
    for a in (xa, ya):
        a.page_table.copy_(dev(table))
        a.seq_len.fill_(288)
    for i in range(2):
        refill(x_bufs, xa, i, False, loaded.parent)
        refill(y_bufs, ya, i, False, loaded.parent)
        assert all(np.array_equal(p, q) for p, q in zip(x.run(), y.run())), i
        p, q = xa.out.float(), ya.out.float()
        assert float((p - q).abs().max()) <= 2.0 ** -7 * float(q.abs().max())

"""Verify steps of a hybrid model in which a request cannot go on: its pages
are full or missing, or its temperature is no temperature. It is reported, stays as it was in
front of the step in every part of its state (recurrent, conv, pages, length),
is passed over by later steps, and the others are not touched by any of it."""
import numpy as np
import pytest

from tests.gpu_util import say
from tests.test_gpu_attn import host
from tests.test_gpu_hybrid import WORKLOADS, make, refill

pytestmark = pytest.mark.gpu


def spoil(a, kind, r):
    """Request r cannot go on from here; what takes it back."""
    if kind == "temperature":
        old = float(a.temperature[r])
        a.temperature[r] = -1.0 if r else float("nan")
        return lambda: a.temperature.__setitem__(r, old)
    if kind == "full":
        old = int(a.seq_len[r])
        a.seq_len[r] = 5 * 32                                      # five pages of 32 slots
        return lambda: a.seq_len.__setitem__(r, old)
    old = a.page_table[r].clone()
    at = int(a.seq_len[r]) // 32
    a.page_table[r, at:] = -1 if r else 12                         # 12 pages: 0 to 11
    return lambda: a.page_table.__setitem__(r, old)


def parts(bufs, a, r):
    return [host(t).copy() for t in (bufs.conv_state[:, r], a.seq_len[r])] + [
        host(c[:, a.page_table[r].long().clamp(0, 11)]).copy() for c in (a.k_cache, a.v_cache)]


@pytest.mark.parametrize("R,T,S,P", [(1, 1, 16, 1), (7, 17, 16, 5), (300, 64, 32, 4)])
@pytest.mark.parametrize("temp,source", [(True, True), (False, False), (False, True)])
def test_accept_hold(R, T, S, P, temp, source):
    """Every reason to hold a request beside requests that go on."""
    import torch
    import hybrid_recurrent_state_amd as hrs
    rng = np.random.default_rng(R + T)
    N = R * P
    pages = rng.permutation(N).reshape(R, P).astype(np.int32)
    n = rng.integers(0, T, R).astype(np.int32)
    lens = rng.integers(0, np.maximum(P * S - n, 1)).astype(np.int32)
    lens[n + 1 + lens > P * S] = 0
    path = np.full((R, T), -1, dtype=np.int32)
    for r in range(R):
        path[r, :n[r] + 1] = np.sort(rng.permutation(T)[:n[r] + 1])
    node = path[np.arange(R), n]
    tau, held = rng.uniform(0, 2, R).astype(np.float32), np.zeros(R, dtype=np.int32)
    bonus, last, at = (rng.integers(0, 99, R).astype(np.int32) for _ in range(3))
    for r in range(R):
        kind = rng.integers(0, 16)
        if kind == 0: n[r] = rng.choice([-1, T, 2 ** 31 - 1, -2 ** 31])
        elif kind == 1: node[r] = rng.choice([-1, T])
        elif kind == 2: path[r, n[r]] = rng.choice([-1, T])
        elif kind == 3: lens[r] = rng.choice([-1, P * S - n[r], 2 ** 31 - 1])
        elif kind == 4: pages[r, (lens[r] + n[r]) // S] = rng.choice([-1, N, -2 ** 31])
        elif kind == 5: pages[r, lens[r] // S] = rng.choice([-1, N])
        elif kind == 6: tau[r] = rng.choice([-1.0, np.nan, -np.inf])
        elif kind == 7: held[r] = 1
        elif kind == 8 and (lens[r] + n[r]) // S + 1 < P: pages[r, (lens[r] + n[r]) // S + 1:] = -1      # not needed yet
        elif kind == 9: tau[r] = rng.choice([0.0, np.inf])
        elif kind == 10: lens[r] = P * S - n[r] - 1                                                      # just fits
    ok = [held[r] == 0 and 0 <= n[r] < T and 0 <= node[r] < T and (not temp or tau[r] >= 0) and lens[r] >= 0
          and int(lens[r]) + int(n[r]) + 1 <= P * S
          and all(0 <= path[r, i] < T and 0 <= pages[r, (lens[r] + i) // S] < N for i in range(n[r] + 1)) for r in range(R)]
    dev = lambda x: torch.from_numpy(x.copy()).cuda()
    d = dict(accept_node=dev(node), accept_len=dev(n), path=dev(path), bonus=dev(bonus), held=dev(held), last_node=dev(last))
    at_dev = dev(at)
    hrs.accept_hold(dev(pages), dev(lens), *d.values(), N, S, held_node=at_dev if source else None,
                    temperature=dev(tau) if temp else None)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy() for k, v in d.items()}
    for r in range(R):
        assert got["held"][r] == (0 if ok[r] else 1), r
        assert np.array_equal(got["path"][r], path[r] if ok[r] else np.full(T, -1)), r
        for k, x in (("accept_node", node), ("accept_len", n), ("bonus", bonus)):
            assert got[k][r] == (x[r] if ok[r] else -1), (k, r)
        assert got["last_node"][r] == (node[r] if ok[r] else last[r]), r
        assert int(at_dev[r]) == (last[r] if source and not ok[r] and not held[r] else at[r]), r
    say(f"  {sum(ok)} of {R} go on")


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kind,sample", [("temperature", True), ("full", True), ("full", False), ("missing", False),
                                         ("missing", True)])
@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_a_request_that_cannot_go_on_is_held(w, at, kind, sample, graph):
    """Beside an undisturbed run of the same steps: request r stops in front
    of step `at`."""
    import torch
    r = at % 2
    o = 1 - r
    bufs, a, step, loaded = make(w, sample)
    ref_bufs, ra, ref, _ = make(w, sample)
    if graph:
        step.capture_graph()
        ref.capture_graph()
    go = lambda s: s.replay() if graph else s.run()
    bufs.accept_len.fill_(2)                     # what memory may hold in front of the first step
    bufs.path.fill_(0)
    for i in range(at):
        refill(bufs, a, i, sample, loaded.parent)
        refill(ref_bufs, ra, i, sample, loaded.parent)
        assert all(np.array_equal(x, y) for x, y in zip(go(step), go(ref)))
    # the state of request r in front of step `at`, from a copy of the run so far
    ref.materialize() if at else None
    want_state = host(ref_bufs.state[:, r]).copy()
    undo = spoil(a, kind, r)
    before = parts(bufs, a, r)
    for i in range(at, at + 3):
        refill(bufs, a, i, sample, loaded.parent)
        refill(ref_bufs, ra, i, sample, loaded.parent)
        n_acc, bonus = go(step)
        n_ref, b_ref = go(ref)
        say(f"step {i}: accepted {n_acc.tolist()} beside {n_ref.tolist()}")
        assert (n_acc[r], bonus[r]) == (-1, -1)
        assert (n_acc[o], bonus[o]) == (n_ref[o], b_ref[o])
        assert int(bufs.accept_node[r]) == -1 and bool((bufs.path[r] == -1).all())
        for x, y in zip(parts(bufs, a, r), before):
            assert np.array_equal(x, y)
        for x, y in ((bufs.out[:, o], ref_bufs.out[:, o]), (a.out[:, o], ra.out[:, o]), (a.seq_len[o], ra.seq_len[o]),
                     (bufs.conv_state[:, o], ref_bufs.conv_state[:, o]), (bufs.path[o], ref_bufs.path[o])):
            assert np.array_equal(host(x), host(y)), i
        undo()                                   # held until a new speculation all the same
        before = parts(bufs, a, r) if i == at else before
    # the canonical state: the other's after its last accepted position, this one's from in front of step `at`
    step.materialize()
    ref.materialize()
    torch.cuda.synchronize()
    assert np.array_equal(host(bufs.state[:, r]), want_state)
    assert np.array_equal(host(bufs.state[:, o]), host(ref_bufs.state[:, o]))


@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_a_held_request_goes_on_in_a_new_speculation(w):
    """Pages given, a new step object from the canonical states: both requests
    go on as in a run that was never held."""
    from hybrid_recurrent_state_amd.step import HybridVerifyStep
    bufs, a, step, loaded = make(w, False)
    ref_bufs, ra, ref, _ = make(w, False)
    for s, b, x in ((step, bufs, a), (ref, ref_bufs, ra)):
        refill(b, x, 0, False, loaded.parent)
        s.run()
    undo = spoil(a, "missing", 1)
    refill(bufs, a, 1, False, loaded.parent)
    n_acc, _ = step.run()
    assert n_acc[1] == -1 and n_acc[0] >= 0
    undo()
    step.materialize()
    ref.materialize()
    assert np.array_equal(host(bufs.state[:, 1]), host(ref_bufs.state[:, 1]))
    again = HybridVerifyStep(bufs, a, parent=loaded.parent)
    ref2 = HybridVerifyStep(ref_bufs, ra, parent=loaded.parent)
    refill(bufs, a, 2, False, loaded.parent)
    refill(ref_bufs, ra, 2, False, loaded.parent)
    x, y = again.run(), ref2.run()
    assert (x[0][1], x[1][1]) == (y[0][1], y[1][1]) and x[0][1] >= 0
    assert np.array_equal(host(bufs.out[:, 1]), host(ref_bufs.out[:, 1]))
    assert np.array_equal(host(a.out[:, 1]), host(ra.out[:, 1]))

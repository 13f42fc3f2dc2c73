"""accept_sample_filtered on the GPU against the float64 oracle.

Whole numbers must be equal: the oracle reports how far acceptance and draw are
from their borders (as in test_gpu_sample.py), and inputs that are too near fail
the test by themselves. A top-p whose border lies within what the sums are off
by (below: 18 u of a row's weights) may fall on either side of it: the results
have to be those of one side.
token_prob: a weight in 64 bits over a sum; rows that are settled by a list have
that in 64 bits too, the others sum weights good to 2 ulp of the exponential and
one of the factor beside it (3 u, u = 2^-24; 2^-44 of the largest each for
being whole numbers, over V of them) or, without limits, add up to 64 of them in
float32 (eight, then eight sums: 15 u); every result is rounded once: 19 u + V
2^-43 bounds all of it.
"""
import itertools

import numpy as np
import pytest

from oracle import sample as osm
from oracle.common import widen
from oracle.filter import filtered
from tests.test_gpu_attn import dev, host, hrs  # noqa: F401
from tests.test_gpu_sample import Block, cast

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Filtered(Block):
    """A block of drafts with limits per request; drafts that were picked are likely ones."""

    def __init__(self, R, T, V, dtype="bf16", tree=False, draft=None, temp=True, spread=2.5, seed=0, k=None, p=None, m=None,
                 head=0):
        super().__init__(R, T, V, dtype, tree, draft, temp, spread, seed)
        self.k = None if k is None else np.resize(np.array(k, np.int32), R)
        self.p = None if p is None else np.resize(np.array(p, np.float32), R)
        self.m = None if m is None else np.resize(np.array(m, np.float32), R)
        if head:
            rng = np.random.default_rng(seed + 99)
            z = widen(self.logits).astype(np.float32)
            at = np.argsort(rng.random((R, T, V)), -1)[..., :head]
            np.put_along_axis(z, at, (12 + 2.5 * rng.standard_normal((R, T, head))).astype(np.float32), -1)
            self.logits = cast(z, dtype)
            for r in range(R):
                for t in range(1, T):
                    par = t - 1 if self.parent is None else self.parent[r, t]
                    self.tokens[r, t] = at[r, par, rng.integers(head)]

    def limit(self, r):
        return (0 if self.k is None else int(self.k[r]), 1.0 if self.p is None else float(self.p[r]),
                0.0 if self.m is None else float(self.m[r]))

    def run(self, hrs, status=None, ws=None):
        import torch
        R, T, V = self.logits.shape
        n = hrs.accept_sample_filtered_workspace_bytes(R, T, V)
        assert n > 0
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        d = lambda x: None if x is None else dev(x)
        hrs.accept_sample_filtered(*self.args(), ws, top_k=d(self.k), top_p=d(self.p), min_p=d(self.m),
                                   draft_probs=d(self.draft), temperature=d(self.temp), parent=self.parent, status=status)
        return [host(x) for x in self.outs]

    def check(self, got, requests=None, what="", margins=True):
        prob, node, length, path, bonus = got
        R, T, V = self.logits.shape
        for r in range(R) if requests is None else requests:
            tau = 1.0 if self.temp is None else float(self.temp[r])
            k, p, m = self.limit(r)
            sides = []
            for t in range(T):
                row = {}
                for q in (p, p - 18 * U, p + 18 * U) if 0 < p < 1 else (p,):
                    x, n = filtered(self.logits[r, t], tau, k, q, m)
                    row.setdefault(n, x)
                sides.append(list(row.values()))
            wrong = []
            for rows in itertools.product(*sides):
                ref = osm.accept_from(np.stack(rows), self.tokens[r], self.u[r], None if self.draft is None else self.draft[r],
                                      None if self.parent is None else self.parent[r])
                if margins:
                    assert ref.accept_margin > 2e-5 and ref.bonus_margin > 1e-9, (what, r, ref.accept_margin, ref.bonus_margin)
                tol = (19 * U + V * 2.0 ** -43) * ref.token_prob + 2.0 ** -126
                same = ((int(node[r]), int(length[r]), int(bonus[r])) == (ref.accept_node, ref.accept_len, ref.bonus) and
                        np.array_equal(path[r], ref.path) and bool(np.all(np.abs(prob[r] - ref.token_prob) <= tol)))
                if same:
                    break
                wrong.append((ref, prob[r], node[r], length[r], path[r], bonus[r]))
            else:
                raise AssertionError((what, r, wrong[0]))


LIMITS = dict(k=dict(k=20), k1=dict(k=1), k64=dict(k=64), k65=dict(k=65), k400=dict(k=400), p=dict(p=0.8), p0=dict(p=0.0),
              m=dict(m=0.05), all=dict(k=50, p=0.9, m=0.02), large=dict(k=3000, p=0.97),
              mixed=dict(k=[0, 7, 0, 300], p=[0.9, 1.0, 1.0, 0.5], m=[0.0, 0.0, 0.1, 0.001]), none=dict(),
              off=dict(k=[0, -5, 10 ** 9], p=[1.0, np.nan, 7.0], m=[0.0, -1.0, np.nan]))
SHAPES = [(1, 1, 8, "f32", False, None, 0), (1, 1, 8, "bf16", False, "f32", 0), (4, 5, 264, "bf16", False, "f32", 0),
          (4, 9, 1000, "f32", True, None, 0), (3, 4, 8200, "bf16", False, "bf16", 30), (4, 3, 16392, "f32", False, None, 40),
          (2, 3, 32768, "bf16", True, None, 0), (1, 3, 151936, "bf16", False, "f32", 40), (1, 2, 151936, "f32", False, None, 0)]


@pytest.mark.parametrize("limits", LIMITS, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: f"R{c[0]}T{c[1]}V{c[2]}{c[3]}{'t' if c[4] else ''}{c[5] or ''}h{c[6]}")
def test_filtered_vs_oracle(hrs, shape, limits):
    R, T, V, dt, tree, draft, head = shape
    b = Filtered(R, T, V, dt, tree, draft, head=head, **LIMITS[limits])
    b.check(b.run(hrs), what=limits)


def test_without_limits_as_accept_sample(hrs):
    b = Filtered(5, 17, 5000, "bf16", draft="f32")
    got, plain = b.run(hrs), Block.run(b, hrs)
    assert all(np.array_equal(x, y) for x, y in zip(got[1:], plain[1:]))
    assert np.allclose(got[0], plain[0], rtol=64 * U, atol=0)


def test_many_requests_over_several_launches(hrs):
    b = Filtered(130, 30, 64, "bf16", tree=True, k=[5, 0], p=[0.9, 0.7, 1.0], m=[0.0, 0.01])
    b.check(b.run(hrs), what="130 trees")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [0.0, -3.0e38, 5.5])
def test_rows_of_ties(hrs, dtype, value):
    """Everything equal, or all but a few: ties go by index, in lists and in rows that no list holds."""
    V = 20000
    b = Filtered(8, 1, V, dtype, temp=False, k=[3, 100, 700, 0, 0, 9000, 2, 0], p=[1, 1, 1, 0.25, 1, 0.5, 0.4, 0.999],
                 m=[0, 0, 0, 0, 0.5, 0, 0, 0])
    z = np.full((8, 1, V), value, np.float32)
    z[4:, 0, 777:V:1000] = 7.0
    b.logits = cast(z, dtype)
    b.u[:, 0] = [0.5, 0.995, 0.3, 0.77, 0.21, 0.63, 0.9, 0.02]
    b.check(b.run(hrs), what="ties", margins=False)


def test_masked_vocabularies(hrs):
    """All but a few tokens at the type's lowest value or -inf, as a grammar leaves them."""
    V = 40000
    b = Filtered(6, 2, V, "bf16", temp=True, k=[20, 0, 100, 20, 0, 0], p=[0.9, 0.9, 1.0, 0.9, 0.5, 1.0], m=[0, 0, 0, 0, 0, 0.01])
    z = widen(b.logits).astype(np.float32)
    on = np.zeros(V, bool)
    on[[5, 17000, 17001, 30000, 39999]] = True
    z[:3, :, ~on] = -3.3895314e38
    z[3:, :, ~on] = -np.inf
    b.logits = cast(z, "bf16")
    b.tokens[:, 1] = 17001
    b.check(b.run(hrs), what="masked", margins=False)


def test_special_rows(hrs):
    f = np.float32
    V = 24
    b = Filtered(9, 3, V, "f32", tree=True, k=[2, 5, 3, 3, 1, 4, 4, 0, 6], p=[1, 0.7, 0.5, 0.5, 1, 0.9, 0.5, 0.6, 0.9],
                 m=[0, 0, 0.1, 0.1, 0, 0, 0, 0.5, 0])
    b.parent = np.tile(np.array([-1, 0, 0], dtype=np.int32), (9, 1))
    b.temp = np.array([0, np.inf, 1, 1, 1, 1, 1e-30, 1, 1e30], dtype=f)
    b.logits[0, 0, [3, 9, 11]] = 50
    b.tokens[0] = [0, 9, 11]
    b.logits[1, 0, 5] = -np.inf
    b.logits[2, 0, :] = np.nan
    b.logits[3, 0, :] = -np.inf
    b.logits[4, 0, [2, 20]] = np.inf
    b.logits[5, 0, ::2] = np.nan
    b.tokens[5] = [0, -1, V]
    b.tokens[6] = [0, 4, 4]
    b.tokens[7] = [0, int(np.argmin(b.logits[7, 0])), int(np.argmin(b.logits[7, 0]))]
    b.u[:, 1:] = [0.9, 0.95]
    b.check(b.run(hrs), what="special rows", margins=False)


@pytest.mark.parametrize("V", [4096, 30000])
def test_signalling_nan_and_signed_zeros(hrs, V):
    b = Filtered(2, 1, V, "bf16", temp=False, k=[40, 600])
    b.logits[:, 0, ::3] = 0x7F81          # NaN with its top mantissa bit clear
    b.logits[:, 0, 1::3] = 0x8000
    b.logits[:, 0, 2::3] = 0x0000
    b.logits[:, 0, 5] = 0x3F80
    b.u[:, 0] = [0.99, 0.9995]
    b.check(b.run(hrs), what="zeros", margins=False)


def test_bad_temperatures_are_left_alone_and_counted(hrs):
    import torch
    b = Filtered(4, 3, 64, "bf16", k=5)
    b.temp = np.array([1, -1, np.nan, 0.5], dtype=np.float32)
    status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    got = b.run(hrs, status=status)
    assert status.tolist() == [2, 9, 9, 9]
    for x in got:
        assert np.all(x[1:3] == -7)
    b.check(got, requests=[0, 3], what="beside bad temperatures")


def test_a_rejected_token_that_was_all_there_was(hrs):
    """top-k 1 leaves one token; rejected all the same (u = 1), the rest is empty and the row itself is drawn from."""
    for V in (64, 20000):
        b = Filtered(2, 2, V, "f32", temp=False, k=[1, 0], p=[1.0, 1e-6])
        b.tokens[:, 1] = np.argmax(b.logits[:, 0], -1)
        b.u[:] = [0.5, 1.0]
        got = b.run(hrs)
        assert got[2].tolist() == [0, 0] and got[4].tolist() == b.tokens[:, 1].tolist()


def test_spread_of_draws(hrs):
    V, R = 64, 4096
    row = (np.random.default_rng(0).standard_normal(V) * 2).astype(np.float32)
    b = Filtered(1, 1, V, "f32", temp=False)
    b.logits = np.ascontiguousarray(np.broadcast_to(row, (R, 1, V)))
    b.tokens = np.zeros((R, 1), dtype=np.int32)
    b.u = (((np.arange(R) + 0.5) / R).astype(np.float32))[:, None].copy()
    b.k, b.p = np.full(R, 20, np.int32), np.full(R, 0.9, np.float32)
    count = np.bincount(b.run(hrs)[4], minlength=V)
    assert np.all(np.abs(count - R * filtered(row, 1.0, 20, 0.9)[0]) <= 1.001)


@pytest.mark.parametrize("head", [0, 40])
def test_repeat_guard_and_graph(hrs, head):
    import torch
    make = lambda seed: Filtered(3, 17, 8200, "bf16", draft="f32", seed=seed, k=[20, 0, 900], p=[0.95, 0.9, 1.0], head=head)
    b = make(0)
    first = b.run(hrs)
    n = hrs.accept_sample_filtered_workspace_bytes(3, 17, 8200)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    again = b.run(hrs, ws=ws[256:-256])
    assert all(np.array_equal(x, y) for x, y in zip(first, again))
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[-256:] == 0xA5).all())
    a = b.args()
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    dq, tau, k, p = dev(b.draft), dev(b.temp), dev(b.k), dev(b.p)
    call = hrs.accept_sample_filtered_call(*a, work, top_k=k, top_p=p, draft_probs=dq, temperature=tau)
    outs = b.outs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2, 3):
        c = make(seed)
        for t, x in zip(a[:3], (c.logits, c.tokens, c.u)):
            t.copy_(dev(x))
        dq.copy_(dev(c.draft))
        tau.copy_(dev(c.temp))
        graph.replay()
        torch.cuda.synchronize()
        got = [host(x) for x in outs]
        eager = c.run(hrs)
        assert all(np.array_equal(x, y) for x, y in zip(got, eager))
        c.check(got, what=f"replay {seed}")


def test_even_rows_of_many_requests_on_two_streams(hrs):
    """Rows without a list, whose last block draws: many requests, two calls at once, every call as when alone."""
    import torch
    cases = [Filtered(40, 3, 30000, "bf16", draft="f32", seed=1, p=[0.9, 0.6]),
             Filtered(300, 1, 16392, "f32", seed=2, k=[0, 3000], p=[0.95])]
    want = [c.run(hrs) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    calls, keep = [], []
    for c in cases:
        a = c.args()
        ws = torch.full((hrs.accept_sample_filtered_workspace_bytes(*c.logits.shape),), 0xFF, dtype=torch.uint8, device="cuda")
        d = lambda x: None if x is None else dev(x)
        more = dict(top_k=d(c.k), top_p=d(c.p), draft_probs=d(c.draft), temperature=d(c.temp))
        calls.append(hrs.accept_sample_filtered_call(*a, ws, **more))
        keep.append((a, ws, more))
    for _ in range(4):
        for c in cases:
            for o in c.outs:
                o.fill_(-7)
        torch.cuda.synchronize()
        for call, st in zip(calls, streams):
            call(st)
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert all(np.array_equal(host(x), y) for x, y in zip(c.outs, w))

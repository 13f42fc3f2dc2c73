"""accept_sample on the GPU against the float64 oracle.

Whole numbers must be equal. That a decision is not a matter of rounding is a
property of the inputs, which the oracle reports: every acceptance decision
is at least 2e-5 (relative) from its border and every drawn token's borders at
least 1e-9 of the total away, or the test says so and fails for its inputs.
token_prob: e^x in float32 with |x| = |z - m| / tau: the argument's rounding
(2 u |x|), the exponential (2 u), and as much again for the row's sum, whose
terms carry their own |x| (weighted by p, so at most max|x| over the terms
that matter: bounded here by sum p |x|), one rounding of the result.
"""
import numpy as np
import pytest

from oracle import sample as osm
from oracle.common import widen
from synth import bf16_bits
from tests.test_gpu_attn import dev, host, random_tree
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def hrs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import hybrid_recurrent_state_amd as m
    return m


def cast(x, dtype):
    x = np.ascontiguousarray(x, dtype=np.float32)
    return x if dtype == "f32" else bf16_bits(x)


class Block:
    def __init__(self, R, T, V, dtype="bf16", tree=False, draft=None, temp=True, spread=2.5, seed=0):
        rng = np.random.default_rng(seed + R * 7 + T * 3 + V)
        z = rng.standard_normal((R, T, V)) * spread
        self.logits = cast(z, dtype)
        self.temp = rng.uniform(0.5, 1.5, R).astype(np.float32) if temp else None
        tau = self.temp if temp else np.ones(R)
        self.u = rng.random((R, T), dtype=np.float32)
        self.tokens = np.zeros((R, T), dtype=np.int32)
        self.draft = None
        self.parent = np.stack([random_tree(rng, T) for _ in range(R)]) if tree else None
        if draft:
            y = z / tau[:, None, None] + 0.4 * rng.standard_normal((R, T, V))
            q = np.exp(y - y.max(-1, keepdims=True))
            q /= q.sum(-1, keepdims=True)
            self.draft = cast(q, draft)
            for r in range(R):
                for t in range(1, T):
                    self.tokens[r, t] = osm.draw(widen(self.draft[r, t - 1]), rng.random())[0]
        else:
            for r in range(R):
                for t in range(1, T):
                    p = t - 1 if self.parent is None else self.parent[r, t]
                    top = np.argsort(-(z[r, p] / tau[r] + rng.gumbel(size=V)))
                    self.tokens[r, t] = top[0]

    def args(self):
        import torch
        R, T, V = self.logits.shape
        e = lambda *s, d=torch.int32, f=-7: torch.full(s, f, dtype=d, device="cuda")
        self.outs = [e(R, T, d=torch.float32), e(R), e(R), e(R, T), e(R)]
        return (dev(self.logits), dev(self.tokens), dev(self.u), *self.outs)

    def run(self, hrs, status=None, ws=None):
        import torch
        R, T, V = self.logits.shape
        n = hrs.accept_sample_workspace_bytes(R, T, V)
        assert n > 0
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        a = self.args()
        hrs.accept_sample(*a, ws, draft_probs=None if self.draft is None else dev(self.draft),
                          temperature=None if self.temp is None else dev(self.temp), parent=self.parent, status=status)
        return [host(x) for x in self.outs]

    def check(self, got, requests=None, what="", margins=True):
        prob, node, length, path, bonus = got
        R, T, V = self.logits.shape
        kept = 0
        for r in range(R) if requests is None else requests:
            tau = 1.0 if self.temp is None else float(self.temp[r])
            ref = osm.accept(self.logits[r], self.tokens[r], self.u[r], None if self.draft is None else self.draft[r], tau,
                             None if self.parent is None else self.parent[r])
            if margins:
                assert ref.accept_margin > 2e-5 and ref.bonus_margin > 1e-9, (what, r, ref.accept_margin, ref.bonus_margin)
            assert (int(node[r]), int(length[r])) == (ref.accept_node, ref.accept_len), (what, r)
            assert np.array_equal(path[r], ref.path), (what, r)
            assert int(bonus[r]) == ref.bonus, (what, r)
            kept += ref.accept_len
            for t in range(T):
                p = t - 1 if self.parent is None else int(self.parent[r, t])
                tol = U          # p = 1 / n at the limits of the temperature: the result's own rounding
                if t > 0 and 0 <= self.tokens[r, t] < V and 0 < tau < np.inf:
                    z = widen(self.logits[r, p])
                    ok = np.isfinite(z)
                    x = np.abs(z[ok] - (z[ok].max() if ok.any() else 0)) / tau
                    pr = osm.probabilities(self.logits[r, p], tau)[ok]
                    own = abs(z[self.tokens[r, t]] - z[ok].max()) / tau if ok[self.tokens[r, t]] else 0.0
                    tol = (4 * own + 4 * float(np.sum(pr * x)) + 8) * U
                assert abs(prob[r, t] - ref.token_prob[t]) <= tol * ref.token_prob[t] + 2.0 ** -126, (what, r, t)
        say(f"  sample {what} {self.logits.shape}: {kept} drafts kept")


CASES = [
    # R, T, V, dtype, tree, draft, temp
    (1, 1, 8, "f32", False, None, False), (1, 1, 8, "bf16", False, "f32", True), (2, 2, 16, "bf16", False, "bf16", True),
    (3, 17, 1000, "bf16", False, "f32", True), (2, 9, 1024, "f32", False, "bf16", True), (4, 23, 4104, "bf16", True, None, True),
    (3, 64, 520, "f32", True, None, True), (2, 64, 264, "bf16", False, "f32", False), (2, 5, 16384, "bf16", False, "f32", True),
    (1, 4, 16392, "f32", False, "f32", True), (1, 3, 151936, "bf16", False, "f32", True), (2, 17, 32768, "f32", True, None, True),
    (5, 6, 40, "f32", False, None, True), (1, 3, 2048, "bf16", False, "bf16", True), (1, 4, 4096, "bf16", True, None, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"R{c[0]}T{c[1]}V{c[2]}{c[3]}{'t' if c[4] else ''}{c[5] or ''}")
def test_sample_vs_oracle(hrs, case):
    R, T, V, dt, tree, draft, temp = case
    b = Block(R, T, V, dt, tree, draft, temp)
    b.check(b.run(hrs), what="grid")


def test_sample_many_requests_over_several_launches(hrs):
    b = Block(130, 30, 64, "bf16", tree=True)
    b.check(b.run(hrs), what="130 trees")


@pytest.mark.parametrize("draft", [None, "f32"])
def test_sample_everything_accepted_and_nothing_accepted(hrs, draft):
    b = Block(2, 9, 512, "f32", draft=draft)
    b.u[0, 1:] = 0.0
    b.u[1, 1:] = 1.0                  # u q < p fails wherever q >= p: not certain with drafts, certain without
    got = b.run(hrs)
    b.check(got, what="all and none", margins=False)
    assert int(got[2][0]) == 8


def test_sample_special_rows(hrs):
    """Temperature 0 and infinity, NaN, infinities, empty rows, tokens out of
    range, repeated children."""
    f = np.float32
    V = 24
    b = Block(8, 3, V, "f32", tree=True)
    b.parent = np.tile(np.array([-1, 0, 0], dtype=np.int32), (8, 1))
    b.temp = np.array([0, np.inf, 1, 1, 1, 1, 1e-30, 1], dtype=f)
    b.logits[0, 0, [3, 9, 11]] = 50
    b.tokens[0] = [0, 9, 3]
    b.logits[1, 0, 5] = -np.inf
    b.logits[2, 0, :] = np.nan
    b.logits[3, 0, :] = -np.inf
    b.logits[4, 0, [2, 20]] = np.inf
    b.logits[5, 0, ::2] = np.nan
    b.tokens[5] = [0, -1, V]
    b.tokens[6] = [0, 4, 4]
    b.tokens[7] = [0, int(np.argmin(b.logits[7, 0]))] * 1 + [int(np.argmin(b.logits[7, 0]))]
    b.u[:, 1:] = [0.9, 0.95]
    b.check(b.run(hrs), what="special rows", margins=False)


def test_sample_draft_equal_to_target_and_zero_drafts(hrs):
    """q = p leaves a rest of rounding errors at most; a draft row of zeros
    accepts whatever the target can produce."""
    b = Block(2, 4, 256, "f32", draft="f32", temp=False)
    b.draft[1] = 0.0
    b.u[:] = 0.5
    got = b.run(hrs)
    assert got[2].tolist()[1] == 3
    b.check(got, requests=[1], what="zero drafts", margins=False)
    b.draft[0, 0] = 0
    b.draft[0, 0, 7] = 1.0
    b.logits[0, 0] = -np.inf
    b.logits[0, 0, 7] = 1.0
    b.tokens[0, 1] = 9               # never in the target: rejected; the rest max(p - q, 0) is zero everywhere
    got = b.run(hrs)
    assert (got[1][0], got[4][0]) == (0, 7)


def test_sample_bad_temperatures_are_left_alone_and_counted(hrs):
    import torch
    b = Block(4, 3, 64, "bf16")
    b.temp = np.array([1, -1, np.nan, 0.5], dtype=np.float32)
    status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    got = b.run(hrs, status=status)
    assert status.tolist() == [2, 9, 9, 9]
    for x in got:
        assert np.all(x[1:3] == -7)
    b.check(got, requests=[0, 3], what="beside bad temperatures")


def test_sample_extreme_uniforms(hrs):
    b = Block(4, 1, 96, "f32", temp=False)
    b.logits[:, 0, 90:] = -np.inf
    b.logits[:, 0, :3] = -np.inf
    b.u[:, 0] = [0.0, 1.0, 2.0, -1.0]
    got = b.run(hrs)
    assert got[4].tolist() == [3, 89, 89, 3]


def test_sample_spread_of_draws_is_the_targets(hrs):
    """4,096 stratified random numbers on one row draw every token as often
    as its probability says, to one count per border."""
    V, R = 64, 4096
    rng = np.random.default_rng(0)
    row = (rng.standard_normal(V) * 2).astype(np.float32)
    b = Block(1, 1, V, "f32", temp=False)
    b.logits = np.ascontiguousarray(np.broadcast_to(row, (R, 1, V)))
    b.tokens = np.zeros((R, 1), dtype=np.int32)
    b.u = (((np.arange(R) + 0.5) / R).astype(np.float32))[:, None].copy()
    got = b.run(hrs)
    count = np.bincount(got[4], minlength=V)
    assert np.all(np.abs(count - R * osm.probabilities(row, 1.0)) <= 1.001)


def test_sample_repeat_guard_and_graph(hrs):
    import torch
    b = Block(3, 17, 8200, "bf16", draft="f32")
    first = b.run(hrs)
    R, T, V = b.logits.shape
    n = hrs.accept_sample_workspace_bytes(R, T, V)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    again = b.run(hrs, ws=ws[256:-256])
    assert all(np.array_equal(x, y) for x, y in zip(first, again))
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[-256:] == 0xA5).all())
    # a captured call on changed inputs, eager work in between
    a = b.args()
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    dq, tau = dev(b.draft), dev(b.temp)
    call = hrs.accept_sample_call(*a, work, draft_probs=dq, temperature=tau)
    outs = b.outs
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (1, 2, 3):
        c = Block(3, 17, 8200, "bf16", draft="f32", seed=seed)
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

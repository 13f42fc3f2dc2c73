"""attn_verify_span on the GPU: what a query does not count leaves its result
alone, bit for bit, also where it is finite and large; what it counts is seen,
also where it is not a number."""
import numpy as np
import pytest

from oracle import attn as oa
from oracle.common import widen
from tests.test_gpu_attn import KINDS, Attn, cast, host
from tests.test_gpu_attn_runs import Runs, block_shape

pytestmark = pytest.mark.gpu

NEG = {"f32": np.float32(-np.inf), "bf16": np.uint16(0xFF80)}


@pytest.fixture(scope="module")
def hrs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import hybrid_recurrent_state_amd as m
    return m


def toward(q, size, dtype):
    """A key whose products with the query q are large and positive."""
    return cast(size * np.sign(widen(q)), dtype)


def path_of(parent, t):
    out = []
    while t >= 0:
        out.append(t)
        t = int(parent[t])
    return out


@pytest.mark.parametrize("size", [40.0, 1e8])
@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])       # 9 to 108 rows a key head: every class of blocks
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_large_keys_off_the_path_change_nothing(hrs, dtype, cache, d, group, size):
    """Keys of other branches with scores of a hundred (a hundred million) for
    the positions that count them, in a tile behind tiles of the context that have set every
    row's reference; a row's own keys in that tile are a little larger than
    the context's, so that its maximum grows without its reference having to
    move."""
    import torch
    rows, ts, blocks, _ = block_shape(cache, d, 9 * group)
    n = 5 * blocks * ts // 4
    a = Runs(2, 9, group, 2, d, 64, [n, n // 2 + 3], dtype, cache, True, 0, seed=d + group)
    a.scale = 0.3 * d ** -0.5
    for t in range(9):
        a.k[:, t] = cast(0.5 * widen(a.q)[:, t, ::group], dtype)
    clean = a.run(hrs)
    k0 = a.k.copy()
    for node in (0, 4, 8):
        a.k = k0.copy()
        for r in range(2):
            off = [t for t in range(9) if t not in path_of(a.parent[r], node)]
            for t in off:
                for h in range(2):
                    a.k[r, t, h] = toward(a.q[r, t, h * group], size, dtype)
        got = a.run(hrs)
        assert torch.equal(got[:, node], clean[:, node]), node
        assert not torch.equal(got, clean)


@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f32")])
def test_large_keys_behind_the_window_change_nothing(hrs, dtype, cache, group):
    """Slots that only the first positions' windows still reach."""
    import torch
    T, W, n = 9, 50, 200
    a = Attn(1, T, 2 * group, 2, 64, 16, [n], dtype, cache, window=W, seed=group)
    clean = a.run(hrs)
    for t in (3, 8):                          # the first slot that position t counts is n + t - W + 1
        for j in range(n - W + 1, n + t - W + 1):
            for h in range(2):
                a.kc[a.pages[0][j // 16], h, j % 16] = toward(a.q[0, 0, h * group], 40.0, cache)
        got = a.run(hrs)
        assert torch.equal(got[:, t:], clean[:, t:]), t
        assert not torch.equal(got[:, 0], clean[:, 0])


@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_scale_that_is_not_a_number_is_seen(hrs, dtype, cache, group):
    a = Attn(2, 9, 2 * group, 2, 64, 16, [100, 0], dtype, cache, scale=float("nan"))
    assert np.isnan(widen(host(a.run(hrs)))).all()


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_scale_that_is_not_a_number(hrs, d, group, which):
    """Seen by every query that counts a cached slot of its head, by no other:
    not by the other head's, by a request without a context's, nor by those
    whose window ends at their own position."""
    import torch
    a = Attn(2, 9, 2 * group, 2, d, 16, [100, 0], "bf16", "f8", seed=group)
    clean = a.run(hrs)
    keep, bad = getattr(a, which), getattr(a, which).copy()
    bad[1] = np.nan
    setattr(a, which, bad)
    got = a.run(hrs)
    assert bool(torch.isnan(got[0, :, group:]).all())
    assert torch.equal(got[0, :, :group], clean[0, :, :group]) and torch.equal(got[1], clean[1])
    a.window = 1
    setattr(a, which, keep)
    clean = a.run(hrs)
    setattr(a, which, bad)
    assert torch.equal(a.run(hrs), clean)


@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("n", [0, 100, 3000])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f32")])
def test_scores_of_minus_infinity_alone_have_no_softmax(hrs, dtype, cache, n, group):
    """Every score of one head is -inf: 0 / 0. The other head's are not
    touched, and one finite score is enough."""
    import torch
    a = Attn(1, 9, 2 * group, 2, 64, 16, [n], dtype, cache, seed=group)
    a.q = np.abs(a.q) if dtype == "f32" else a.q & np.uint16(0x7FFF)
    clean = a.run(hrs)
    a.kc[:, 1], a.k[:, :, 1] = NEG[cache], NEG[dtype]
    got = a.run(hrs)
    assert bool(torch.isnan(got[:, :, group:]).all())
    assert torch.equal(got[:, :, :group], clean[:, :, :group])
    a.k[:, 0, 1] = 0                                       # the root counts for everybody
    got = widen(host(a.run(hrs)))
    for t in range(9):
        assert np.array_equal(got[0, t, group:], np.broadcast_to(widen(a.v[0, 0, 1]), (group, 64))), t


@pytest.mark.parametrize("power", [20, 24, 27, 33, 60, 100])
@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_scores_far_out_leave_the_largest(hrs, dtype, cache, group, power):
    """Scores of about 2^power, the largest twice the second: the result is
    that slot's value, however the scores are rounded. The slot lies in the
    context or is the root of the span."""
    n = 3000
    for where in (5, 2500, n):
        a = Attn(1, 9, 2 * group, 2, 64, 16, [n], dtype, cache, seed=group, scale=1.0)
        rng = np.random.default_rng(power)
        a.q, a.k = cast(np.zeros(a.q.shape), dtype), cast(np.zeros(a.k.shape), dtype)
        # One product a score, whose rounding with the scale is not exact.
        a.q[..., 3] = cast(np.full(1, 1.4140625 * 2.0 ** (power // 2)), dtype)
        size = 2.0 ** (power - power // 2)
        a.scale = 1.37
        if cache == "f8":
            a.kc[:] = 0
            a.kc[..., 3] = rng.integers(0x28, 0x31, a.kc.shape[:3]).astype(np.uint8)      # 0.25 to 0.5
            a.ks = np.full(2, 1.1 * size, dtype=np.float32)
            one = np.uint8(0x39)                                                          # 1.125
        else:
            a.kc[:] = cast(np.zeros(a.kc.shape), cache)
            a.kc[..., 3] = cast(rng.uniform(0.25, 0.5, a.kc.shape[:3]) * size, cache)
            one = cast(np.full(1, 1.1328125 * size), cache)
        if where < n:
            a.kc[a.pages[0][where // 16], :, where % 16, 3] = one
            page = a.vc[a.pages[0][where // 16], :, where % 16]
            want = oa.widen_cache(page) * (1.0 if a.vs is None else a.vs.astype(np.float64)[:, None])
        else:
            a.k[0, 0, :, 3] = cast(np.full(1, 1.1328125 * size), dtype)
            want = widen(a.v)[0, 0]
        got = widen(host(a.run(hrs)))[0].reshape(9, 2, group, 64)
        tol = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -22) * np.abs(want[None, :, None]) * 1.01 + (2.0 ** -11 if cache == "f8" else 2.0 ** -15 if dtype == "bf16" else 0) * np.abs(want[None, :, None])
        assert np.all(np.abs(got - want[None, :, None]) <= tol), where


@pytest.mark.parametrize("power", [22, 24, 25, 26, 27, 28, 31, 34])
@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_scores_far_out_in_small_steps(hrs, dtype, cache, group, power):
    """Scores of 2^power that grow along the context in steps of an ulp or a
    few: whatever their rounding makes of the differences, weights are
    positive and add up to one, so results lie within the values."""
    n = 3000
    a = Attn(1, 3, 2 * group, 2, 64, 16, [n], dtype, cache, seed=group, scale=float(np.log(2.0)))
    a.q, a.k = cast(np.zeros(a.q.shape), dtype), cast(np.zeros(a.k.shape), dtype)
    a.q[..., 0] = cast(np.full(1, 2.0 ** power), dtype)
    a.q[..., 1] = cast(np.full(1, 2.0 ** max(power - 23, 1)), dtype)
    step = np.minimum(np.arange(n) // 150, 15)
    one = {"f8": np.uint8(0x38), "bf16": np.uint16(0x3F80), "f32": np.float32(1)}[cache]
    small = oa.quantize_e4m3(np.arange(16.0), None) if cache == "f8" else cast(np.arange(16.0), cache)
    a.kc[:] = 0
    a.kc[..., 0] = one
    for j in range(n):
        a.kc[a.pages[0][j // 16], :, j % 16, 1] = small[step[j]]
    if cache == "f8":
        a.ks = np.full(2, 1.0, dtype=np.float32)
    got = widen(host(a.run(hrs)))
    v = oa.widen_cache(a.vc) * (1.0 if a.vs is None else a.vs.astype(np.float64)[None, :, None, None])
    assert np.isfinite(got).all() and np.abs(got).max() <= np.abs(v).max() * (1 + 2.0 ** -7)

"""accept_sample_filtered where its counts, sums and arguments end: zeros of
both signs at the last value that is counted, temperatures and logits at the
ends of float32, weights that are all off the same way, borders a rounding away
from top-p or below zero, and rows of more than a million logits.

Tolerances of test_gpu_filter.py but where a test derives its own.
"""
import numpy as np
import pytest

from oracle.common import widen
from oracle.filter import filtered
from tests.test_gpu_attn import hrs  # noqa: F401
from tests.test_gpu_filter import Filtered, U
from tests.test_gpu_sample import cast

pytestmark = pytest.mark.gpu


# The largest logit's bits: zero is the last value that is counted one by one
# (0x3BFF), the last but one, none of them; and with a temperature at which
# e^-48 of the largest weight is exactly zero's.
@pytest.mark.parametrize("top,tau", [(0x3BFF, 1.0), (0x3BFE, 1.0), (0x3C00, 1.0), (0x3BC0, 2.0 ** -13)])
@pytest.mark.parametrize("mixed", [False, True])
def test_zeros_of_both_signs_where_counting_ends(hrs, top, tau, mixed):
    n = 10000                                          # of each sign
    ks = [n + 1, n, 1 + n // 2, 2 * n + 1, n + 2, 2 * n]
    b = Filtered(len(ks), 2, 20008, "bf16", temp=False, k=ks)
    b.temp = np.full(len(ks), tau, np.float32)
    b.logits[:] = 0xFF80                               # -inf
    b.logits[:, :, 0] = top
    zeros = np.repeat(np.array([0x0000, 0x8000], np.uint16), n)
    b.logits[:, :, 1:2 * n + 1] = np.random.default_rng(1).permutation(zeros) if mixed else zeros
    b.tokens[:, 1] = [2 * n, n, n // 2 + 1, 2 * n, n + 1, 2 * n]
    b.u[:, 1] = 0.99
    b.u[:, 0] = [0.9995, 0.7, 0.9995, 0.9995, 0.3, 0.9995]
    b.check(b.run(hrs), what="zeros", margins=False)


def extreme(dtype, kind, R, V, seed=3):
    """Logits and a temperature at the ends of float32."""
    rng = np.random.default_rng(seed)
    low = -3.4028235e38 if dtype == "f32" else -3.3895314e38
    if kind == "inf":                                  # half of them masked with the lowest number
        z = rng.standard_normal((R, 2, V)) * 2.5
        z[:, :, rng.random(V) < 0.5] = low
        return z, np.inf
    if kind == "all":                                  # differences past the largest number
        z = rng.uniform(-1, 1, (R, 2, V)) * -low
        z[:, :, 7] = -low
        return z, 1e38
    if kind == "large":
        return rng.standard_normal((R, 2, V)) * 2e37, 1e37
    return rng.integers(0, 40, (R, 2, V)) * 1e-41, 1e-40        # below the smallest normal number


EXTREME = [("f32", "inf"), ("f32", "all"), ("f32", "large"), ("f32", "small"), ("bf16", "inf"), ("bf16", "all"), ("bf16", "large")]


@pytest.mark.parametrize("dtype,kind", EXTREME)
def test_temperatures_at_the_ends_of_float32(hrs, dtype, kind):
    V = 16392
    b = Filtered(5, 2, V, dtype, temp=False, k=[0, 0, 6000, 0, 9000], p=[1.0, 0.3, 1.0, 1.0, 0.7], m=[0, 0, 0, 0.4, 0.01])
    z, tau = extreme(dtype, kind, 5, V)
    b.logits = cast(z, dtype)
    b.temp = np.full(5, tau, np.float32)
    rng = np.random.default_rng(5)
    b.tokens[:, 1] = np.argsort(-widen(b.logits[:, 0]), -1)[:, 11]
    b.u[:] = rng.uniform(0.05, 0.95, b.u.shape)
    b.check(b.run(hrs), what=kind, margins=False)


def test_weights_that_are_off_the_same_way(hrs):
    """2^20 logits whose difference to the largest is 0.49 of a float32 step short of the next number: in float32 every
    weight would be off by 0.49 * 2^-19 / 1.25 of it, 12.5 u, all in one direction (9.3 u of the sum).
    All but one stay. A weight: 2 u of the exponential, u of the factor for what its argument leaves, half of 2^-42 for being
    a whole number, 0.7 u of e^-12.8; the result's own rounding u: 5 u."""
    V = 1 << 20
    b = Filtered(1, 2, V, "f32", temp=False, k=V - 1)
    b.temp = np.array([1.25], np.float32)
    b.logits[:] = np.float32(-0.49 * 2.0 ** -19)
    b.logits[:, :, 1000] = np.float32(16 + 2.0 ** -19)
    b.tokens[:, 1] = 1000
    prob = b.run(hrs)[0][0, 1]
    want = filtered(b.logits[0, 0], 1.25, V - 1)[0][1000]
    assert abs(prob - want) <= 5 * U * want, (prob - want) / want / U


def test_weights_as_whole_numbers_in_a_very_long_row(hrs):
    """2^24 logits that weigh e^-16.1 each beside one: half a unit of 2^-38 each, for sums that could hold 2^24 of the largest,
    was 272 u of them; the sum says how many fit (2^-50: 0.1 u). Else as above."""
    V = 1 << 24
    b = Filtered(1, 2, 64, "f32", temp=False, k=V - 1)
    b.logits = np.zeros((1, 2, V), np.float32)
    b.logits[:, :, 1000] = 16.109375
    b.tokens[:, 1] = 1000
    prob = b.run(hrs)[0][0, 1]
    want = 1 / (1 + (V - 2) * np.exp(-16.109375))
    assert abs(prob - want) <= 5 * U * want, (prob - want) / want / U


@pytest.mark.parametrize("dtype,V", [("bf16", 4096), ("f32", 4096), ("f32", 40000), ("bf16", 40000)])
def test_borders_a_rounding_away_from_top_p(hrs, dtype, V):
    """top-p is the cumulative share of a token rounded to float32, so whether that token reaches it is decided 2^-25 or so
    from the border: by the 64-bit sums of a row that top-k leaves to its list. A 64-bit weight over such a sum is rounded
    once; 2 u."""
    R = 64
    rng = np.random.default_rng(V)
    b = Filtered(R, 2, V, dtype, temp=True, k=rng.integers(3, 120, R))
    b.p = np.ones(R, np.float32)
    for r in range(R):
        p, n = filtered(b.logits[r, 0], float(b.temp[r]), int(b.k[r]))
        z = widen(b.logits[r, 0])
        order = np.lexsort((np.arange(V), -z))[:n]
        c = np.cumsum(p[order])
        j = int(rng.integers(0, n - 1))
        b.p[r] = np.float32(c[j] / c[-1])
        if abs(float(b.p[r]) * c[-1] - c[j]) < 1e-11:
            b.p[r] = np.nextafter(b.p[r], np.float32(1))
        b.tokens[r, 1] = order[j + 1]                  # stays only if the j-th does not reach the share
    prob = b.run(hrs)[0]
    for r in range(R):
        want = filtered(b.logits[r, 0], float(b.temp[r]), int(b.k[r]), float(b.p[r]))[0][b.tokens[r, 1]]
        assert abs(prob[r, 1] - want) <= 2 * U * want + 2.0 ** -126, (r, prob[r, 1], want)


LONG = [("f32", 600008, dict(p=0.9)), ("f32", 600008, dict(k=300000, m=1e-4)), ("bf16", 1100008, dict(p=0.9)),
        ("bf16", 1100008, dict(k=700000, p=0.97))]


@pytest.mark.parametrize("dtype,V,limits", LONG, ids=str)
def test_rows_of_a_million_logits(hrs, dtype, V, limits):
    b = Filtered(1, 2, V, dtype, **limits)
    b.check(b.run(hrs), what="long")


@pytest.mark.parametrize("dtype,V", [("f32", 600008), ("bf16", 1100008)])
def test_ties_far_into_a_long_row(hrs, dtype, V):
    b = Filtered(3, 1, V, dtype, temp=False, k=[500001, 0, 262145], p=[1.0, 0.75, 1.0])
    b.logits = cast(np.full((3, 1, V), 1.5, np.float32), dtype)
    b.u[:, 0] = [0.99999, 0.6, 0.5]
    b.check(b.run(hrs), what="far ties", margins=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [-4.0, -8.0])
def test_even_rows_with_their_border_below_zero(hrs, dtype, shift):
    b = Filtered(4, 3, 30000, dtype, draft="f32", temp=False, k=[0, 12000, 0, 0], p=[0.9, 1.0, 0.97, 1.0], m=[0, 0, 0, 0.01])
    b.logits = cast(widen(b.logits) + shift, dtype)
    b.check(b.run(hrs), what=f"shifted by {shift}")

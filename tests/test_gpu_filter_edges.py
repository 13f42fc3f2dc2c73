"""accept_sample_filtered where its counts, sums and arguments end: zeros of
both signs at the last value that is counted, temperatures and logits at the
ends of float32, weights that are all off the same way.

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

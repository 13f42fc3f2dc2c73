"""attn_verify_span on the GPU: the softmax weights of bf16 spans keep more bits
than bf16 for the product with the values, and small ones are not lost.

Scores are exact here: a query has one element that is not zero, so a score is
one product of two 8-bit mantissas (4-bit ones of an e4m3 cache). A weight is
then off by the roundings of the factor of the scores (3 u), of the exponent's
argument (u) and of the exponential (2 u), u = 2^-24, and by what the product
keeps of it:
  bf16 values: the upper 8 bits, cut off, and the rest (below 2^-7 of it)
    rounded to bf16 (2^-8 of it), made larger by 2^-40 of the weight: 2^-15 +
    2^-40.
  e4m3 values: float16, 2^-11, and 2^-25 beside a reference weight of 2^7 at
    least, which the largest weight is not below: 2^-32 of the sum of the
    weights for every slot.
"""
import numpy as np
import pytest

from oracle.common import widen
from tests.test_gpu_attn import OUT, U, Attn, cast, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hrs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import hybrid_recurrent_state_amd as m
    return m


KEEPS = {"bf16": 2.0 ** -15 + 2.0 ** -40, "f8": 2.0 ** -11, "f32": 0.0}


def check(a, got):
    from oracle import attn as oa
    got = widen(host(got))
    top = max(float(np.max(np.abs(oa.widen_cache(a.vc)))) * (1 if a.vs is None else float(a.vs.max())), float(np.max(np.abs(widen(a.v)))))
    for r in range(a.shape[0]):
        ref, absv, reach, n = oa.attn_span(a.q[r], a.k[r], a.v[r], a.kc, a.vc, a.pages[r], a.lens[r],
                                           None if a.parent is None else a.parent[r], a.scale, a.window, a.ks, a.vs,
                                           want_bound=True)
        rel = 2 * (4 * U) * reach + (2 * n + 16) * U + KEEPS[a.cache] + (KEEPS["bf16"] if a.cache == "f8" else 0)
        e = rel[..., None] * absv + (n[..., None] * 2.0 ** -32 * top if a.cache == "f8" else 0)
        tol = e + OUT[a.dtype] * (np.abs(ref) + e)
        err = np.abs(got[r] - ref)
        assert np.all(err <= tol), (r, float(np.max(err / tol)), int((err > tol).sum()))


@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])       # 9 to 108 rows a key head: every class of blocks
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")])
def test_weights_keep_their_bits(hrs, dtype, cache, d, group):
    a = Attn(2, 9, 2 * group, 2, d, 16, [200, 77], dtype, cache, seed=group, scale=1.0)
    q = np.zeros(a.q.shape, dtype=np.float32)
    for t in range(9):
        for h in range(2 * group):
            q[:, t, h, (7 * t + 5 * h) % d] = 2.5
    a.q = cast(q, dtype)
    check(a, a.run(hrs))


@pytest.mark.parametrize("less", [12, 16, 20, 28])         # in log2
@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")])
def test_small_weights_of_many_slots_count(hrs, dtype, cache, group, less):
    """One slot has a large weight and a value of zero: the result is what
    thousands of slots of 2^-12 to 2^-28 of its weight add up to."""
    n = 20000
    a = Attn(1, 2, 2 * group, 2, 64, 64, [n], dtype, cache, seed=group, scale=float(np.log(2.0)))
    a.q = cast(np.zeros(a.q.shape), dtype)
    a.q[..., 0] = cast(np.full((), 1.0), dtype)
    a.k, a.v = (cast(np.zeros(a.k.shape), dtype) for _ in range(2))
    one = {"f8": np.uint8(0x38), "bf16": np.uint16(0x3F80), "f32": np.float32(1)}[cache]
    a.kc[:], a.vc[:] = 0, one
    if cache == "f8":
        a.ks, a.vs = np.full(2, 1.0, dtype=np.float32), np.full(2, 1.0, dtype=np.float32)
    peak = a.pages[0][5], 5                                 # slot 5 * 64 + 5
    a.vc[peak[0], :, peak[1]] = 0
    a.kc[peak[0], :, peak[1], 0] = {"f8": np.uint8({12: 0x54, 16: 0x58, 20: 0x5A, 28: 0x5E}[less]),
                                    "bf16": cast(np.full((), less), "bf16")[()], "f32": np.float32(less)}[cache]
    check(a, a.run(hrs))

"""accept_sample_filtered where its counts, sums and arguments end.

Tolerances of test_gpu_filter.py but where a test derives its own.
"""
import numpy as np
import pytest

from tests.test_gpu_attn import hrs  # noqa: F401
from tests.test_gpu_filter import Filtered

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

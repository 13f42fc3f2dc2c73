"""accept_sample with temperatures and logits at the ends of float32.
Tolerances of test_gpu_sample.py.
"""
import numpy as np
import pytest

from oracle.common import widen
from tests.test_gpu_filter_edges import EXTREME, extreme
from tests.test_gpu_sample import Block, cast, hrs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,kind", EXTREME)
def test_accept_sample_at_the_ends_of_float32(hrs, dtype, kind):
    V = 16392
    b = Block(3, 2, V, dtype, temp=False)
    z, tau = extreme(dtype, kind, 3, V)
    b.logits = cast(z, dtype)
    b.temp = np.full(3, tau, np.float32)
    b.tokens[:, 1] = np.argsort(-widen(b.logits[:, 0]), -1)[:, 11]
    b.u[:] = np.random.default_rng(6).uniform(0.05, 0.95, b.u.shape)
    b.check(b.run(hrs), what=kind, margins=False)

"""attn_verify_shared with more than 256 rows of a key head in a launch (at
most 256 requests): last blocks with few rows and waves without any, several
launches of different size, short and refused requests, far pages.

Tolerances as in test_gpu_shared.py.
"""
import numpy as np
import pytest

from tests.test_gpu_attn import dev, hrs  # noqa: F401
from tests.test_gpu_shared import WIDE, Large, Shared

pytestmark = pytest.mark.gpu


def rows(a):
    R, T, Hq, Hkv, _, _ = a.shape
    return min(R, 256) * T * (Hq // Hkv)


@pytest.mark.parametrize("dtype,cache", WIDE)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("R,T,group", [(87, 3, 1), (65, 1, 4), (193, 1, 2), (145, 1, 4), (29, 5, 4)])
def test_last_blocks_of_few_rows(hrs, dtype, cache, d, R, T, group):
    """261, 260, 386, 580 and 580 rows in blocks of 192 (heads of 64: of 256)."""
    a = Large(R, T, 2 * group, 2, d, 32, 700, [700 + (11 * r) % 60 for r in range(R)], dtype, cache, seed=R)
    a.ptable[5] = -1
    assert rows(a) > 256
    a.check(a.run(hrs), [0, R // 2, R - 1], what=f"{rows(a)} rows")


@pytest.mark.parametrize("dtype,cache", WIDE)
@pytest.mark.parametrize("R,T,tree", [(300, 2, False), (500, 2, False), (130, 25, True)])
def test_several_launches(hrs, dtype, cache, R, T, tree):
    """The last one smaller: in the same path (500 requests, 130 trees) or not (300)."""
    a = Large(R, T, 4, 2, 64, 16, 400, [400 + (7 * r) % 50 for r in range(R)], dtype, cache, tree=tree, seed=R)
    assert rows(a) > 256
    got = a.run(hrs)
    a.check(got, sorted({0, 121, 122, 129, 255, 256, 257, R - 1} & set(range(R))), what=f"{R} requests")
    import torch
    assert torch.equal(got, a.run(hrs))


@pytest.mark.parametrize("dtype,cache", WIDE)
def test_short_empty_and_refused_requests_in_a_large_batch(hrs, dtype, cache):
    """The shared slots end at the shortest context; refused requests do not count."""
    import torch
    for lens in ([0] + [900 + r for r in range(79)], [900 + r for r in range(79)] + [130], [-1, 10 ** 9] + [900] * 78):
        a = Large(80, 1, 8, 2, 128, 16, 800, [max(0, n) if n < 2000 else 0 for n in lens], dtype, cache)
        a.lens = lens
        status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
        got = a.run(hrs, status=status)
        bad = [r for r, n in enumerate(lens) if not 0 <= n <= a.pages.shape[1] * 16]
        assert status.tolist() == [len(bad), 9, 9, 9]
        assert all(bool((got[r] == 77).all()) for r in bad)
        a.check(got, sorted({0, 1, 2, 40, 79} - set(bad)), what=f"lengths {lens[0]}, {lens[-1]}")


def test_far_pages_in_a_large_batch(hrs):
    """Pages behind 2^31 elements."""
    import torch
    N, H, S, d = 70000, 4, 64, 128          # 2.3e9 elements a side, 4.6 GB
    a = Large(70, 2, 8, 4, d, S, 1030, [1040 + r % 60 for r in range(70)])
    assert rows(a) > 256
    big = [torch.zeros(N, H, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    step = 69999 // a.N
    far = (np.arange(a.N) * step + 69999 - step * (a.N - 1)).astype(np.int32)
    for b, c in zip(big, (a.kc, a.vc)):
        b[torch.from_numpy(far).long().cuda()] = dev(c)
    t = a.tensors(hrs)
    t.update(k_cache=big[0], v_cache=big[1], prefix_table=dev(far[a.ptable]), page_table=dev(far[a.pages]))
    hrs.attn_verify_shared(**t)
    a.check(t["out"], [0, 35, 69], what="far pages")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_float32_spans_in_a_large_batch(hrs, d):
    """These stay on the kernels for up to 128 rows a block."""
    a = Shared(45, 3, 8, 2, d, 32, 700, [700 + (11 * r) % 60 for r in range(45)], "f32", "f32")
    a.ptable[7] = -1
    a.check(a.run(hrs), [0, 22, 44], what="float32")

"""Refusals and hand-worked lists of kv_pages_reserve up to the end of a
request's table and without some of the requests, on the host as in
test_boundary_pages.py."""
import numpy as np
import pytest

from oracle import pages as op
from tests.test_boundary_attn import t
from tests.test_boundary_host import FAKE, MIS, hrs
from tests.test_boundary_pages import DESC, RESERVE, args, call
from tests.test_oracle_pages import i32


def reserve(**kw):
    return call("kv_pages_reserve", hrs.PagesDesc, RESERVE, dict(DESC, clip=0, skip=None), kw, extra=(1 << 20,))[0]


@pytest.mark.parametrize("clip,want", [(0, hrs.HRS_EDEVICE), (1, hrs.HRS_EDEVICE), (2, hrs.HRS_EINVAL), (-1, hrs.HRS_EINVAL)])
def test_clip_is_one_of_two(clip, want):
    assert reserve(clip=clip) == want
    assert call("kv_pages_release", hrs.PagesDesc, ["keep_len", "page_table", "n_held", "free_pages", "n_free", "status",
                                                    "workspace"], dict(DESC, clip=clip), {}, extra=(1 << 20,))[0] == want


def test_hand_worked():
    """Tables of four pages of 16: request 0 has 48 slots and may get its last page, 1 has all, 2 is past the end."""
    for clip, held, slots, missed in ((False, [3, 4, 4], [-1] * 3, 3), (True, [4, 4, 4], [112, 111, -1], 1)):
        table, have, free = i32([0, 1, 2, -1], [3, 4, 5, 6], [8, 10, 11, 0]), i32(3, 4, 4), i32(9, 7, -1, -1)
        n, got, bad = op.reserve([48, 63, 65], [17] * 3, table, have, free, 2, 16, 17, n_pages=12, clip=clip)
        assert have.tolist() == held and bad == missed
        assert [int(x) for x in got[:, 0]] == slots and (got[1, 1:] == -1).all() and n == (1 if clip else 2)
        assert not clip or ((got[0, :16] == 112 + np.arange(16)).all() and got[0, 16] == -1)


def test_skip():
    assert reserve(skip=FAKE) == hrs.HRS_EDEVICE and reserve(skip=MIS) == hrs.HRS_EALIGN
    # The first request's three pages would leave one for the second, which needs two.
    for skip, held, left in ((None, [3, 0], 1), ([1, 0], [0, 2], 2)):
        table, have, free = np.full((2, 4), -1, np.int32), i32(0, 0), i32(3, 1, 0, 2)
        n, slots, missed = op.reserve([0, 0], [40, 20], table, have, free, 4, 16, 40, skip=skip)
        assert have.tolist() == held and n == left and missed == (skip is None)
        assert skip is None or ((slots[0] == -1).all() and (table[0] == -1).all())


def test_binding_refuses_wrong_tensors():
    import torch
    i32_ = torch.int32
    ok = dict(args(), seq_len=t(4, dtype=i32_), skip=t(4, dtype=i32_), n_pos=3, clip=True)
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_pages_reserve(**ok)
    with pytest.raises(TypeError):
        hrs.kv_pages_reserve(**{**ok, "skip": t(4, dtype=torch.bool)})
    with pytest.raises(ValueError):
        hrs.kv_pages_reserve(**{**ok, "skip": t(3, dtype=i32_)})
    with pytest.raises(ValueError, match="overlaps"):
        hrs.kv_pages_reserve(**{**ok, "skip": ok["n_held"]})

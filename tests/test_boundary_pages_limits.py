"""Refusals and hand-worked lists of kv_pages_reserve up to the end of a
request's table, on the host as in test_boundary_pages.py."""
import numpy as np
import pytest

from oracle import pages as op
from tests.test_boundary_host import hrs
from tests.test_boundary_pages import DESC, call, release, RESERVE
from tests.test_oracle_pages import i32


def reserve(**kw):
    return call("kv_pages_reserve", hrs.PagesDesc, RESERVE, dict(DESC, clip=0), kw, extra=(1 << 20,))[0]


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

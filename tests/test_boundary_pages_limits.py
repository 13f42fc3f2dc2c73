"""Refusals and hand-worked lists of kv_pages_reserve_step (up to the end of a
request's table, without some of the requests), on the host as in
test_boundary_pages.py."""
import numpy as np
import pytest

from oracle import pages as op
from tests.test_boundary_attn import t
from tests.test_boundary_host import FAKE, MIS, hrs
from tests.test_boundary_pages import DESC, RESERVE, args, call
from tests.test_oracle_pages import i32


NAMES = RESERVE[:2] + ["skip"] + RESERVE[2:]


def reserve(nbytes=1 << 20, **kw):
    return call("kv_pages_reserve_step", hrs.PagesDesc, NAMES, DESC, kw, extra=(nbytes,))[0]


def test_rejections():
    optional = ("n_new", "skip", "slot_map", "status")
    assert reserve() == hrs.HRS_EDEVICE
    assert reserve(**{n: None for n in optional}) == hrs.HRS_EDEVICE
    for bad in (dict(n_req=0), dict(n_req=4097), dict(n_pos=0), dict(n_pages=0), dict(page_size=48), dict(table_len=0),
                dict(n_prefix=5), dict(n_prefix=0), dict(nbytes=24)):
        assert reserve(**bad) == hrs.HRS_EINVAL, bad
    for name in NAMES:
        if name not in optional:
            assert reserve(**{name: None}) == hrs.HRS_EINVAL, name
        assert reserve(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert hrs.lib.kv_pages_reserve_step(None, *[FAKE] * 11, 1 << 20, None) == hrs.HRS_EINVAL


def test_hand_worked():
    """Tables of four pages of 16: request 0 has 48 slots and may get its last page, 1 has all, 2 is past the end."""
    for clip, held, slots, missed in ((False, [3, 4, 4], [-1] * 3, 3), (True, [4, 4, 4], [112, 111, -1], 1)):
        table, have, free = i32([0, 1, 2, -1], [3, 4, 5, 6], [8, 10, 11, 0]), i32(3, 4, 4), i32(9, 7, -1, -1)
        n, got, bad = op.reserve([48, 63, 65], [17] * 3, table, have, free, 2, 16, 17, n_pages=12, clip=clip)
        assert have.tolist() == held and bad == missed
        assert [int(x) for x in got[:, 0]] == slots and (got[1, 1:] == -1).all() and n == (1 if clip else 2)
        assert not clip or ((got[0, :16] == 112 + np.arange(16)).all() and got[0, 16] == -1)


def test_skip():
    # The first request's three pages would leave one for the second, which needs two.
    for skip, held, left in ((None, [3, 0], 1), ([1, 0], [0, 2], 2)):
        table, have, free = np.full((2, 4), -1, np.int32), i32(0, 0), i32(3, 1, 0, 2)
        n, slots, missed = op.reserve([0, 0], [40, 20], table, have, free, 4, 16, 40, skip=skip)
        assert have.tolist() == held and n == left and missed == (skip is None)
        assert skip is None or ((slots[0] == -1).all() and (table[0] == -1).all())


def test_binding_refuses_wrong_tensors():
    import torch
    i32_ = torch.int32
    ok = dict(args(), seq_len=t(4, dtype=i32_), skip=t(4, dtype=i32_), n_pos=3)
    for more in (dict(), dict(skip=None)):
        with pytest.raises(ValueError, match="GPU"):
            hrs.kv_pages_reserve_step(**{**ok, **more})
    with pytest.raises(TypeError):
        hrs.kv_pages_reserve_step(**{**ok, "skip": t(4, dtype=torch.bool)})
    with pytest.raises(ValueError):
        hrs.kv_pages_reserve_step(**{**ok, "skip": t(3, dtype=i32_)})
    with pytest.raises(ValueError, match="overlaps"):
        hrs.kv_pages_reserve_step(**{**ok, "skip": ok["n_held"]})

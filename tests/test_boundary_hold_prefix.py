"""Refusals of accept_hold_behind on the host, as in test_boundary_hold.py."""
import ctypes

import pytest

from tests.test_boundary_attn import t
from tests.test_boundary_hold import NAMES
from tests.test_boundary_host import FAKE, MIS, hrs

DESC = dict(n_req=2, n_pos=5, n_pages=8, page_size=16, table_len=4)


def hold(prefix_len=0, ptr=None, **kw):
    p = {n: FAKE for n in NAMES}
    p.update(ptr or {})
    d = hrs.HoldDesc(**{**DESC, **kw})
    return hrs.lib.accept_hold_behind(ctypes.byref(d), prefix_len, *p.values(), None)


def test_rejections():
    for n, want in ((0, hrs.HRS_EDEVICE), (100, hrs.HRS_EDEVICE), (2 ** 31 - 1, hrs.HRS_EDEVICE), (-1, hrs.HRS_EINVAL)):
        assert hold(n) == want
    for bad in (dict(n_req=0), dict(n_pos=65), dict(n_pages=0), dict(page_size=48), dict(table_len=1 << 27)):
        assert hold(16, **bad) == hrs.HRS_EINVAL, bad
    for name in NAMES:
        if name not in ("temperature", "held_node"):
            assert hold(16, {name: None}) == hrs.HRS_EINVAL, name
        assert hold(16, {name: MIS}) == hrs.HRS_EALIGN, name
    assert hrs.lib.accept_hold_behind(None, 16, *[FAKE] * 10, None) == hrs.HRS_EINVAL


def test_binding_refuses_wrong_tensors():
    import torch
    i32 = torch.int32
    ok = dict(page_table=t(2, 3, dtype=i32), seq_len=t(2, dtype=i32), accept_node=t(2, dtype=i32),
              accept_len=t(2, dtype=i32), path=t(2, 5, dtype=i32), bonus=t(2, dtype=i32), held=t(2, dtype=i32),
              last_node=t(2, dtype=i32), n_pages=4, page_size=16, prefix_len=20)
    with pytest.raises(ValueError, match="GPU"):
        hrs.accept_hold_behind(**ok)
    with pytest.raises(ValueError):
        hrs.accept_hold_behind(**{**ok, "held": t(3, dtype=i32)})
    with pytest.raises(ValueError, match="overlaps"):
        hrs.accept_hold_behind(**{**ok, "last_node": ok["held"]})

"""Refusals of accept_hold on the host, as in test_boundary_attn.py: device
pointers are fake, a well-formed call ends in HRS_EDEVICE."""
import pytest

from tests.test_boundary_attn import call, t
from tests.test_boundary_host import FAKE, MIS, hrs

NAMES = ["page_table", "seq_len", "temperature", "accept_node", "accept_len", "path", "bonus", "held", "last_node",
         "held_node"]


def hold(**kw):
    return call("accept_hold", hrs.HoldDesc, NAMES, dict(n_req=2, n_pos=5, n_pages=8, page_size=16, table_len=4), kw)[0]


def test_hold_rejections():
    assert hold() == hrs.HRS_EDEVICE
    assert hold(temperature=None, held_node=None, n_pos=64, page_size=1024) == hrs.HRS_EDEVICE
    for bad in (dict(n_req=0), dict(n_req=65536), dict(n_pos=0), dict(n_pos=65), dict(n_pages=0), dict(page_size=8),
                dict(page_size=48), dict(page_size=2048), dict(table_len=0), dict(table_len=1 << 27)):
        assert hold(**bad) == hrs.HRS_EINVAL, bad
    for name in NAMES:
        if name not in ("temperature", "held_node"):
            assert hold(**{name: None}) == hrs.HRS_EINVAL, name
        assert hold(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert hrs.lib.accept_hold(None, *[FAKE] * 10, None) == hrs.HRS_EINVAL


def test_binding_refuses_wrong_tensors():
    import torch
    i32, f32 = torch.int32, torch.float32
    ok = dict(page_table=t(2, 3, dtype=i32), seq_len=t(2, dtype=i32), accept_node=t(2, dtype=i32),
              accept_len=t(2, dtype=i32), path=t(2, 5, dtype=i32), bonus=t(2, dtype=i32), held=t(2, dtype=i32),
              last_node=t(2, dtype=i32), n_pages=4, page_size=16)
    with pytest.raises(ValueError, match="GPU"):
        hrs.accept_hold(**ok)
    for bad, err in ((dict(page_table=t(3, 3, dtype=i32)), ValueError), (dict(path=t(10, dtype=i32)), ValueError),
                     (dict(held=t(3, dtype=i32)), ValueError), (dict(held_node=t(2, dtype=f32)), TypeError),
                     (dict(temperature=t(3, dtype=f32)), ValueError), (dict(bonus=None), ValueError),
                     (dict(seq_len=t(4, dtype=i32)[::2]), ValueError)):
        with pytest.raises(err):
            hrs.accept_hold(**{**ok, **bad})

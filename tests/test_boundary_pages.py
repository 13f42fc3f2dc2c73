"""Refusals of kv_pages_reserve and kv_pages_release on the host, as in
test_boundary_attn.py: device pointers are fake, a well-formed call ends in
HRS_EDEVICE."""
import ctypes

import pytest

from tests.test_boundary_attn import call, t
from tests.test_boundary_host import FAKE, MIS, hrs

RESERVE = ["seq_len", "n_new", "prefix_table", "page_table", "n_held", "free_pages", "n_free", "slot_map", "status",
           "workspace"]
RELEASE = ["keep_len", "page_table", "n_held", "free_pages", "n_free", "status", "workspace"]
DESC = dict(n_req=2, n_pos=5, n_pages=8, page_size=16, table_len=4, n_prefix=2)


def reserve(nbytes=1 << 20, **kw):
    return call("kv_pages_reserve", hrs.PagesDesc, RESERVE, DESC, kw, extra=(nbytes,))[0]


def release(nbytes=1 << 20, **kw):
    return call("kv_pages_release", hrs.PagesDesc, RELEASE, DESC, kw, extra=(nbytes,))[0]


@pytest.mark.parametrize("fn,names,optional", [(reserve, RESERVE, ("n_new", "slot_map", "status")),
                                               (release, RELEASE, ("status",))])
def test_rejections(fn, names, optional):
    assert fn() == hrs.HRS_EDEVICE
    assert fn(**{n: None for n in optional}) == hrs.HRS_EDEVICE
    assert fn(n_req=4096, n_pos=1 << 20, page_size=1024, n_prefix=4) == hrs.HRS_EDEVICE
    for bad in (dict(n_req=0), dict(n_req=4097), dict(n_pos=0), dict(n_pos=(1 << 20) + 1), dict(n_pages=0),
                dict(page_size=8), dict(page_size=48), dict(page_size=2048), dict(table_len=0), dict(table_len=1 << 27),
                dict(n_prefix=-1), dict(n_prefix=5), dict(nbytes=24)):
        assert fn(**bad) == hrs.HRS_EINVAL, bad
    for name in names:
        if name not in optional:
            assert fn(**{name: None}) == hrs.HRS_EINVAL, name
        assert fn(**{name: MIS}) == hrs.HRS_EALIGN, name
    d = hrs.PagesDesc(**DESC)
    assert fn(nbytes=hrs.lib.kv_pages_workspace_bytes(ctypes.byref(d))) == hrs.HRS_EDEVICE
    assert fn(nbytes=hrs.lib.kv_pages_workspace_bytes(ctypes.byref(d)) - 1) == hrs.HRS_EINVAL


def test_prefix_goes_with_its_table():
    assert reserve(n_prefix=0) == hrs.HRS_EINVAL
    assert reserve(n_prefix=0, prefix_table=None) == hrs.HRS_EDEVICE
    assert release(n_prefix=0) == hrs.HRS_EDEVICE


def test_no_descriptor_and_workspace_sizes():
    assert hrs.lib.kv_pages_reserve(None, *[FAKE] * 10, 1 << 20, None) == hrs.HRS_EINVAL
    assert hrs.lib.kv_pages_release(None, *[FAKE] * 7, 1 << 20, None) == hrs.HRS_EINVAL
    assert hrs.lib.kv_pages_workspace_bytes(None) == 0
    assert hrs.kv_pages_workspace_bytes(0) == 0 and hrs.kv_pages_workspace_bytes(4097) == 0
    assert 0 < hrs.kv_pages_workspace_bytes(1) < hrs.kv_pages_workspace_bytes(4096)


def args():
    import torch
    i32 = torch.int32
    return dict(page_table=t(4, 3, dtype=i32), n_held=t(4, dtype=i32), free_pages=t(9, dtype=i32), n_free=t(1, dtype=i32),
                workspace=t(4096, dtype=torch.uint8), page_size=16, status=t(4, dtype=i32))


def test_binding_refuses_wrong_tensors():
    import torch
    i32, f32 = torch.int32, torch.float32
    ok = dict(args(), seq_len=t(4, dtype=i32), n_new=t(4, dtype=i32), prefix_table=t(2, dtype=i32),
              slot_map=t(4, 6, dtype=torch.int64))
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_pages_reserve(**ok)
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_pages_reserve(**{**ok, "n_new": None, "prefix_table": None, "slot_map": None, "n_pos": 3})
    for bad, err in ((dict(page_table=t(12, dtype=i32)), ValueError), (dict(n_held=t(3, dtype=i32)), ValueError),
                     (dict(seq_len=t(4, dtype=f32)), TypeError), (dict(n_new=t(5, dtype=i32)), ValueError),
                     (dict(slot_map=t(4, 6, dtype=i32)), TypeError), (dict(slot_map=t(24, dtype=torch.int64)), ValueError),
                     (dict(slot_map=t(4, 6, dtype=torch.int64), n_pos=5), ValueError), (dict(n_free=t(2, dtype=i32)), ValueError),
                     (dict(prefix_table=t(2, 1, dtype=i32)), ValueError), (dict(free_pages=t(3, 3, dtype=i32)), ValueError),
                     (dict(seq_len=None), ValueError), (dict(workspace=None), ValueError)):
        with pytest.raises(err):
            hrs.kv_pages_reserve(**{**ok, **bad})
    for bad in (dict(n_held=ok["seq_len"]), dict(prefix_table=ok["page_table"][0]), dict(status=ok["n_held"]),
                dict(n_free=ok["free_pages"][:1]), dict(workspace=ok["slot_map"])):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.kv_pages_reserve(**{**ok, **bad})
    ok = dict(args(), keep_len=t(4, dtype=i32), n_prefix=2)
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_pages_release(**ok)
    for bad in (dict(n_held=ok["keep_len"]), dict(free_pages=ok["page_table"].view(-1)), dict(status=ok["n_free"])):
        with pytest.raises(ValueError, match="overlaps|status"):
            hrs.kv_pages_release(**{**ok, **bad})

"""Refusals of attn_verify_shared on the host, as in test_boundary_attn.py:
device pointers are fake, a well-formed call ends in HRS_EDEVICE."""
import ctypes

import pytest

from tests.test_boundary_attn import BF, CACHE, CHAIN, F8, F32, TREE, parents, t
from tests.test_boundary_host import FAKE, MIS, hrs

NAMES = ["q", "k", "v", "k_cache", "v_cache", "prefix_table", "prefix_len", "page_table", "seq_len", "k_scale", "v_scale",
         "out", "status", "workspace"]


def shared(ws=None, cache=None, prefix_pages=3, **kw):
    desc = dict(n_req=2, n_pos=4, n_heads=4, n_kvheads=2, d=64, dtype=BF, q_stride=0, k_stride=0, v_stride=0, scale=0.125,
                window=0, cache=hrs.CacheDesc(**{**CACHE, **(cache or {})}), topo=CHAIN, parent=None)
    ptr = {n: FAKE for n in NAMES}
    ptr.update(k_scale=None, v_scale=None)
    for key, val in kw.items():
        (ptr if key in ptr else desc)[key] = val
    if desc["parent"] is not None:
        keep, desc["parent"] = parents(desc["parent"])
    d = hrs.AttnDesc(**desc)
    need = hrs.lib.attn_verify_shared_workspace_bytes(ctypes.byref(d))
    return hrs.lib.attn_verify_shared(ctypes.byref(d), prefix_pages, *ptr.values(), need if ws is None else ws(need), None)


def test_rejections():
    assert shared() == hrs.HRS_EDEVICE and shared(status=None) == hrs.HRS_EDEVICE
    assert shared(cache=dict(dtype=F8), k_scale=FAKE + 4, v_scale=FAKE + 8) == hrs.HRS_EDEVICE
    assert shared(dtype=F32, cache=dict(dtype=F32), n_req=4096) == hrs.HRS_EDEVICE
    assert shared(topo=TREE, parent=[[-1, 0, 0, 2]] * 2, window=3, q_stride=512) == hrs.HRS_EDEVICE
    assert shared(n_req=4096, n_pos=64, n_heads=64, n_kvheads=1, d=256, prefix_pages=1 << 20) == hrs.HRS_EDEVICE
    for bad in (dict(n_req=0), dict(n_req=4097), dict(n_heads=3), dict(n_kvheads=0), dict(n_heads=130), dict(dtype=F8),
                dict(window=-1), dict(q_stride=64), dict(v_stride=-8), dict(topo=5), dict(cache=dict(page_size=8)),
                dict(cache=dict(table_len=0)), dict(cache=dict(dtype=F32)), dict(k_scale=FAKE), dict(workspace=None),
                dict(ws=lambda n: n - 1), dict(prefix_pages=0), dict(prefix_pages=-1), dict(prefix_pages=1 << 27)):
        assert shared(**bad) == hrs.HRS_EINVAL, bad
    for name in NAMES:
        if name not in ("k_scale", "v_scale", "status"):
            assert shared(**{name: None}) == hrs.HRS_EINVAL, name
        if name not in ("k_scale", "v_scale"):
            assert shared(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert shared(cache=dict(dtype=F8), k_scale=FAKE + 2) == hrs.HRS_EALIGN
    for d in (16, 96, 512):
        assert shared(d=d, ws=lambda n: 1 << 40) == hrs.HRS_EUNSUPPORTED
    assert shared(n_pos=0) == shared(n_pos=65) == shared(topo=TREE) == hrs.HRS_EGEOMETRY
    assert hrs.lib.attn_verify_shared(None, 1, *[FAKE] * 14, 1 << 40, None) == hrs.HRS_EINVAL


def test_workspace_sizes():
    assert hrs.attn_verify_shared_workspace_bytes(1, 1, 1, 1, 64) > 0
    for bad in ((0, 1, 4, 2, 64), (1, 65, 4, 2, 64), (1, 1, 5, 2, 64), (1, 1, 4, 2, 80)):
        assert hrs.attn_verify_shared_workspace_bytes(*bad) == 0
    assert hrs.lib.attn_verify_shared_workspace_bytes(None) == 0
    # a launch takes 256 requests at most
    assert hrs.attn_verify_shared_workspace_bytes(256, 4, 8, 2, 64) == hrs.attn_verify_shared_workspace_bytes(4096, 4, 8, 2, 64)


def test_binding_refuses_wrong_tensors():
    import torch
    i32, f32 = torch.int32, torch.float32
    ok = dict(q=t(2, 3, 4, 64), k=t(2, 3, 2, 64), v=t(2, 3, 2, 64), k_cache=t(5, 2, 16, 64), v_cache=t(5, 2, 16, 64),
              prefix_table=t(4, dtype=i32), prefix_len=t(1, dtype=i32), page_table=t(2, 4, dtype=i32),
              seq_len=t(2, dtype=i32), out=t(2, 3, 4, 64), workspace=t(64, dtype=f32), status=t(4, dtype=i32))
    for more in (dict(), dict(prefix_table=ok["page_table"][0]), dict(status=None)):
        with pytest.raises(ValueError, match="GPU"):
            hrs.attn_verify_shared(**{**ok, **more})
    for bad, err in ((dict(prefix_table=t(2, 2, dtype=i32)), ValueError), (dict(prefix_table=None), ValueError),
                     (dict(prefix_len=t(2, dtype=i32)), ValueError), (dict(prefix_len=t(1, dtype=f32)), TypeError),
                     (dict(prefix_table=t(4, dtype=f32)), TypeError), (dict(seq_len=t(3, dtype=i32)), ValueError),
                     (dict(out=t(2, 3, 4, 64, dtype=f32)), TypeError), (dict(k_scale=t(2, dtype=f32)), ValueError)):
        with pytest.raises(err):
            hrs.attn_verify_shared(**{**ok, **bad})
    for bad in (dict(out=ok["q"]), dict(status=ok["prefix_table"]), dict(workspace=ok["k_cache"].view(-1)),
                dict(prefix_len=ok["status"][:1])):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.attn_verify_shared(**{**ok, **bad})

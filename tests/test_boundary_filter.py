"""Refusals of accept_sample_filtered on the host, as in test_boundary_attn.py:
device pointers are fake, a well-formed call ends in HRS_EDEVICE."""
import ctypes

import pytest

from tests.test_boundary_attn import CHAIN, TREE, call, t
from tests.test_boundary_host import FAKE, MIS, hrs

NAMES = ["logits", "tokens", "uniforms", "draft_probs", "temperature", "top_k", "top_p", "min_p", "token_prob",
         "accept_node", "accept_len", "path", "bonus", "status", "workspace"]
OPTIONAL = ("draft_probs", "temperature", "top_k", "top_p", "min_p", "status")
DESC = dict(n_req=2, n_pos=4, vocab=1024, logit_dtype=hrs.HRS_BF16, draft_dtype=hrs.HRS_F32, topo=CHAIN, parent=None)
PAR = [[-1, 0, 0, 2]] * 2


def run(nbytes=1 << 30, **kw):
    return call("accept_sample_filtered", hrs.SampleDesc, NAMES, DESC, kw, extra=(nbytes,))[0]


def test_rejections():
    assert run() == hrs.HRS_EDEVICE
    assert run(**{n: None for n in OPTIONAL}) == hrs.HRS_EDEVICE
    assert run(topo=TREE, parent=PAR, draft_probs=None) == hrs.HRS_EDEVICE
    assert run(topo=TREE, parent=PAR) == hrs.HRS_EUNSUPPORTED
    for bad in (dict(n_req=0), dict(n_req=65536), dict(vocab=0), dict(vocab=1020), dict(logit_dtype=2), dict(draft_dtype=2),
                dict(topo=3), dict(nbytes=1000), dict(vocab=1 << 30, n_req=300)):
        assert run(**bad) == hrs.HRS_EINVAL, bad
    assert run(topo=TREE, draft_probs=None) == hrs.HRS_EGEOMETRY
    assert run(topo=TREE, draft_probs=None, parent=[[-1, 0, 3, 1]] * 2) == hrs.HRS_EGEOMETRY
    assert run(n_pos=0) in (hrs.HRS_EGEOMETRY, hrs.HRS_EINVAL) and run(n_pos=65) in (hrs.HRS_EGEOMETRY, hrs.HRS_EINVAL)
    for name in NAMES:
        if name not in OPTIONAL:
            assert run(**{name: None}) == hrs.HRS_EINVAL, name
        assert run(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert hrs.lib.accept_sample_filtered(None, *[FAKE] * 15, 1 << 30, None) == hrs.HRS_EINVAL


def test_workspace():
    d = hrs.SampleDesc(2, 4, 1024, hrs.HRS_BF16, hrs.HRS_F32, CHAIN, None)
    n = hrs.lib.accept_sample_filtered_workspace_bytes(ctypes.byref(d))
    assert run(nbytes=n) == hrs.HRS_EDEVICE and run(nbytes=n - 1) == hrs.HRS_EINVAL
    assert n == hrs.accept_sample_filtered_workspace_bytes(2, 4, 1024)
    assert hrs.lib.accept_sample_filtered_workspace_bytes(None) == 0 and hrs.accept_sample_filtered_workspace_bytes(1, 1, 12) == 0
    assert hrs.accept_sample_filtered_workspace_bytes(16, 17, 151936) < 64 << 20


def test_binding_refuses_wrong_tensors():
    import torch
    i32, f32 = torch.int32, torch.float32
    ok = dict(logits=t(2, 4, 64), tokens=t(2, 4, dtype=i32), uniforms=t(2, 4, dtype=f32), token_prob=t(2, 4, dtype=f32),
              accept_node=t(2, dtype=i32), accept_len=t(2, dtype=i32), path=t(2, 4, dtype=i32), bonus=t(2, dtype=i32),
              workspace=t(64, dtype=f32), top_k=t(2, dtype=i32), top_p=t(2, dtype=f32), min_p=t(2, dtype=f32),
              draft_probs=t(2, 4, 64, dtype=f32), temperature=t(2, dtype=f32), status=t(4, dtype=i32))
    for more in (dict(), {n: None for n in OPTIONAL}):
        with pytest.raises(ValueError, match="GPU"):
            hrs.accept_sample_filtered(**{**ok, **more})
    for bad, err in ((dict(top_k=t(2, dtype=f32)), TypeError), (dict(top_p=t(2, dtype=torch.float64)), TypeError),
                     (dict(min_p=t(3, dtype=f32)), ValueError), (dict(logits=t(8, 64)), ValueError),
                     (dict(tokens=None), ValueError), (dict(draft_probs=t(2, 4, 32, dtype=f32)), ValueError),
                     (dict(top_p=t(4, dtype=f32)[::2]), ValueError)):
        with pytest.raises(err):
            hrs.accept_sample_filtered(**{**ok, **bad})
    for bad in (dict(bonus=ok["top_k"]), dict(token_prob=ok["uniforms"]), dict(status=ok["accept_len"]),
                dict(min_p=ok["workspace"][4:6])):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.accept_sample_filtered(**{**ok, **bad})

"""Refusals of qk_norm_rope, attn_verify_span, kv_cache_append and
accept_sample on the host, through the C ABI and the binding. As in
test_boundary_host.py: device pointers are fake, a well-formed call ends in
HRS_EDEVICE (no GPU is visible), and the module runs only where none is."""
import ctypes

import numpy as np
import pytest

from tests.test_boundary_host import FAKE, MIS, hrs

CHAIN, TREE = hrs.HRS_CHAIN, hrs.HRS_TREE
BF, F32, F8 = hrs.HRS_BF16, hrs.HRS_F32, hrs.HRS_F8E4M3


def parents(rows):
    arr = np.ascontiguousarray(np.array(rows, dtype=np.int32).reshape(-1))
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def call(fn, struct, names, desc, kw, extra=()):
    desc, ptr = dict(desc), {n: FAKE for n in names}
    keep = None
    for key, val in kw.items():
        if key in ptr:
            ptr[key] = val
        else:
            assert key in desc, key
            desc[key] = val
    if desc.get("parent") is not None:
        keep, desc["parent"] = parents(desc["parent"])
    d = struct(**desc)
    return getattr(hrs.lib, fn)(ctypes.byref(d), *ptr.values(), *extra, None), keep


def rope(**kw):
    names = ["q", "k", "q_weight", "k_weight", "freq", "seq_len", "q_out", "k_out"]
    desc = dict(n_req=2, n_pos=4, n_heads=4, n_kvheads=2, d=64, rot=32, dtype=BF, q_stride=0, k_stride=0, eps=1e-6,
                weight_offset=0.0, interleaved=0, topo=CHAIN, parent=None)
    return call("qk_norm_rope", hrs.QkDesc, names, desc, kw)[0]


def test_rope_rejections():
    assert rope() == hrs.HRS_EDEVICE
    assert rope(q_weight=None, k_weight=None) == hrs.HRS_EDEVICE
    assert rope(rot=0, freq=None) == hrs.HRS_EDEVICE
    assert rope(n_pos=1 << 20) == hrs.HRS_EDEVICE
    assert rope(topo=TREE, parent=[[-1, 0, 0, 2]] * 2) == hrs.HRS_EDEVICE
    for bad in (dict(n_req=0), dict(n_pos=0), dict(n_pos=(1 << 20) + 1), dict(n_heads=0), dict(n_kvheads=0), dict(dtype=F8),
                dict(dtype=7), dict(topo=2), dict(q=None), dict(k=None), dict(freq=None), dict(seq_len=None),
                dict(q_out=None), dict(k_out=None), dict(q_stride=8), dict(q_stride=260), dict(k_stride=-128),
                dict(n_req=17, n_pos=1 << 20)):
        assert rope(**bad) == hrs.HRS_EINVAL, bad
    for bad in (dict(d=8), dict(d=72, rot=16), dict(d=272), dict(rot=24), dict(rot=80), dict(rot=-16)):
        assert rope(**bad) == hrs.HRS_EUNSUPPORTED, bad
    for name in ("q", "k", "q_weight", "k_weight", "freq", "seq_len", "q_out", "k_out"):
        assert rope(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert rope(topo=TREE) == hrs.HRS_EGEOMETRY
    assert rope(topo=TREE, parent=[[-1, 0, 0, 3]] * 2) == hrs.HRS_EGEOMETRY
    assert rope(topo=TREE, n_pos=65, parent=[list(range(-1, 64))] * 2) == hrs.HRS_EGEOMETRY
    assert hrs.lib.qk_norm_rope(None, *[FAKE] * 8, None) == hrs.HRS_EINVAL


CACHE = dict(n_pages=8, page_size=16, table_len=4, dtype=BF)


def attn(ws=None, cache=None, **kw):
    names = ["q", "k", "v", "k_cache", "v_cache", "page_table", "seq_len", "k_scale", "v_scale", "out", "status", "workspace"]
    desc = dict(n_req=2, n_pos=4, n_heads=4, n_kvheads=2, d=64, dtype=BF, q_stride=0, k_stride=0, v_stride=0, scale=0.125,
                window=0, cache=hrs.CacheDesc(**{**CACHE, **(cache or {})}), topo=CHAIN, parent=None)
    kw = {"k_scale": None, "v_scale": None, **kw}
    d = hrs.AttnDesc(**{**desc, **{k: v for k, v in kw.items() if k in desc and k != "parent"}})
    need = hrs.lib.attn_verify_span_workspace_bytes(ctypes.byref(d))
    return call("attn_verify_span", hrs.AttnDesc, names, desc, kw, (need if ws is None else ws(need),))[0]


def test_attn_rejections():
    assert attn() == hrs.HRS_EDEVICE
    assert attn(status=None) == hrs.HRS_EDEVICE
    assert attn(cache=dict(dtype=F8), k_scale=FAKE + 4, v_scale=FAKE + 8) == hrs.HRS_EDEVICE
    assert attn(dtype=F32, cache=dict(dtype=F32)) == hrs.HRS_EDEVICE
    assert attn(topo=TREE, parent=[[-1, 0, 0, 2]] * 2, window=3, q_stride=512, k_stride=512, v_stride=512) == hrs.HRS_EDEVICE
    for bad in (dict(n_req=0), dict(n_req=4097), dict(n_heads=3), dict(n_heads=0), dict(n_kvheads=0), dict(n_heads=130),
                dict(dtype=F8), dict(window=-1), dict(q_stride=64), dict(k_stride=132), dict(v_stride=-8), dict(topo=5),
                dict(cache=dict(page_size=8)), dict(cache=dict(page_size=48)), dict(cache=dict(page_size=2048)),
                dict(cache=dict(n_pages=0)), dict(cache=dict(table_len=0)), dict(cache=dict(dtype=F32)),
                dict(cache=dict(table_len=1 << 27)), dict(dtype=F32), dict(dtype=F32, cache=dict(dtype=F8)),
                dict(k_scale=FAKE), dict(v_scale=FAKE), dict(workspace=None), dict(ws=lambda n: n - 1)):
        assert attn(**bad) == hrs.HRS_EINVAL, bad
    for name in ("q", "k", "v", "k_cache", "v_cache", "page_table", "seq_len", "out"):
        assert attn(**{name: None}) == hrs.HRS_EINVAL, name
        assert attn(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert attn(workspace=MIS) == hrs.HRS_EALIGN
    assert attn(cache=dict(dtype=F8), k_scale=FAKE + 2) == hrs.HRS_EALIGN
    for d in (16, 96, 512):
        assert attn(d=d, ws=lambda n: 1 << 40) == hrs.HRS_EUNSUPPORTED
    for n in (0, 65):
        assert attn(n_pos=n) == hrs.HRS_EGEOMETRY
    assert attn(topo=TREE) == hrs.HRS_EGEOMETRY
    assert attn(topo=TREE, parent=[[-1, 0, 0, 2], [-1, 0, -1, 2]]) == hrs.HRS_EGEOMETRY
    assert hrs.lib.attn_verify_span(None, *[FAKE] * 12, 1 << 40, None) == hrs.HRS_EINVAL


def test_attn_workspace_sizes():
    assert hrs.attn_verify_span_workspace_bytes(1, 17, 24, 4, 256) > 0
    for bad in ((0, 1, 4, 2, 64), (1, 65, 4, 2, 64), (1, 1, 5, 2, 64), (1, 1, 4, 2, 80)):
        assert hrs.attn_verify_span_workspace_bytes(*bad) == 0
    assert hrs.lib.attn_verify_span_workspace_bytes(None) == 0


def append(cache=None, **kw):
    names = ["k", "v", "k_cache", "v_cache", "page_table", "seq_len", "accept_len", "path", "k_scale", "v_scale",
             "seq_len_out", "status"]
    desc = dict(n_layers=2, n_req=3, n_pos=5, n_kvheads=2, d=64, dtype=BF, k_stride=0, v_stride=0,
                cache=hrs.CacheDesc(**{**CACHE, **(cache or {})}))
    return call("kv_cache_append", hrs.AppendDesc, names, desc, {"k_scale": None, "v_scale": None, **kw})[0]


def test_append_rejections():
    assert append() == hrs.HRS_EDEVICE
    assert append(path=None, seq_len_out=None, status=None, n_pos=1 << 20) == hrs.HRS_EDEVICE
    assert append(cache=dict(dtype=F8), k_scale=FAKE + 4, seq_len_out=FAKE + 64) == hrs.HRS_EDEVICE
    for bad in (dict(n_layers=0), dict(n_layers=65536), dict(n_req=0), dict(n_req=65536), dict(n_pos=0), dict(n_pos=65),
                dict(path=None, n_pos=(1 << 20) + 1), dict(path=None, n_pos=1 << 20, n_req=17), dict(n_kvheads=0),
                dict(dtype=F8), dict(k_stride=64), dict(v_stride=132), dict(cache=dict(page_size=20)), dict(cache=dict(dtype=F32)),
                dict(k_scale=FAKE), dict(v_scale=FAKE)):
        assert append(**bad) == hrs.HRS_EINVAL, bad
    assert append(n_req=5, seq_len_out=FAKE + 16) == hrs.HRS_EINVAL     # overlaps seq_len without being it
    assert append(n_req=5, seq_len=FAKE + 16, seq_len_out=FAKE) == hrs.HRS_EINVAL
    assert append(n_req=4, seq_len_out=FAKE + 16) == hrs.HRS_EDEVICE
    for name in ("k", "v", "k_cache", "v_cache", "page_table", "seq_len", "accept_len"):
        assert append(**{name: None}) == hrs.HRS_EINVAL, name
    for name in ("k", "v", "k_cache", "v_cache", "page_table", "seq_len", "accept_len", "path", "seq_len_out", "status"):
        assert append(**{name: MIS}) == hrs.HRS_EALIGN, name
    for d in (8, 72, 272):
        assert append(d=d) == hrs.HRS_EUNSUPPORTED


def sample(ws=None, **kw):
    names = ["logits", "tokens", "uniforms", "draft_probs", "temperature", "token_prob", "accept_node", "accept_len", "path",
             "bonus", "status", "workspace"]
    desc = dict(n_req=2, n_pos=4, vocab=64, logit_dtype=BF, draft_dtype=F32, topo=CHAIN, parent=None)
    d = hrs.SampleDesc(**{**desc, **{k: v for k, v in kw.items() if k in desc and k != "parent"}})
    need = hrs.lib.accept_sample_workspace_bytes(ctypes.byref(d))
    return call("accept_sample", hrs.SampleDesc, names, desc, kw, (need if ws is None else ws(need),))[0]


def test_sample_rejections():
    tree = dict(topo=TREE, parent=[[-1, 0, 0, 2]] * 2)
    assert sample() == hrs.HRS_EDEVICE
    assert sample(draft_probs=None, temperature=None, status=None, draft_dtype=9) == hrs.HRS_EDEVICE
    assert sample(draft_probs=None, **tree) == hrs.HRS_EDEVICE
    assert sample(**tree) == hrs.HRS_EUNSUPPORTED
    for bad in (dict(n_req=0), dict(n_req=65536, n_pos=1), dict(vocab=0), dict(vocab=12), dict(logit_dtype=F8), dict(draft_dtype=F8),
                dict(topo=3), dict(workspace=None), dict(ws=lambda n: n - 1), dict(n_req=60000, n_pos=64, vocab=151936)):
        assert sample(**bad) == hrs.HRS_EINVAL, bad
    for name in ("logits", "tokens", "uniforms", "token_prob", "accept_node", "accept_len", "path", "bonus"):
        assert sample(**{name: None}) == hrs.HRS_EINVAL, name
    for name in ("logits", "tokens", "uniforms", "draft_probs", "temperature", "token_prob", "accept_node", "accept_len", "path",
                 "bonus", "status", "workspace"):
        assert sample(**{name: MIS}) == hrs.HRS_EALIGN, name
    assert sample(n_pos=0) == hrs.HRS_EGEOMETRY and sample(n_pos=65) == hrs.HRS_EGEOMETRY
    assert sample(topo=TREE, draft_probs=None) == hrs.HRS_EGEOMETRY
    assert sample(topo=TREE, draft_probs=None, parent=[[-1, 0, 0, 2], [-1, 0, 4, 2]]) == hrs.HRS_EGEOMETRY
    assert hrs.accept_sample_workspace_bytes(1, 17, 151936) > 0 and hrs.accept_sample_workspace_bytes(1, 17, 12) == 0


# --- the binding, on CPU tensors: everything but the device is checked first ------

def t(*shape, dtype=None):
    import torch
    return torch.zeros(shape, dtype=dtype or torch.bfloat16)


def test_binding_refuses_wrong_tensors():
    import torch
    i32, f32, f64, f8 = torch.int32, torch.float32, torch.float64, torch.float8_e4m3fn
    ok = dict(q=t(2, 3, 4, 64), k=t(2, 3, 2, 64), q_weight=t(64), k_weight=t(64), freq=t(16, dtype=f64), seq_len=t(2, dtype=i32),
              q_out=t(2, 3, 4, 64), k_out=t(2, 3, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        hrs.qk_norm_rope(**ok)
    for bad, err in ((dict(q=t(2, 3, 256)), ValueError), (dict(k=t(2, 4, 2, 64)), ValueError), (dict(k=t(2, 3, 2, 64, dtype=f32)), TypeError),
                     (dict(freq=t(16, dtype=f32)), TypeError), (dict(seq_len=t(3, dtype=i32)), ValueError), (dict(q=None), ValueError),
                     (dict(q_out=t(2, 3, 64, 4).transpose(2, 3)), ValueError), (dict(q=t(2, 3, 64, 4).transpose(2, 3)), ValueError),
                     (dict(q=t(3, 2, 4, 64).transpose(0, 1)), ValueError), (dict(q=t(2, 3, 4, 68)[..., :64]), ValueError),
                     (dict(q=t(2, 3, 260)[..., :256].unflatten(-1, (4, 64))), ValueError), (dict(q=t(1, 1, 4, 64).expand(2, 3, 4, 64)), ValueError),
                     (dict(q_weight=t(32)), ValueError), (dict(parent=[-1, 0]), ValueError)):
        with pytest.raises(err):
            hrs.qk_norm_rope(**{**ok, **bad})
    with pytest.raises(ValueError, match="GPU"):     # a view of a wider projection is fine
        hrs.qk_norm_rope(**{**ok, "q": t(2, 3, 512)[..., :256].unflatten(-1, (4, 64))})

    ok = dict(q=t(2, 3, 4, 64), k=t(2, 3, 2, 64), v=t(2, 3, 2, 64), k_cache=t(5, 2, 16, 64), v_cache=t(5, 2, 16, 64),
              page_table=t(2, 3, dtype=i32), seq_len=t(2, dtype=i32), out=t(2, 3, 4, 64), workspace=t(64, dtype=f32))
    with pytest.raises(ValueError, match="GPU"):
        hrs.attn_verify_span(**ok)
    for bad, err in ((dict(v=t(2, 3, 1, 64)), ValueError), (dict(v_cache=t(5, 2, 32, 64)), ValueError), (dict(k_cache=t(5, 1, 16, 64)), ValueError),
                     (dict(k_cache=t(5, 2, 16, 64, dtype=f32)), TypeError), (dict(v_cache=t(5, 2, 16, 64).to(f8)), TypeError),
                     (dict(page_table=t(3, 3, dtype=i32)), ValueError), (dict(page_table=t(2, dtype=i32)), ValueError),
                     (dict(k_scale=t(2, dtype=f32)), ValueError), (dict(out=t(2, 3, 4, 64, dtype=f32)), TypeError),
                     (dict(workspace=None), ValueError), (dict(status=t(1, dtype=f32)), TypeError)):
        with pytest.raises(err):
            hrs.attn_verify_span(**{**ok, **bad})

    ok = dict(k=t(2, 2, 3, 2, 64), v=t(2, 2, 3, 2, 64), k_cache=t(2, 5, 2, 16, 64), v_cache=t(2, 5, 2, 16, 64),
              page_table=t(2, 3, dtype=i32), seq_len=t(2, dtype=i32), accept_len=t(2, dtype=i32))
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_cache_append(**ok)
    for bad, err in ((dict(v=t(2, 2, 3, 1, 64)), ValueError), (dict(k_cache=t(1, 5, 2, 16, 64)), ValueError), (dict(path=t(2, 4, dtype=i32)), ValueError),
                     (dict(accept_len=t(2, dtype=f32)), TypeError), (dict(seq_len_out=t(3, dtype=i32)), ValueError),
                     (dict(k_scale=t(2, 2, dtype=f32)), ValueError)):
        with pytest.raises(err):
            hrs.kv_cache_append(**{**ok, **bad})

    ok = dict(logits=t(2, 3, 64), tokens=t(2, 3, dtype=i32), uniforms=t(2, 3, dtype=f32), token_prob=t(2, 3, dtype=f32),
              accept_node=t(2, dtype=i32), accept_len=t(2, dtype=i32), path=t(2, 3, dtype=i32), bonus=t(2, dtype=i32),
              workspace=t(64, dtype=f32))
    with pytest.raises(ValueError, match="GPU"):
        hrs.accept_sample(**ok)
    for bad, err in ((dict(uniforms=t(2, 3, dtype=f64)), TypeError), (dict(draft_probs=t(2, 3, 32, dtype=f32)), ValueError),
                     (dict(draft_probs=t(2, 3, 64, dtype=f64)), TypeError), (dict(temperature=t(1, dtype=f32)), ValueError),
                     (dict(tokens=t(2, 3, dtype=torch.int64)), TypeError), (dict(parent=[[-1, 0]]), ValueError)):
        with pytest.raises(err):
            hrs.accept_sample(**{**ok, **bad})


def test_binding_refuses_outputs_over_inputs():
    """Blocks write their part of an output while others still read: only a
    whole dense side of qk_norm_rope may be its own output."""
    import torch
    n, f = t(2, dtype=torch.int32), t(16, dtype=torch.float64)
    buf = t(4096)
    at = lambda o, *s: buf[o:o + int(np.prod(s))].view(*s)
    q, k = at(0, 2, 3, 4, 64), at(1536, 2, 3, 2, 64)
    qo, ko = t(2, 3, 4, 64), t(2, 3, 2, 64)
    rope = lambda q, k, qo, ko: hrs.qk_norm_rope(q, k, None, None, f, n, qo, ko)
    for ok in ((q, k, q, ko), (q, k, qo, k), (q, k, q, k), (q, k, at(2304, 2, 3, 4, 64), ko)):
        with pytest.raises(ValueError, match="GPU"):
            rope(*ok)
    packed = t(2, 3, 512)
    qp = packed[..., :256].unflatten(-1, (4, 64))
    for bad in ((q, k, at(8, 2, 3, 4, 64), ko), (q, k, at(1528, 2, 3, 4, 64), ko), (q, k, qo, at(1000, 2, 3, 2, 64)),
                (q, k, qo, qo.view(-1)[:768].view(2, 3, 2, 64)), (qp, k, packed.view(-1)[:1536].view(2, 3, 4, 64), ko)):
        with pytest.raises(ValueError, match="overlaps"):
            rope(*bad)
    kc, pt, ws = t(5, 2, 16, 64), t(2, 3, dtype=torch.int32), t(64, dtype=torch.float32)
    v = t(2, 3, 2, 64)
    for out in (q, at(8, 2, 3, 4, 64), at(1600, 2, 3, 4, 64)):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.attn_verify_span(q, k, v, kc, kc, pt, n, out, ws)

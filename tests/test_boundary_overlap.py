"""The binding refuses buffers that a call writes over ones that it reads: some
blocks write while others still read. CPU tensors: everything but the device
is checked first."""
import pytest

from tests.test_boundary_attn import t
from tests.test_boundary_host import hrs


def append_args():
    import torch
    i32 = torch.int32
    return dict(k=t(2, 4, 5, 2, 64), v=t(2, 4, 5, 2, 64), k_cache=t(2, 5, 2, 16, 64), v_cache=t(2, 5, 2, 16, 64),
                page_table=t(4, 4, dtype=i32), seq_len=t(4, dtype=i32), accept_len=t(4, dtype=i32),
                seq_len_out=t(4, dtype=i32), path=t(4, 5, dtype=i32), status=t(4, dtype=i32))


def test_append_refuses_written_buffers_over_others():
    ok = append_args()
    for more in (dict(), dict(seq_len_out=ok["seq_len"]), dict(seq_len_out=None, status=None, path=None), dict(v=ok["k"])):
        with pytest.raises(ValueError, match="GPU"):
            hrs.kv_cache_append(**{**ok, **more})
    n = ok["seq_len"]
    for bad in (dict(seq_len_out=ok["accept_len"]), dict(seq_len_out=ok["path"].view(-1)[4:8]),
                dict(seq_len_out=ok["page_table"][1]), dict(status=ok["accept_len"]), dict(status=n),
                dict(status=ok["seq_len_out"]), dict(status=n, seq_len_out=n), dict(v_cache=ok["k_cache"]),
                dict(k=ok["k_cache"].view(-1)[:5120].view(2, 4, 5, 2, 64)),
                dict(v=ok["k_cache"].view(-1)[512:5632].view(2, 4, 5, 2, 64))):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.kv_cache_append(**{**ok, **bad})
    both = t(12, dtype=n.dtype)
    with pytest.raises(ValueError, match="overlaps"):
        hrs.kv_cache_append(**{**ok, "seq_len": both[:4], "seq_len_out": both[2:6]})
    with pytest.raises(ValueError, match="overlaps"):
        hrs.kv_cache_append(**{**ok, "accept_len": both[:4], "seq_len_out": both[3:7]})
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_cache_append(**{**ok, "seq_len": both[:4], "seq_len_out": both[4:8], "accept_len": both[8:]})


def test_sample_refuses_outputs_over_inputs_or_each_other():
    import torch
    i32, f32 = torch.int32, torch.float32
    ok = dict(logits=t(2, 4, 64), tokens=t(2, 4, dtype=i32), uniforms=t(2, 4, dtype=f32), token_prob=t(2, 4, dtype=f32),
              accept_node=t(2, dtype=i32), accept_len=t(2, dtype=i32), path=t(2, 4, dtype=i32), bonus=t(2, dtype=i32),
              workspace=t(64, dtype=f32), draft_probs=t(2, 4, 64, dtype=f32), temperature=t(2, dtype=f32),
              status=t(4, dtype=i32))
    for more in (dict(), dict(draft_probs=None, temperature=None, status=None), dict(draft_probs=ok["logits"])):
        with pytest.raises(ValueError, match="GPU"):
            hrs.accept_sample(**{**ok, **more})
    for bad in (dict(path=ok["tokens"]), dict(token_prob=ok["uniforms"]), dict(accept_node=ok["accept_len"]),
                dict(bonus=ok["tokens"][1, :2]), dict(status=ok["bonus"]), dict(workspace=ok["draft_probs"].view(-1)),
                dict(temperature=ok["token_prob"][0, :2])):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.accept_sample(**{**ok, **bad})


def test_hold_refuses_written_buffers_over_others():
    import torch
    i32 = torch.int32
    ok = dict(page_table=t(2, 3, dtype=i32), seq_len=t(2, dtype=i32), accept_node=t(2, dtype=i32),
              accept_len=t(2, dtype=i32), path=t(2, 5, dtype=i32), bonus=t(2, dtype=i32), held=t(2, dtype=i32),
              last_node=t(2, dtype=i32), n_pages=4, page_size=16, held_node=t(2, dtype=i32))
    with pytest.raises(ValueError, match="GPU"):
        hrs.accept_hold(**ok)
    for bad in (dict(held=ok["seq_len"]), dict(held_node=ok["last_node"]), dict(bonus=ok["path"][1, :2]),
                dict(last_node=ok["page_table"][0, 1:])):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.accept_hold(**{**ok, **bad})


def test_attention_layer_calls_refuse_outputs_over_any_input():
    import torch
    i32, f32, f64 = torch.int32, torch.float32, torch.float64
    ok = dict(q=t(2, 3, 4, 64), k=t(2, 3, 2, 64), q_weight=t(64), k_weight=t(64), freq=t(16, dtype=f64), seq_len=t(2, dtype=i32),
              q_out=t(2, 3, 4, 64), k_out=t(2, 3, 2, 64))
    for more in (dict(), dict(q_out=ok["q"]), dict(q_out=ok["q"], k_out=ok["k"]), dict(k_weight=ok["q_weight"])):
        with pytest.raises(ValueError, match="GPU"):
            hrs.qk_norm_rope(**{**ok, **more})
    for bad in (dict(q_weight=ok["q_out"].view(-1)[64:128]), dict(freq=ok["k_out"].view(f64).view(-1)[:16]),
                dict(q_out=ok["q"], q_weight=ok["q"].view(-1)[64:128]), dict(seq_len=ok["q_out"].view(i32).view(-1)[:2])):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.qk_norm_rope(**{**ok, **bad})
    ok = dict(q=t(2, 3, 4, 64), k=t(2, 3, 2, 64), v=t(2, 3, 2, 64), k_cache=t(5, 2, 16, 64), v_cache=t(5, 2, 16, 64),
              page_table=t(2, 3, dtype=i32), seq_len=t(4, dtype=i32)[:2], out=t(2, 3, 4, 64), workspace=t(64, dtype=f32),
              status=t(4, dtype=i32))
    for more in (dict(), dict(status=None), dict(v=ok["k"], v_cache=ok["k_cache"])):
        with pytest.raises(ValueError, match="GPU"):
            hrs.attn_verify_span(**{**ok, **more})
    for bad in (dict(status=ok["seq_len"]), dict(workspace=ok["out"].view(-1)), dict(page_table=ok["out"].view(i32).view(-1)[:6].view(2, 3)),
                dict(out=ok["v_cache"].view(-1)[:1536].view(2, 3, 4, 64)), dict(status=ok["workspace"].view(i32))):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.attn_verify_span(**{**ok, **bad})

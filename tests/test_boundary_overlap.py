"""The binding refuses buffers that a call writes over ones that it reads: some
blocks write while others still read. CPU tensors: everything but the device
is checked first."""
import pytest

from tests.test_boundary_attn import t
from tests.test_boundary_host import hrs


def append_args():
    import torch
    i32 = torch.int32
    return dict(k=t(2, 4, 3, 2, 64), v=t(2, 4, 3, 2, 64), k_cache=t(2, 5, 2, 16, 64), v_cache=t(2, 5, 2, 16, 64),
                page_table=t(4, 4, dtype=i32), seq_len=t(4, dtype=i32), accept_len=t(4, dtype=i32),
                seq_len_out=t(4, dtype=i32), path=t(4, 3, dtype=i32), status=t(4, dtype=i32))


def test_append_refuses_written_buffers_over_others():
    ok = append_args()
    for more in (dict(), dict(seq_len_out=ok["seq_len"]), dict(seq_len_out=None, status=None, path=None), dict(v=ok["k"])):
        with pytest.raises(ValueError, match="GPU"):
            hrs.kv_cache_append(**{**ok, **more})
    n = ok["seq_len"]
    for bad in (dict(seq_len_out=ok["accept_len"]), dict(seq_len_out=ok["path"].view(-1)[4:8]),
                dict(seq_len_out=ok["page_table"][1]), dict(status=ok["accept_len"]), dict(status=n),
                dict(status=ok["seq_len_out"]), dict(status=n, seq_len_out=n), dict(v_cache=ok["k_cache"]),
                dict(k=ok["k_cache"].view(-1)[:3072].view(2, 4, 3, 2, 64)),
                dict(v=ok["k_cache"].view(-1)[512:3584].view(2, 4, 3, 2, 64))):
        with pytest.raises(ValueError, match="overlaps"):
            hrs.kv_cache_append(**{**ok, **bad})
    both = t(12, dtype=n.dtype)
    with pytest.raises(ValueError, match="overlaps"):
        hrs.kv_cache_append(**{**ok, "seq_len": both[:4], "seq_len_out": both[2:6]})
    with pytest.raises(ValueError, match="overlaps"):
        hrs.kv_cache_append(**{**ok, "accept_len": both[:4], "seq_len_out": both[3:7]})
    with pytest.raises(ValueError, match="GPU"):
        hrs.kv_cache_append(**{**ok, "seq_len": both[:4], "seq_len_out": both[4:8], "accept_len": both[8:]})

"""Verify steps of a hybrid model: GDN layers with attention layers between
them. The GDN side must be bit for bit what FusedVerifyStep gives for the same
acceptance; attention, the pages and the lengths are checked against the
oracle run on the same history; replays of the captured step equal eager steps
bit for bit."""
import numpy as np
import pytest

from oracle import attn as oa
from oracle import sample as osm
from oracle.common import widen
from synth import QWEN_STACK_CHAIN, QWEN_STACK_TREE, scaled
from tests.gpu_util import say
from tests.test_gpu_attn import Attn, OUT, U, dev, host

pytestmark = pytest.mark.gpu

SMALL = dict(n_layers=3, n_req=2, vocab=512, n_kheads=2, n_vheads=4, conv_channels=2 * 2 * 128 + 4 * 128)
WORKLOADS = [scaled(QWEN_STACK_CHAIN, ring_slots=0, ring_width=0, **SMALL), scaled(QWEN_STACK_TREE, **SMALL)]


def make(w, sample, f8=False, hybrid=True):
    """Step and buffers, filled the same way on every call."""
    import torch
    from hybrid_recurrent_state_amd.step import AttnBuffers, AttnShape, FusedVerifyStep, HybridVerifyStep, StepBuffers
    from synth.device import fill_step, step_shape
    bufs = StepBuffers(step_shape(w))
    loaded = fill_step(bufs, w)
    if not hybrid:
        return bufs, None, FusedVerifyStep(bufs, parent=loaded.parent), loaded
    shape = AttnShape(2, 4, 2, 64, 32, n_pages=12, page_size=32, table_len=5, theta=100.0, f8_cache=f8)
    a = AttnBuffers(shape, bufs.shape)
    rng = np.random.default_rng(5)
    fill = lambda t, gain: t.copy_(torch.from_numpy((rng.standard_normal(tuple(t.shape)) * gain).astype(np.float32)))
    fill(a.qkv, 1.0)
    a.q_weight.copy_(a.q_weight + fill(torch.empty(2, 64), 0.1).to(a.q_weight))
    if f8:
        a.k_scale.fill_(0.02)
        a.v_scale.fill_(0.015)
    a.page_table.copy_(torch.from_numpy(rng.permutation(12)[:10].reshape(2, 5).astype(np.int32)))
    a.uniforms.copy_(torch.from_numpy((rng.random((2, w.n_pos)) * 0.2).astype(np.float32)))
    a.temperature.copy_(torch.tensor([0.7, 1.3]))
    return bufs, a, HybridVerifyStep(bufs, a, parent=loaded.parent, sample=sample), loaded


def refill(bufs, a, i, sample, parent):
    """New projections, logits and random numbers of step i (device, seeded).
    Drafted tokens get some probability, so that paths of several lengths are
    accepted."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(100 + i)
    a.qkv.normal_(generator=g)
    if sample:
        bufs.logits.normal_(generator=g)
        a.uniforms.uniform_(0.0, 0.2, generator=g)
        R, T = bufs.tokens.shape
        tok = bufs.tokens.tolist()
        for r in range(R):
            for t in range(1, T):
                node = t - 1 if parent is None else int(parent[r][t])
                bufs.logits[r, node, tok[r][t]] += 5.0


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("sample", [False, True])
@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_hybrid_steps(w, sample, f8):
    import torch
    bufs, a, step, loaded = make(w, sample, f8)
    plain_bufs, _, plain, _ = make(w, sample, hybrid=False)
    par = loaded.parent
    for i in range(3):
        refill(bufs, a, i, sample, loaded.parent)
        lens = a.seq_len.tolist()
        before = [host(c).copy() for c in (a.k_cache, a.v_cache)]
        acc, bonus = step.run()
        # the GDN side
        if not sample:
            acc_p, bonus_p = plain.run()
            assert np.array_equal(acc, acc_p) and np.array_equal(bonus, bonus_p)
            for name in ("out", "conv_state", "accept_node", "path"):
                assert np.array_equal(host(getattr(bufs, name)), host(getattr(plain_bufs, name))), (i, name)
            assert np.array_equal(host(step.current_ckpt()), host(plain.current_ckpt())), i
        # acceptance
        path = host(bufs.path)
        if sample:
            for r in range(2):
                ref = osm.accept(host(bufs.logits)[r], host(bufs.tokens)[r], host(a.uniforms)[r],
                                 parent=None if par is None else par[r], tau=float(a.temperature[r]))
                assert np.array_equal(path[r], ref.path) and int(acc[r]) == ref.accept_len
                assert int(bonus[r]) == ref.bonus and int(bufs.accept_node[r]) == ref.path[ref.accept_len]
        # attention
        qh, kh, vh = host(a.q_out), host(a.k_out), host(a.v.contiguous())
        for l in range(2):
            for r in range(2):
                c = Attn(1, w.n_pos, 4, 2, 64, 32, [lens[r]], "bf16", "f8" if f8 else "bf16")
                c.q, c.k, c.v = qh[l, r][None], kh[l, r][None], vh[l, r][None]
                c.kc, c.vc, c.N, c.pages = before[0][l], before[1][l], 12, host(a.page_table)[r][None]
                c.ks, c.vs = (host(s)[l] if f8 else None for s in (a.k_scale, a.v_scale))
                c.parent = None if par is None else par[r][None]
                c.check(a.out[l, r][None], what=f"step {i}")
                dep = range(w.n_pos) if par is None else oa.depths(par[r])
                ref = oa.norm_rope(host(a.q.contiguous())[l, r], host(a.q_weight)[l], host(a.freq), lens[r], dep, 1e-6)
                size = np.abs(oa.norm_rope(host(a.q.contiguous())[l, r], host(a.q_weight)[l], [], lens[r], dep, 1e-6))
                size[..., :16] = size[..., 16:32] = size[..., :16] + size[..., 16:32]
                tol = 32 * U * size * (1 + OUT["bf16"]) + OUT["bf16"] * np.abs(ref)
                assert np.all(np.abs(widen(qh[l, r]) - ref) <= tol)
                # the pages after the step
                for rows, b, s in ((kh, before[0], c.ks), (vh, before[1], c.vs)):
                    src = oa.quantize_e4m3(widen(rows[l, r]), s) if f8 else rows[l, r]
                    oa.append(src, b[l], c.pages[0], lens[r], path[r], int(acc[r]) + 1)
        for c, b in zip((a.k_cache, a.v_cache), before):
            assert np.array_equal(host(c), b)
        assert a.seq_len.tolist() == [n + int(x) + 1 for n, x in zip(lens, acc)]
        assert int(a.status[:, 0].abs().sum()) == 0
        say(f"step {i}: accepted {list(map(int, acc))}")


@pytest.mark.parametrize("sample", [False, True])
@pytest.mark.parametrize("w", WORKLOADS, ids=["chain", "tree"])
def test_hybrid_graph_replays(w, sample):
    import torch
    e_bufs, ea, eager, _ = make(w, sample)
    g_bufs, ga, graphed, loaded = make(w, sample)
    graphed.capture_graph()
    scratch = torch.randn(1 << 20, device="cuda")
    for i in range(5):
        refill(e_bufs, ea, i, sample, loaded.parent)
        refill(g_bufs, ga, i, sample, loaded.parent)
        assert all(np.array_equal(x, y) for x, y in zip(eager.run(), graphed.replay())), i
        for x, y in ((e_bufs.path, g_bufs.path), (e_bufs.out, g_bufs.out), (e_bufs.conv_state, g_bufs.conv_state),
                     (ea.q_out, ga.q_out), (ea.out, ga.out), (ea.k_cache, ga.k_cache), (ea.v_cache, ga.v_cache),
                     (ea.seq_len, ga.seq_len), (eager.current_ckpt(), graphed.current_ckpt())):
            assert np.array_equal(host(x), host(y)), i
        scratch.mul_(1.0001).add_(0.5)
        torch.cuda.synchronize()


def test_hybrid_layer_order_is_checked():
    from hybrid_recurrent_state_amd.step import AttnBuffers, AttnShape, HybridVerifyStep, StepBuffers
    from synth.device import step_shape
    bufs = StepBuffers(step_shape(WORKLOADS[0]))
    for after in ([2, 1], [0], [0, 3]):
        a = AttnBuffers(AttnShape(2, 4, 2, 64, 32, 12, 32, 5, after=after), bufs.shape)
        with pytest.raises(ValueError, match="after"):
            HybridVerifyStep(bufs, a)

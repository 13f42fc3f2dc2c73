"""One verify step over a stack of GDN layers, on one stream, one host sync.

Order of the step (all on the caller's stream):
  for each layer: conv1d_verify_span, then gdn_verify_span (checkpoints on)
  accept_greedy over the target logits
  rollback_restore of every layer to the accepted position (index stays on
  the device)
  ring_set_2d, ring_get_2d of the step's hidden-feature rows
then one device-to-host copy of the accepted lengths and bonus tokens,
which is the step's only synchronisation (lucebox PR #533, "feat: DFlash
support for tensor-parallel Qwen3.6 targets", Changes: restore SSM and conv
state on device and synchronize once after rollback).

Buffers are allocated once by ``StepBuffers`` (device memory through torch)
and every descriptor and pointer of the step is computed once by
``VerifyStep``, so launching a step is a fixed sequence of C calls.

Variants: ``ZeroCopyVerifyStep`` starts
each span from the previous span's accepted checkpoint in place (no rollback
copy, conv state rebuilt from the accepted path) and ``FusedVerifyStep`` adds
one fused kernel per layer (conv, SiLU, q/k/v split, q/k L2 norm and the
gated delta rule) to it. ``HybridVerifyStep`` adds the model's attention
layers between the GDN layers (norm and rotation, attention over a paged
cache, accepted rows into the pages) and acceptance by sampling; also for
requests that share a prefix, whose page tables grow from a free list and that
sample after top-k, top-p and min-p.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import List, Optional, Sequence

import numpy as np

from . import (AcceptDesc, ConvAdvanceDesc, ConvDesc, GdnDesc, GdnLayerDesc, HRS_BF16, HRS_CHAIN, HRS_F32, HRS_TREE,
               HrsError, RingDesc, RingRun, RollbackDesc, SpanSource, accept_greedy_workspace_bytes, accept_hold_behind_call,
               accept_sample_call, accept_sample_filtered_call, accept_sample_filtered_workspace_bytes,
               accept_sample_workspace_bytes, attn_verify_shared_call, attn_verify_shared_workspace_bytes,
               attn_verify_span_call, attn_verify_span_workspace_bytes, kv_cache_append_call, kv_pages_release_call,
               kv_pages_reserve_step_call, kv_pages_workspace_bytes, lib, qk_norm_rope_call)


@dataclasses.dataclass(frozen=True)
class StepShape:
    n_layers: int
    n_req: int
    n_pos: int
    n_kheads: int
    n_vheads: int
    d_k: int
    d_v: int
    bf16: bool                 # q/k/v/a/b and conv dtype (state is always f32)
    conv_channels: int
    conv_width: int = 4
    vocab: int = 0             # 0: no logits; accept_node is provided directly
    ring_slots: int = 0        # 0: no feature ring
    ring_width: int = 0

    @property
    def gdn_bytes_per_layer(self) -> int:
        """Algorithmic HBM bytes of one gdn_verify_span call with capture:
        read q, k, v, a, b and the state once; write every checkpoint and
        every output once."""
        R, T, Hk, Hv, dk, dv = self.n_req, self.n_pos, self.n_kheads, self.n_vheads, self.d_k, self.d_v
        e = 2 if self.bf16 else 4
        reads = R * T * (2 * Hk * dk + Hv * dv + 2 * Hv) * e + R * Hv * dv * dk * 4
        writes = R * T * Hv * dv * dk * 4 + R * T * Hv * dv * 4
        return reads + writes

    @property
    def layer_bytes_per_layer(self) -> int:
        """Algorithmic HBM bytes of one fused gdn_layer_verify_span call: read
        x, the conv weights, the conv state, a, b and the initial state once;
        write every checkpoint and every output once (q, k, v and the conv
        output never reach memory)."""
        R, T, Hv, dk, dv, C, W = (self.n_req, self.n_pos, self.n_vheads, self.d_k, self.d_v, self.conv_channels,
                                  self.conv_width)
        e = 2 if self.bf16 else 4
        reads = (R * T * C + C * W + R * (W - 1) * C + 2 * R * T * Hv) * e + R * Hv * dv * dk * 4
        writes = R * T * Hv * dv * dk * 4 + R * T * Hv * dv * 4
        return reads + writes

    @property
    def conv_bytes_per_layer(self) -> int:
        R, T, C, W = self.n_req, self.n_pos, self.conv_channels, self.conv_width
        e = 2 if self.bf16 else 4
        return R * T * C * e + C * W * e + R * (W - 1) * C * e + R * T * (W - 1) * C * e + R * T * C * 4

    @property
    def accept_bytes(self) -> int:
        e = 2 if self.bf16 else 4
        return self.n_req * self.n_pos * self.vocab * e

    @property
    def rollback_bytes(self) -> int:
        """Read + write of one checkpoint per (layer, request), state and conv."""
        e = 2 if self.bf16 else 4
        per = self.n_vheads * self.d_v * self.d_k * 4 + (self.conv_width - 1) * self.conv_channels * e
        return 2 * self.n_layers * self.n_req * per

    @property
    def ring_bytes(self) -> int:
        """set + get: each moves n_req * n_pos rows in and out."""
        return 2 * 2 * self.n_req * self.n_pos * self.ring_width * 2


class StepBuffers:
    """Device buffers of one step, laid out [L, ...] per layer (torch owned)."""

    def __init__(self, shape: StepShape, device="cuda"):
        import torch
        s = shape
        dt = torch.bfloat16 if s.bf16 else torch.float32
        L, R, T, Hk, Hv, dk, dv, C, W = (s.n_layers, s.n_req, s.n_pos, s.n_kheads, s.n_vheads, s.d_k, s.d_v,
                                         s.conv_channels, s.conv_width)
        e = lambda *shp, dtype=dt: torch.empty(shp, dtype=dtype, device=device)
        self.shape = s
        self.q = e(L, R, T, Hk, dk)
        self.k = e(L, R, T, Hk, dk)
        self.v = e(L, R, T, Hv, dv)
        self.a = e(L, R, T, Hv)
        self.b = e(L, R, T, Hv)
        self.state = e(L, R, Hv, dv, dk, dtype=torch.float32)
        self.ckpt = e(L, R, T, Hv, dv, dk, dtype=torch.float32)
        self.out = e(L, R, T, Hv, dv, dtype=torch.float32)
        self.x = e(L, R, T, C)
        self.w = e(L, C, W)
        self.conv_state = e(L, R, W - 1, C)
        self.conv_ckpt = e(L, R, T, W - 1, C)
        self.y = e(L, R, T, C, dtype=torch.float32)
        self.tokens = e(R, T, dtype=torch.int32)
        self.argmax = e(R, T, dtype=torch.int32)
        self.accept_node = torch.zeros(R, dtype=torch.int32, device=device)
        self.accept_len = e(R, dtype=torch.int32)
        self.path = e(R, T, dtype=torch.int32)
        self.bonus = e(R, dtype=torch.int32)
        self.status = torch.zeros(4, dtype=torch.int32, device=device)
        self.logits = e(R, T, s.vocab) if s.vocab else None
        self.workspace = None
        if s.vocab:
            nbytes = accept_greedy_workspace_bytes(R, T, s.vocab, HRS_BF16 if s.bf16 else HRS_F32)
            self.workspace = torch.empty(max(16, nbytes), dtype=torch.uint8, device=device)
        self.ring = e(R, s.ring_slots, s.ring_width, dtype=torch.bfloat16) if s.ring_slots else None
        self.packed_in = e(R * T, s.ring_width, dtype=torch.bfloat16) if s.ring_slots else None
        self.packed_out = e(R * T, s.ring_width, dtype=torch.bfloat16) if s.ring_slots else None
        # Host mirror of the step's only device-to-host transfer.
        self.host_result = torch.empty(2 * R, dtype=torch.int32, pin_memory=True)
        self.dev_result = torch.empty(2 * R, dtype=torch.int32, device=device)


def _check(st: int, name: str) -> None:
    if st != 0:
        raise HrsError(st, name)


class VerifyStep:
    """Precomputed launch sequence of one verify step.

    parent: None (chain) or host ints [R, T] (draft trees, one per request).
    runs: ring runs (ring_id, start_pos, n_rows, packed_row) for set and get.
    """

    def __init__(self, bufs: StepBuffers, parent=None, runs: Optional[Sequence[tuple]] = None,
                 silu: bool = False, q_scale: float = 1.0):
        s = bufs.shape
        self.bufs = bufs
        L, R, T = s.n_layers, s.n_req, s.n_pos
        self.topo = HRS_TREE if parent is not None else HRS_CHAIN
        dt = HRS_BF16 if s.bf16 else HRS_F32
        if parent is not None:
            self._parent = np.ascontiguousarray(np.broadcast_to(np.asarray(parent, dtype=np.int32), (R, T)))
            par_p = self._parent.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        else:
            self._parent, par_p = None, None
        self.gdn_desc = GdnDesc(R, T, s.n_kheads, s.n_vheads, s.d_k, s.d_v, dt, q_scale, self.topo, par_p)
        self.conv_desc = ConvDesc(R, T, s.conv_channels, s.conv_width, dt, int(silu), self.topo, par_p)
        self.accept_desc = AcceptDesc(R, T, s.vocab, dt, self.topo, par_p) if s.vocab else None
        self.rb_desc = RollbackDesc(L, R, T, s.n_vheads, s.d_k, s.d_v, s.conv_channels, s.conv_width, dt)
        self.runs = list(runs or [])
        if s.ring_slots and self.runs:
            self._runs_arr = (RingRun * len(self.runs))(*[RingRun(*map(int, r)) for r in self.runs])
            self.ring_desc = RingDesc(R, s.ring_slots, s.ring_width, HRS_BF16, R * T, len(self.runs),
                                      self._runs_arr)
        else:
            self.ring_desc = None

        b = bufs
        ptr = lambda t, l: t[l].data_ptr()
        self.layer_args: List[tuple] = []
        for l in range(L):
            self.layer_args.append((
                (ptr(b.x, l), ptr(b.w, l), ptr(b.conv_state, l), ptr(b.conv_ckpt, l), ptr(b.y, l)),
                (ptr(b.q, l), ptr(b.k, l), ptr(b.v, l), ptr(b.a, l), ptr(b.b, l), ptr(b.state, l),
                 ptr(b.ckpt, l), ptr(b.out, l)),
            ))
        if s.vocab:
            self.accept_args = (b.logits.data_ptr(), b.tokens.data_ptr(), b.argmax.data_ptr(),
                                b.accept_node.data_ptr(), b.accept_len.data_ptr(), b.path.data_ptr(),
                                b.bonus.data_ptr(), b.workspace.data_ptr(),
                                b.workspace.numel())
        self.rb_args = (b.ckpt.data_ptr(), b.state.data_ptr(), b.conv_ckpt.data_ptr(), b.conv_state.data_ptr(),
                        b.accept_node.data_ptr(), b.status.data_ptr())
        self.gdn_p = ctypes.byref(self.gdn_desc)
        self.conv_p = ctypes.byref(self.conv_desc)
        self.rb_p = ctypes.byref(self.rb_desc)

    # -- pieces -------------------------------------------------------------
    def launch_layer(self, l: int, stream: int, events=None) -> None:
        """conv then GDN of layer l. events: optional (start, stop) raw
        hipEvent_t handles recorded by the GDN dispatch itself."""
        conv_a, gdn_a = self.layer_args[l]
        _check(lib.conv1d_verify_span(self.conv_p, *conv_a, stream), "conv1d_verify_span")
        if events is None:
            _check(lib.gdn_verify_span(self.gdn_p, *gdn_a, stream), "gdn_verify_span")
        else:
            _check(lib.gdn_verify_span_timed(self.gdn_p, *gdn_a, stream, events[0], events[1]), "gdn_verify_span")

    def launch_conv(self, l: int, stream: int) -> None:
        """The conv span of layer l alone."""
        _check(lib.conv1d_verify_span(self.conv_p, *self.layer_args[l][0], stream), "conv1d_verify_span")

    def launch_gdn(self, l: int, stream: int, events=None) -> None:
        """The GDN span of layer l alone (its inputs as the step leaves them).
        events: optional (start, stop) raw hipEvent_t handles recorded by the
        dispatch itself."""
        if events is None:
            _check(lib.gdn_verify_span(self.gdn_p, *self.layer_args[l][1], stream), "gdn_verify_span")
        else:
            _check(lib.gdn_verify_span_timed(self.gdn_p, *self.layer_args[l][1], stream, events[0], events[1]),
                   "gdn_verify_span")

    def launch_accept(self, stream: int) -> None:
        if self.accept_desc is not None:
            _check(lib.accept_greedy(ctypes.byref(self.accept_desc), *self.accept_args, stream), "accept_greedy")

    def launch_rollback(self, stream: int) -> None:
        _check(lib.rollback_restore(self.rb_p, *self.rb_args, stream), "rollback_restore")

    def launch_ring(self, stream: int) -> None:
        if self.ring_desc is None:
            return
        b = self.bufs
        _check(lib.ring_set_2d(ctypes.byref(self.ring_desc), b.ring.data_ptr(), b.packed_in.data_ptr(), stream),
               "ring_set_2d")
        _check(lib.ring_get_2d(ctypes.byref(self.ring_desc), b.ring.data_ptr(), b.packed_out.data_ptr(), stream),
               "ring_get_2d")

    # -- whole step -----------------------------------------------------------
    def launch(self, stream=None, gdn_events=None) -> None:
        """Issue the whole step on ``stream`` (torch stream or raw handle); no sync.

        gdn_events: optional list of (start, stop) raw hipEvent_t handles per
        layer (see ``event_handle``), recorded by each GDN dispatch.
        """
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        for l in range(self.bufs.shape.n_layers):
            self.launch_layer(l, h, None if gdn_events is None else gdn_events[l])
        self.launch_accept(h)
        self.launch_rollback(h)
        self.launch_ring(h)

    def _gather(self) -> None:
        """Device-side gather of accepted lengths and bonus tokens into one buffer."""
        b = self.bufs
        R = self.bufs.shape.n_req
        b.dev_result[:R].copy_(b.accept_len)
        b.dev_result[R:].copy_(b.bonus)

    def _host(self):
        b = self.bufs
        R = self.bufs.shape.n_req
        b.host_result.copy_(b.dev_result)   # blocking copy into pinned memory
        return b.host_result[:R].numpy().copy(), b.host_result[R:].numpy().copy()

    def finish(self):
        """The step's single host sync: accepted lengths and bonus tokens."""
        self._gather()
        return self._host()

    def run(self, stream=None):
        self.launch(stream)
        return self.finish()

    # -- graph launch ---------------------------------------------------------
    def capture_graph(self) -> None:
        """Record the whole step (every kernel and the device-side gather of
        the results) into one HIP graph. Buffers, descriptors and pointers
        are fixed, so replaying the graph is exactly one step. The graph holds
        kernel launches and device copies only (no memset nodes)."""
        import torch
        self.graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(self.graph, stream=side):
            self.launch(side)
            self._gather()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()

    def replay(self):
        """One step by graph replay, then the step's single host sync."""
        self.graph.replay()
        return self._host()


class ZeroCopyVerifyStep(VerifyStep):
    """Verify step with zero-copy rollback (gdn_verify_span_from) and compact
    conv state (conv1d_verify_span_nocapture + conv_state_advance).

    Two checkpoint buffers alternate between steps: step i writes buffer i % 2
    and its spans start from buffer (i - 1) % 2 at the accepted position that
    step i - 1's acceptance left in ``accept_node`` (the first step starts from
    ``state``). Nothing is copied to roll back; the conv state is rebuilt from
    the x rows along the accepted path. ``materialize()`` writes the canonical
    recurrent state into ``state`` (rollback_restore) when a caller needs it.
    Needs logits (acceptance produces the path the conv state follows).
    """

    def __init__(self, bufs: StepBuffers, parent=None, runs: Optional[Sequence[tuple]] = None,
                 silu: bool = False, q_scale: float = 1.0):
        import torch
        super().__init__(bufs, parent, runs, silu, q_scale)
        s = bufs.shape
        if not s.vocab:
            raise ValueError("zero-copy rollback needs logits: the conv state follows the accepted path")
        L, R, T = s.n_layers, s.n_req, s.n_pos
        if getattr(bufs, "ckpt2", None) is None:
            bufs.ckpt2 = torch.empty_like(bufs.ckpt)
        self.ckpts = (bufs.ckpt, bufs.ckpt2)
        b = bufs
        dt = HRS_BF16 if s.bf16 else HRS_F32
        self.adv_desc = ConvAdvanceDesc(L, R, T, s.conv_channels, s.conv_width, dt)
        self.adv_p = ctypes.byref(self.adv_desc)
        self.adv_args = (b.x.data_ptr(), b.conv_state.data_ptr(), b.path.data_ptr(), b.accept_len.data_ptr(), None)
        ptr = lambda t, l: t[l].data_ptr()
        self.conv_args = [(ptr(b.x, l), ptr(b.w, l), ptr(b.conv_state, l), ptr(b.y, l)) for l in range(L)]
        # [c][l]: inputs and outputs of layer l when writing checkpoint buffer c.
        self.srcs = [[SpanSource(ptr(self.ckpts[1 - c], l), b.accept_node.data_ptr(), T) for l in range(L)]
                     for c in range(2)]
        self.gdn_io = [[(ptr(b.q, l), ptr(b.k, l), ptr(b.v, l), ptr(b.a, l), ptr(b.b, l), ptr(self.ckpts[c], l),
                         ptr(b.out, l)) for l in range(L)] for c in range(2)]
        self.first = True
        self.cur = 0

    def launch_layer(self, l: int, stream: int, events=None) -> None:
        _check(lib.conv1d_verify_span_nocapture(self.conv_p, *self.conv_args[l], stream),
               "conv1d_verify_span_nocapture")
        q, k, v, a, bb, ck, out = self.gdn_io[self.cur][l]
        if self.first:
            _check(lib.gdn_verify_span(self.gdn_p, q, k, v, a, bb, self.layer_args[l][1][5], ck, out, stream),
                   "gdn_verify_span")
        else:
            _check(lib.gdn_verify_span_from(self.gdn_p, ctypes.byref(self.srcs[self.cur][l]), q, k, v, a, bb, ck,
                                            out, None, stream), "gdn_verify_span_from")

    def launch_rollback(self, stream: int) -> None:
        # The rollback of the recurrent state is the next step's source index;
        # only the conv state is rebuilt.
        _check(lib.conv_state_advance(self.adv_p, *self.adv_args, stream), "conv_state_advance")

    def launch(self, stream=None, gdn_events=None) -> None:
        super().launch(stream, gdn_events=None)
        self.first = False
        self.cur ^= 1

    def current_ckpt(self):
        """Checkpoint buffer written by the last launched step."""
        return self.ckpts[self.cur ^ 1]

    def materialize(self, stream=None) -> None:
        """state <- checkpoint of the accepted position of the last step (all layers)."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        s = self.bufs.shape
        d = RollbackDesc(s.n_layers, s.n_req, s.n_pos, s.n_vheads, s.d_k, s.d_v, 0, 0, HRS_F32)
        b = self.bufs
        _check(lib.rollback_restore(ctypes.byref(d), self.current_ckpt().data_ptr(), b.state.data_ptr(), None, None,
                                    b.accept_node.data_ptr(), b.status.data_ptr(), h), "rollback_restore")

    def capture_graph(self) -> None:
        """Record two HIP graphs, one per checkpoint-buffer parity: graph c
        writes buffer c and starts every span from buffer 1 - c at the
        accepted position the previous step left in ``accept_node``. Replays
        alternate between them, as eager steps alternate buffers. The first
        step of a speculation starts from ``state`` and is launched eagerly
        (``replay`` does that by itself when no step has run yet)."""
        import torch
        first, cur = self.first, self.cur
        self.graphs = []
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        try:
            self.first = False
            for c in (0, 1):
                self.cur = c
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    VerifyStep.launch(self, side)
                    self._gather()
                self.graphs.append(g)
        finally:
            self.first, self.cur = first, cur
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()

    def replay(self):
        """One step by replaying the graph of the current buffer parity (the
        first step of a speculation eagerly), then the step's single host
        sync."""
        if self.first:
            return self.run()
        self.graphs[self.cur].replay()
        self.cur ^= 1
        return self._host()


class FusedVerifyStep(ZeroCopyVerifyStep):
    """Zero-copy verify step whose layers run in their own order in one kernel
    each (gdn_layer_verify_span: conv, SiLU, split, q/k L2 norm and the gated
    delta rule). q, k and v are computed on the chip from x, so the q, k, v
    and y buffers are not used. Rollback as in ZeroCopyVerifyStep: the next
    spans start from the accepted checkpoint, the conv state is rebuilt from
    the accepted path (conv_state_advance).
    """

    def __init__(self, bufs: StepBuffers, parent=None, runs: Optional[Sequence[tuple]] = None,
                 silu: bool = True, q_scale: float = 1.0, l2_eps: float = 1e-6):
        super().__init__(bufs, parent, runs, silu, q_scale)
        s = bufs.shape
        if s.conv_channels != 2 * s.n_kheads * s.d_k + s.n_vheads * s.d_v:
            raise ValueError("the fused layer needs conv channels = 2*Hk*d_k + Hv*d_v (q | k | v)")
        self.layer_desc = GdnLayerDesc(self.gdn_desc, s.conv_width, int(silu), float(l2_eps))
        self.layer_p = ctypes.byref(self.layer_desc)
        b = bufs
        L = s.n_layers
        ptr = lambda t, l: t[l].data_ptr()
        self.fused_in = [(ptr(b.x, l), ptr(b.w, l), ptr(b.conv_state, l), ptr(b.a, l), ptr(b.b, l))
                         for l in range(L)]
        self.fused_out = [[(ptr(self.ckpts[c], l), ptr(b.out, l)) for l in range(L)] for c in range(2)]

    def launch_layer(self, l: int, stream: int, events=None) -> None:
        ck, out = self.fused_out[self.cur][l]
        if self.first:
            state, src = self.layer_args[l][1][5], None
        else:
            state, src = None, ctypes.byref(self.srcs[self.cur][l])
        _check(lib.gdn_layer_verify_span(self.layer_p, *self.fused_in[l], state, src, ck, out, None, stream),
               "gdn_layer_verify_span")


@dataclasses.dataclass(frozen=True)
class AttnShape:
    """The attention layers of a hybrid model and their paged cache."""
    n_layers: int
    n_heads: int
    n_kvheads: int
    head_dim: int
    rotary_dim: int            # multiple of 16, at most head_dim; 0: no rotation
    n_pages: int               # pages of one layer
    page_size: int             # slots of one page
    table_len: int             # pages one request may hold
    theta: float = 1e7
    eps: float = 1e-6
    weight_offset: float = 0.0
    f8_cache: bool = False     # float8_e4m3fn pages with a scale per layer and key head
    after: Optional[Sequence[int]] = None   # the GDN layer each attention layer follows; default: evenly spread
    prefix_len: int = 0        # leading slots that all requests share (read once for all of them); seq_len counts them
    page_list: bool = False    # tables grow from and shrink into a free list on the device, step by step


class AttnBuffers:
    """Device buffers of the attention layers beside a step's StepBuffers.

    qkv [L,R,T,Hq+2Hkv,d] is each layer's projection; q_out, k_out its
    normalised and rotated heads. page_table holds distinct pages per request
    and seq_len [R] the slots that count (the step advances them itself).
    uniforms [R,T] and temperature [R] are read where acceptance samples,
    top_k, top_p and min_p [R] (none to start with) where it is filtered.
    held [R] marks requests that could not go on (see HybridVerifyStep).

    With a prefix, prefix_table names its pages, the last one possibly in part:
    that one is of no request's table, each has a page of its own in its place.
    seq_len starts at the prefix's length; a request with less is held.
    With a page list, free_pages [n_pages] and n_free [1] start with every page
    behind the prefix's, which are pages 0, 1, ... then, and n_held [R] with
    none: the step fills and cuts page_table itself."""

    def __init__(self, shape: AttnShape, step: StepShape, device="cuda"):
        import torch
        s, R, T = shape, step.n_req, step.n_pos
        dt = torch.bfloat16 if step.bf16 else torch.float32
        L, Hq, Hkv, d = s.n_layers, s.n_heads, s.n_kvheads, s.head_dim
        e = lambda *shp, dtype=dt: torch.empty(shp, dtype=dtype, device=device)
        z = lambda *shp, dtype=torch.int32: torch.zeros(shp, dtype=dtype, device=device)
        self.shape = s
        self.qkv = e(L, R, T, Hq + 2 * Hkv, d)
        self.q, self.k, self.v = self.qkv.split([Hq, Hkv, Hkv], dim=3)
        self.q_weight = torch.full((L, d), 1.0 - s.weight_offset, dtype=dt, device=device)
        self.k_weight = self.q_weight.clone()
        self.freq = None
        if s.rotary_dim:
            i = torch.arange(s.rotary_dim // 2, dtype=torch.float64, device=device)
            self.freq = s.theta ** (-2.0 * i / s.rotary_dim)
        self.q_out = e(L, R, T, Hq, d)
        self.k_out = e(L, R, T, Hkv, d)
        self.out = e(L, R, T, Hq, d)
        pages = (L, s.n_pages, Hkv, s.page_size, d)
        if s.f8_cache:
            self.k_cache, self.v_cache = (z(*pages, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
            self.k_scale, self.v_scale = (torch.ones(L, Hkv, device=device) for _ in range(2))
        else:
            self.k_cache, self.v_cache = z(*pages, dtype=dt), z(*pages, dtype=dt)
            self.k_scale = self.v_scale = None
        self.page_table = z(R, s.table_len)
        self.seq_len = torch.full((R,), s.prefix_len, dtype=torch.int32, device=device)
        whole, pages = s.prefix_len // s.page_size, -(-s.prefix_len // s.page_size)
        self.prefix_table = torch.arange(pages, dtype=torch.int32, device=device) if s.prefix_len else None
        self.prefix_len = torch.full((1,), s.prefix_len, dtype=torch.int32, device=device) if s.prefix_len else None
        self.free_pages = None
        if s.page_list:
            if whole > s.table_len or pages > s.n_pages:
                raise ValueError(f"a prefix of {pages} pages, {s.table_len} entries a table, {s.n_pages} pages")
            self.free_pages = torch.arange(s.n_pages, dtype=torch.int32, device=device).roll(-pages)
            self.n_free = torch.full((1,), s.n_pages - pages, dtype=torch.int32, device=device)
            self.n_held = z(R)
            self.page_table.fill_(-1)
            self.whole_prefix = self.prefix_table[:whole] if whole else None
        # Refused requests, one row per call (its first word counts): attention
        # layers 0..L-1, then acceptance, then the append; with a page list
        # the requests whose next span finds no pages, and the release.
        self.status = z(L + 2, 4)
        self.page_status = z(2, 4)
        self.uniforms = z(R, T, dtype=torch.float32)
        self.token_prob = z(R, T, dtype=torch.float32)
        self.temperature = torch.ones(R, device=device)
        self.top_k, self.top_p, self.min_p = z(R), torch.ones(R, device=device), torch.zeros(R, device=device)
        self.held = z(R)
        self.last_node = z(R)
        # Where a held request's recurrent state is: a position of checkpoint
        # buffer 0 or 1, or -1.
        self.held_node = [z(R), z(R)]
        nbytes = max(attn_verify_span_workspace_bytes(R, T, Hq, Hkv, d),
                     attn_verify_shared_workspace_bytes(R, T, Hq, Hkv, d) if s.prefix_len else 0,
                     kv_pages_workspace_bytes(R) if s.page_list else 0,
                     accept_sample_workspace_bytes(R, T, step.vocab) if step.vocab else 0,
                     accept_sample_filtered_workspace_bytes(R, T, step.vocab) if step.vocab else 0)
        self.workspace = e(max(16, nbytes), dtype=torch.uint8)   # one stream: the calls take turns


class HybridVerifyStep(FusedVerifyStep):
    """FusedVerifyStep of a model whose GDN layers alternate with attention
    layers. After GDN layer ``after[i]`` comes attention layer i: norm and
    rotation of its projection, then attention of the span over the layer's
    pages and the draft's own paths. Behind acceptance (greedy, or by sampling
    with ``sample``: ``uniforms`` and ``temperature`` of the AttnBuffers) the
    accepted rows of all attention layers go into their pages and ``seq_len``
    advances, so replays of the captured step carry on by themselves.

    A request that cannot go on is held (accept_hold_behind): its accepted rows do not
    fit in its page table, a page for them is not there, they would begin inside
    a prefix that all requests read, or its temperature is negative or NaN. The
    step then reports -1 as its accepted length and bonus token and leaves its
    pages, length, conv and recurrent state as they were; so do all later steps.
    The other requests go on. To take it up again:
    ``materialize()`` (which writes every request's recurrent state, a held
    one's from in front of the step that held it), give it what it lacks, and
    start a new speculation with a new HybridVerifyStep.

    ``filtered`` samples after top-k, top-p and min-p (accept_sample_filtered:
    ``top_k``, ``top_p``, ``min_p`` of the AttnBuffers). A shape with a prefix
    reads its slots once for all requests (attn_verify_shared). With a page list
    a step takes the pages of its span's slots, up to the table's end, before
    its layers and gives those that the accepted rows leave empty back behind
    the append. Requests are served in their order until one's pages are not all
    there, so a request is held for want of pages where the list has too few for
    the requests up to it; held ones take none. A request that ends gives its
    own back through kv_pages_release.
    """

    def __init__(self, bufs: StepBuffers, attn: AttnBuffers, parent=None, runs: Optional[Sequence[tuple]] = None,
                 silu: bool = True, q_scale: float = 1.0, l2_eps: float = 1e-6, sample: bool = False,
                 filtered: bool = False):
        super().__init__(bufs, parent, runs, silu, q_scale, l2_eps)
        s, b, n = attn.shape, attn, bufs.shape.n_layers
        self.attn = attn
        b.held.zero_()
        for node in b.held_node:
            node.fill_(-1)
        after = [(i + 1) * n // s.n_layers - 1 for i in range(s.n_layers)] if s.after is None else list(s.after)
        if len(after) != s.n_layers or any(not 0 <= l < n for l in after) or after != sorted(after):
            raise ValueError(f"after: {after}, expected {s.n_layers} ascending GDN layers of {n}")
        scale = lambda t, i: None if t is None else t[i]
        self.attn_calls: List[list] = [[] for _ in range(n)]
        for i, l in enumerate(after):
            self.attn_calls[l] += [
                qk_norm_rope_call(b.q[i], b.k[i], b.q_weight[i], b.k_weight[i], b.freq, b.seq_len, b.q_out[i],
                                  b.k_out[i], self._parent, s.eps, s.weight_offset),
                attn_verify_shared_call(b.q_out[i], b.k_out[i], b.v[i], b.k_cache[i], b.v_cache[i], b.prefix_table,
                                        b.prefix_len, b.page_table, b.seq_len, b.out[i], b.workspace, self._parent,
                                        k_scale=scale(b.k_scale, i), v_scale=scale(b.v_scale, i), status=b.status[i])
                if s.prefix_len else
                attn_verify_span_call(b.q_out[i], b.k_out[i], b.v[i], b.k_cache[i], b.v_cache[i], b.page_table,
                                      b.seq_len, b.out[i], b.workspace, self._parent,
                                      k_scale=scale(b.k_scale, i), v_scale=scale(b.v_scale, i), status=b.status[i])]
        sample_args = (bufs.logits, bufs.tokens, b.uniforms, b.token_prob, bufs.accept_node, bufs.accept_len,
                       bufs.path, bufs.bonus, b.workspace)
        more = dict(temperature=b.temperature, parent=self._parent, status=b.status[-2])
        self.sample_call = None
        if filtered:
            self.sample_call = accept_sample_filtered_call(*sample_args, top_k=b.top_k, top_p=b.top_p, min_p=b.min_p,
                                                           **more)
        elif sample:
            self.sample_call = accept_sample_call(*sample_args, **more)
        sample = sample or filtered
        # By the checkpoint buffer that a step's spans start from; None: from ``state``.
        self.hold_calls = {c: accept_hold_behind_call(
            b.page_table, b.seq_len, bufs.accept_node, bufs.accept_len, bufs.path, bufs.bonus, b.held, b.last_node,
            s.n_pages, s.page_size, s.prefix_len, held_node=None if c is None else b.held_node[c],
            temperature=b.temperature if sample else None) for c in (None, 0, 1)}
        self.append_call = kv_cache_append_call(
            b.k_out, b.v, b.k_cache, b.v_cache, b.page_table, b.seq_len, bufs.accept_len, b.seq_len, bufs.path,
            b.k_scale, b.v_scale, b.status[-1])
        self.reserve_call = self.release_call = None
        if s.page_list:
            lists = (b.page_table, b.n_held, b.free_pages, b.n_free, b.workspace)
            whole = 0 if b.whole_prefix is None else b.whole_prefix.shape[0]
            self.reserve_call = kv_pages_reserve_step_call(
                b.seq_len, *lists, page_size=s.page_size, n_pos=bufs.shape.n_pos, prefix_table=b.whole_prefix,
                status=b.page_status[0], skip=b.held)
            self.release_call = kv_pages_release_call(b.seq_len, *lists, page_size=s.page_size, n_prefix=whole,
                                                      status=b.page_status[1])

    def launch_layer(self, l: int, stream: int, events=None) -> None:
        if l == 0 and self.reserve_call is not None:
            self.reserve_call(stream)
        super().launch_layer(l, stream, events)
        for call in self.attn_calls[l]:
            call(stream)

    def launch_accept(self, stream: int) -> None:
        if self.sample_call is None:
            super().launch_accept(stream)
        else:
            self.sample_call(stream)
        self.hold_calls[None if self.first else 1 - self.cur](stream)

    def launch_rollback(self, stream: int) -> None:
        super().launch_rollback(stream)
        self.append_call(stream)
        if self.release_call is not None:
            self.release_call(stream)

    def materialize(self, stream=None) -> None:
        """state <- every request's recurrent state after its last accepted
        position (held ones': in front of the step that held them)."""
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        s, b = self.bufs.shape, self.bufs
        d = RollbackDesc(s.n_layers, s.n_req, s.n_pos, s.n_vheads, s.d_k, s.d_v, 0, 0, HRS_F32)
        for c in (0, 1):
            _check(lib.rollback_restore(ctypes.byref(d), self.ckpts[c].data_ptr(), b.state.data_ptr(), None, None,
                                        self.attn.held_node[c].data_ptr(), b.status.data_ptr(), h), "rollback_restore")
        super().materialize(stream)

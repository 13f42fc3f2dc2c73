"""Python binding of libhrs: verify-span checkpoints, greedy acceptance and
on-device rollback for Gated DeltaNet layers on MI355X (gfx950).

Argument marshalling only. Every function here takes torch tensors that
live on the GPU, checks that they are contiguous and of the expected dtype,
and passes raw pointers, sizes and the current HIP stream to the C ABI in
include/hrs.h; all computation happens in the HIP kernels of libhrs.so. A
negative status from the library raises ``HrsError``.

The library must be built first (``python hybrid_recurrent_state_amd/csrc/build.py``
or ``__graft_entry__.build()``); importing this package without it raises
ImportError, so nothing silently falls back to another implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhrs.so")

HRS_OK, HRS_EINVAL, HRS_EGEOMETRY, HRS_EALIGN, HRS_EDEVICE, HRS_EUNSUPPORTED = 0, -1, -2, -3, -4, -5
HRS_F32, HRS_BF16, HRS_F8E4M3 = 0, 1, 2
HRS_CHAIN, HRS_TREE = 0, 1
HRS_MAX_POS = 64
GEOMETRY_CLASSES = {0: "OK", 1: "NULL", 2: "TRUNCATED", 3: "ROOT", 4: "RANGE", 5: "FORWARD", 6: "NOT_CHAIN"}


class HrsError(RuntimeError):
    def __init__(self, status: int, func: str):
        self.status = status
        detail = ""
        if status == HRS_EDEVICE:
            detail = f"; HIP error {lib.hrs_last_hip_error()}: {lib.hrs_last_hip_error_string().decode()}"
        super().__init__(f"{func}: {strerror(status)} (status {status}){detail}")


# --- C structs (mirror include/hrs.h) -------------------------------------
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_p = ctypes.c_void_p


class GdnDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("n_kheads", _i32), ("n_vheads", _i32),
                ("d_k", _i32), ("d_v", _i32), ("in_dtype", _i32), ("q_scale", ctypes.c_float),
                ("topo", _i32), ("parent", ctypes.POINTER(_i32))]


class ChunkedDesc(ctypes.Structure):
    _fields_ = [("gdn", GdnDesc), ("log_gates", _i32), ("out_dtype", _i32)]


class GdnLayerDesc(ctypes.Structure):
    _fields_ = [("gdn", GdnDesc), ("conv_width", _i32), ("silu", _i32), ("l2_eps", ctypes.c_float)]


class ConvDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("channels", _i32), ("width", _i32),
                ("dtype", _i32), ("silu", _i32), ("topo", _i32), ("parent", ctypes.POINTER(_i32))]


class AcceptDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("vocab", _i32), ("logit_dtype", _i32),
                ("topo", _i32), ("parent", ctypes.POINTER(_i32))]


class SpanSource(ctypes.Structure):
    _fields_ = [("ckpt", _p), ("node", _p), ("n_pos", _i32)]


class ConvAdvanceDesc(ctypes.Structure):
    _fields_ = [("n_layers", _i32), ("n_req", _i32), ("n_pos", _i32), ("channels", _i32), ("width", _i32),
                ("dtype", _i32)]


class RollbackDesc(ctypes.Structure):
    _fields_ = [("n_layers", _i32), ("n_req", _i32), ("n_pos", _i32), ("n_vheads", _i32),
                ("d_k", _i32), ("d_v", _i32), ("conv_channels", _i32), ("conv_width", _i32),
                ("conv_dtype", _i32)]


class RingRun(ctypes.Structure):
    _fields_ = [("ring_id", _i32), ("start_pos", _i32), ("n_rows", _i32), ("packed_row", _i32)]


class RingDesc(ctypes.Structure):
    _fields_ = [("n_rings", _i32), ("n_slots", _i32), ("width", _i32), ("dtype", _i32),
                ("n_packed_rows", _i32), ("n_runs", _i32), ("runs", ctypes.POINTER(RingRun))]


class QkDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("n_heads", _i32), ("n_kvheads", _i32), ("d", _i32), ("rot", _i32),
                ("dtype", _i32), ("q_stride", _i64), ("k_stride", _i64), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("interleaved", _i32), ("topo", _i32),
                ("parent", ctypes.POINTER(_i32))]


class CacheDesc(ctypes.Structure):
    _fields_ = [("n_pages", _i32), ("page_size", _i32), ("table_len", _i32), ("dtype", _i32)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("n_heads", _i32), ("n_kvheads", _i32), ("d", _i32),
                ("dtype", _i32), ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("scale", ctypes.c_float), ("window", _i32), ("cache", CacheDesc), ("topo", _i32),
                ("parent", ctypes.POINTER(_i32))]


class AppendDesc(ctypes.Structure):
    _fields_ = [("n_layers", _i32), ("n_req", _i32), ("n_pos", _i32), ("n_kvheads", _i32), ("d", _i32),
                ("dtype", _i32), ("k_stride", _i64), ("v_stride", _i64), ("cache", CacheDesc)]


class SampleDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("vocab", _i32), ("logit_dtype", _i32), ("draft_dtype", _i32),
                ("topo", _i32), ("parent", ctypes.POINTER(_i32))]


class HoldDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("n_pages", _i32), ("page_size", _i32), ("table_len", _i32)]


class PagesDesc(ctypes.Structure):
    _fields_ = [("n_req", _i32), ("n_pos", _i32), ("n_pages", _i32), ("page_size", _i32), ("table_len", _i32),
                ("n_prefix", _i32)]


# Exported symbols and their signatures (every function of include/hrs.h).
_SIGNATURES = {
    "hrs_validate_tree": (_i32, [ctypes.POINTER(_i32), _i32, _i32, ctypes.POINTER(_i32)]),
    "gdn_verify_span": (_i32, [ctypes.POINTER(GdnDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p]),
    "gdn_verify_span_timed": (_i32, [ctypes.POINTER(GdnDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p]),
    "gdn_verify_span_from": (_i32, [ctypes.POINTER(GdnDesc), ctypes.POINTER(SpanSource), _p, _p, _p, _p, _p, _p,
                                    _p, _p, _p]),
    "gdn_span_chunked_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(ChunkedDesc)]),
    "gdn_span_chunked": (_i32, [ctypes.POINTER(ChunkedDesc), _p, _p, _p, _p, _p, _p, _p, _p, _p, ctypes.c_size_t,
                                _p]),
    "gdn_layer_verify_span": (_i32, [ctypes.POINTER(GdnLayerDesc), _p, _p, _p, _p, _p, _p,
                                     ctypes.POINTER(SpanSource), _p, _p, _p, _p]),
    "conv1d_verify_span_nocapture": (_i32, [ctypes.POINTER(ConvDesc), _p, _p, _p, _p, _p]),
    "conv_state_advance": (_i32, [ctypes.POINTER(ConvAdvanceDesc), _p, _p, _p, _p, _p, _p]),
    "conv1d_verify_span": (_i32, [ctypes.POINTER(ConvDesc), _p, _p, _p, _p, _p, _p]),
    "accept_greedy_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(AcceptDesc)]),
    "accept_greedy": (_i32, [ctypes.POINTER(AcceptDesc), _p, _p, _p, _p, _p, _p, _p, _p,
                             ctypes.c_size_t, _p]),
    "accept_greedy_noalloc": (_i32, [ctypes.POINTER(AcceptDesc), _p, _p, _p, _p, _p, _p, _p, _p]),
    "rollback_restore": (_i32, [ctypes.POINTER(RollbackDesc), _p, _p, _p, _p, _p, _p, _p]),
    "ring_set_2d": (_i32, [ctypes.POINTER(RingDesc), _p, _p, _p]),
    "ring_get_2d": (_i32, [ctypes.POINTER(RingDesc), _p, _p, _p]),
    "qk_norm_rope": (_i32, [ctypes.POINTER(QkDesc)] + [_p] * 9),
    "attn_verify_span_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(AttnDesc)]),
    "attn_verify_span": (_i32, [ctypes.POINTER(AttnDesc)] + [_p] * 12 + [ctypes.c_size_t, _p]),
    "attn_verify_shared_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(AttnDesc)]),
    "attn_verify_shared": (_i32, [ctypes.POINTER(AttnDesc), _i32] + [_p] * 14 + [ctypes.c_size_t, _p]),
    "kv_cache_append": (_i32, [ctypes.POINTER(AppendDesc)] + [_p] * 13),
    "accept_sample_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(SampleDesc)]),
    "accept_sample": (_i32, [ctypes.POINTER(SampleDesc)] + [_p] * 12 + [ctypes.c_size_t, _p]),
    "accept_sample_filtered_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(SampleDesc)]),
    "accept_sample_filtered": (_i32, [ctypes.POINTER(SampleDesc)] + [_p] * 15 + [ctypes.c_size_t, _p]),
    "accept_hold": (_i32, [ctypes.POINTER(HoldDesc)] + [_p] * 11),
    "accept_hold_behind": (_i32, [ctypes.POINTER(HoldDesc), _i32] + [_p] * 11),
    "kv_pages_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(PagesDesc)]),
    "kv_pages_reserve": (_i32, [ctypes.POINTER(PagesDesc)] + [_p] * 10 + [ctypes.c_size_t, _p]),
    "kv_pages_reserve_step": (_i32, [ctypes.POINTER(PagesDesc)] + [_p] * 11 + [ctypes.c_size_t, _p]),
    "kv_pages_release": (_i32, [ctypes.POINTER(PagesDesc)] + [_p] * 7 + [ctypes.c_size_t, _p]),
    "hrs_strerror": (ctypes.c_char_p, [_i32]),
    "hrs_abi_version": (_i32, []),
    "hrs_last_hip_error": (_i32, []),
    "hrs_last_hip_error_string": (ctypes.c_char_p, []),
}
EXPORTED = tuple(_SIGNATURES)


def _hip_runtimes_mapped():
    """Distinct HIP runtime files mapped into this process."""
    found = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                if "libamdhip64" in line:
                    found.add(os.path.realpath(line.split()[-1]))
    except OSError:
        pass
    return found


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python hybrid_recurrent_state_amd/csrc/build.py`")
    # torch owns device memory and streams. Its HIP runtime must be the one
    # this library binds to: load torch first, so that the library's
    # libamdhip64.so.7 dependency resolves (by soname) to the runtime that is
    # already in the process instead of a second copy from /opt/rocm.
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise ImportError(f"two HIP runtimes are loaded ({sorted(runtimes)}); libhrs must share torch's")
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def strerror(status: int) -> str:
    return lib.hrs_strerror(int(status)).decode()


def abi_version() -> int:
    return int(lib.hrs_abi_version())


def _check(status: int, func: str) -> None:
    if status != HRS_OK:
        raise HrsError(status, func)


# --- marshalling helpers --------------------------------------------------

def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return HRS_F32
    if t.dtype == torch.bfloat16:
        return HRS_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


class _Checks:
    """Rejects, before anything is launched, a tensor that the kernels would
    read or write out of bounds or as the wrong type. Calls check each
    tensor's shape (the library takes every size from the leading tensor),
    dtype and layout; on_gpu() then checks that all of them are on the GPU."""

    def __init__(self):
        self.seen = []

    def __call__(self, name: str, t, shape=None, dtypes=None, optional: bool = False) -> None:
        if t is None:
            if optional:
                return
            raise ValueError(f"{name} is required")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if dtypes is not None and t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        self.seen.append((name, t))

    def status(self, status, optional: bool = True) -> None:
        self("status", status, None, _i32t(), optional)
        if status is not None and status.numel() < 1:
            raise ValueError("status needs at least one int32")

    def on_gpu(self) -> None:
        for name, t in self.seen:
            if not t.is_cuda:
                raise ValueError(f"{name} must be a GPU tensor")


def _in_dtypes(name: str, t):
    """The input dtype of a call (f32 or bf16), checked on its leading tensor."""
    torch = _torch()
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.float32 or torch.bfloat16")
    return (t.dtype,)


def _f32():
    return (_torch().float32,)


def _i32t():
    return (_torch().int32,)


def _stream(stream) -> Optional[int]:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _parent_array(parent, n_req: int, n_pos: int):
    """Host int32 [n_req * n_pos] array (a single [n_pos] row is repeated).

    The library reads exactly n_req * n_pos entries, so any other size is
    rejected here instead of being over-read or silently truncated."""
    if parent is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(parent, dtype=np.int32)).reshape(-1)
    if arr.size == n_pos and n_req > 1:
        arr = np.ascontiguousarray(np.tile(arr, n_req))
    if arr.size != n_req * n_pos:
        raise ValueError(f"parent: {arr.size} entries, expected {n_pos} (one row for every request) "
                         f"or {n_req * n_pos} ({n_req} requests x {n_pos} positions)")
    return arr, arr.ctypes.data_as(ctypes.POINTER(_i32))


# --- entry points (same names as the C ABI) -------------------------------

def validate_tree(parent, n_pos: Optional[int] = None, require_chain: bool = False):
    """Run the host geometry guard. Returns (status, class name)."""
    cls = _i32(-1)
    if parent is None:
        st = lib.hrs_validate_tree(None, int(n_pos or 0), int(require_chain), ctypes.byref(cls))
    else:
        arr = np.ascontiguousarray(np.asarray(parent, dtype=np.int32)).reshape(-1)
        n = arr.size if n_pos is None else int(n_pos)
        st = lib.hrs_validate_tree(arr.ctypes.data_as(ctypes.POINTER(_i32)), n, int(require_chain),
                                   ctypes.byref(cls))
    return int(st), GEOMETRY_CLASSES.get(cls.value, "?")


hrs_validate_tree = validate_tree


def event_handle(ev) -> int:
    """Raw hipEvent_t of a torch.cuda.Event (created by recording it once)."""
    if not ev.cuda_event:
        ev.record()
    return ev.cuda_event


def gdn_verify_span(q, k, v, a, b, state, ckpt, out, parent=None, q_scale: float = 1.0, stream=None,
                    events=None):
    """q, k [R,T,Hk,dk]; v [R,T,Hv,dv]; a, b [R,T,Hv] (f32 or bf16);
    state [R,Hv,dv,dk] f32; ckpt [R,T,Hv,dv,dk] f32 or None; out [R,T,Hv,dv] f32.
    parent: None (chain) or host ints [R,T] / [T] (tree).
    events: optional (start, stop) torch.cuda.Event pair recorded by the
    kernel dispatch itself (gdn_verify_span_timed)."""
    R, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = _in_dtypes("q", q)
    chk = _Checks()
    chk("q", q, None, dt)
    chk("k", k, (R, T, Hk, dk), dt)
    chk("v", v, (R, T, Hv, dv), dt)
    chk("a", a, (R, T, Hv), dt)
    chk("b", b, (R, T, Hv), dt)
    chk("state", state, (R, Hv, dv, dk), _f32())
    chk("ckpt", ckpt, (R, T, Hv, dv, dk), _f32(), optional=True)
    chk("out", out, (R, T, Hv, dv), _f32())
    par, par_p = _parent_array(parent, R, T)
    chk.on_gpu()
    d = GdnDesc(R, T, Hk, Hv, dk, dv, _dtype_code(q), float(q_scale),
                HRS_TREE if parent is not None else HRS_CHAIN, par_p)
    args = (ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(state), _ptr(ckpt), _ptr(out),
            _stream(stream))
    if events is None:
        st = lib.gdn_verify_span(*args)
    else:
        st = lib.gdn_verify_span_timed(*args, event_handle(events[0]), event_handle(events[1]))
    _check(st, "gdn_verify_span")


def gdn_verify_span_from(src_ckpt, src_node, q, k, v, a, b, ckpt, out, parent=None, status=None,
                         q_scale: float = 1.0, stream=None):
    """Zero-copy rollback: like gdn_verify_span, but request r starts from
    src_ckpt[r][src_node[r]] (src_ckpt [R,Tp,Hv,dv,dk] f32, src_node [R] int32,
    both on the device) instead of a state buffer."""
    R, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = _in_dtypes("q", q)
    chk = _Checks()
    chk("q", q, None, dt)
    chk("k", k, (R, T, Hk, dk), dt)
    chk("v", v, (R, T, Hv, dv), dt)
    chk("a", a, (R, T, Hv), dt)
    chk("b", b, (R, T, Hv), dt)
    chk("src_ckpt", src_ckpt, None, _f32())
    chk("src_ckpt", src_ckpt, (R, src_ckpt.shape[1], Hv, dv, dk), _f32())
    chk("src_node", src_node, (R,), _i32t())
    chk("ckpt", ckpt, (R, T, Hv, dv, dk), _f32())
    chk("out", out, (R, T, Hv, dv), _f32())
    chk.status(status)
    par, par_p = _parent_array(parent, R, T)
    chk.on_gpu()
    d = GdnDesc(R, T, Hk, Hv, dk, dv, _dtype_code(q), float(q_scale),
                HRS_TREE if parent is not None else HRS_CHAIN, par_p)
    src = SpanSource(_ptr(src_ckpt), _ptr(src_node), src_ckpt.shape[1])
    st = lib.gdn_verify_span_from(ctypes.byref(d), ctypes.byref(src), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                                  _ptr(ckpt), _ptr(out), _ptr(status), _stream(stream))
    _check(st, "gdn_verify_span_from")


def gdn_span_chunked_workspace_bytes(n_req: int, n_pos: int, n_kheads: int, n_vheads: int, d: int = 128) -> int:
    """Device workspace bytes gdn_span_chunked needs for these sizes."""
    g = GdnDesc(n_req, n_pos, n_kheads, n_vheads, d, d, HRS_BF16, 1.0, HRS_CHAIN, None)
    return int(lib.gdn_span_chunked_workspace_bytes(ctypes.byref(ChunkedDesc(g, 0, HRS_F32))))


def gdn_span_chunked(q, k, v, a, b, state, ckpt, out, workspace, q_scale: float = 1.0, log_gates: bool = False,
                     stream=None):
    """Chunked (64-position) gated delta rule over a long chain span: same
    arguments as gdn_verify_span without a parent; ckpt None updates state
    in place. log_gates: `a` holds log decays. out may be f32 or bf16.
    workspace: device tensor of at least gdn_span_chunked_workspace_bytes."""
    R, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    torch = _torch()
    dt = _in_dtypes("q", q)
    chk = _Checks()
    chk("q", q, None, dt)
    chk("k", k, (R, T, Hk, dk), dt)
    chk("v", v, (R, T, Hv, dv), dt)
    chk("a", a, (R, T, Hv), dt)
    chk("b", b, (R, T, Hv), dt)
    chk("state", state, (R, Hv, dv, dk), _f32())
    chk("ckpt", ckpt, (R, T, Hv, dv, dk), _f32(), optional=True)
    chk("out", out, (R, T, Hv, dv), (torch.float32, torch.bfloat16))
    chk("workspace", workspace)
    chk.on_gpu()
    g = GdnDesc(R, T, Hk, Hv, dk, dv, _dtype_code(q), float(q_scale), HRS_CHAIN, None)
    d = ChunkedDesc(g, int(bool(log_gates)), _dtype_code(out))
    nbytes = workspace.numel() * workspace.element_size()
    st = lib.gdn_span_chunked(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(state), _ptr(ckpt),
                              _ptr(out), _ptr(workspace), nbytes, _stream(stream))
    _check(st, "gdn_span_chunked")


def gdn_layer_verify_span(x, conv_w, conv_state, a, b, ckpt, out, n_kheads: int, d_k: int, state=None,
                          src_ckpt=None, src_node=None, parent=None, status=None, q_scale: float = 1.0,
                          l2_eps: float = 1e-6, silu: bool = True, stream=None):
    """One GDN layer in its own order (conv, SiLU, split, q/k L2 norm, gated
    delta rule) in one kernel. x [R,T,C] with C = 2*Hk*dk + Hv*dv, channels
    [q | k | v]; conv_w [C,4]; conv_state [R,3,C] (read only); a, b [R,T,Hv];
    ckpt [R,T,Hv,dv,dk] f32; out [R,T,Hv,dv] f32. The initial state is either
    state [R,Hv,dv,dk] f32 or src_ckpt[r][src_node[r]] (zero-copy)."""
    R, T, C = x.shape
    Hv = a.shape[2]
    dv = (C - 2 * n_kheads * d_k) // Hv
    if Hv < 1 or C != 2 * n_kheads * d_k + Hv * dv:
        raise ValueError(f"x: {C} channels do not split into q, k ({n_kheads} x {d_k} each) and {Hv} v heads")
    dt = _in_dtypes("x", x)
    chk = _Checks()
    chk("x", x, None, dt)
    chk("conv_w", conv_w, (C, conv_w.shape[1] if conv_w is not None and conv_w.dim() == 2 else 4), dt)
    chk("conv_state", conv_state, (R, conv_w.shape[1] - 1, C), dt)
    chk("a", a, (R, T, Hv), dt)
    chk("b", b, (R, T, Hv), dt)
    chk("ckpt", ckpt, (R, T, Hv, dv, d_k), _f32())
    chk("out", out, (R, T, Hv, dv), _f32())
    chk("state", state, (R, Hv, dv, d_k), _f32(), optional=True)
    if src_ckpt is not None:
        chk("src_ckpt", src_ckpt, None, _f32())
        chk("src_ckpt", src_ckpt, (R, src_ckpt.shape[1], Hv, dv, d_k), _f32())
        chk("src_node", src_node, (R,), _i32t())
    chk.status(status)
    par, par_p = _parent_array(parent, R, T)
    chk.on_gpu()
    g = GdnDesc(R, T, n_kheads, Hv, d_k, dv, _dtype_code(x), float(q_scale),
                HRS_TREE if parent is not None else HRS_CHAIN, par_p)
    d = GdnLayerDesc(g, conv_w.shape[1], int(bool(silu)), float(l2_eps))
    src = None
    if src_ckpt is not None:
        src = ctypes.byref(SpanSource(_ptr(src_ckpt), _ptr(src_node), src_ckpt.shape[1]))
    st = lib.gdn_layer_verify_span(ctypes.byref(d), _ptr(x), _ptr(conv_w), _ptr(conv_state), _ptr(a), _ptr(b),
                                   _ptr(state), src, _ptr(ckpt), _ptr(out), _ptr(status), _stream(stream))
    _check(st, "gdn_layer_verify_span")


def conv1d_verify_span_nocapture(x, w, conv_state, y, parent=None, silu: bool = False, stream=None):
    """conv output y only; conv_state [R,W-1,C] is read only."""
    R, T, C = x.shape
    dt = _in_dtypes("x", x)
    chk = _Checks()
    chk("x", x, None, dt)
    chk("w", w, None, dt)
    W = w.shape[1] if w.dim() == 2 else 0
    chk("w", w, (C, W), dt)
    chk("conv_state", conv_state, (R, W - 1, C), dt)
    chk("y", y, (R, T, C), _f32())
    par, par_p = _parent_array(parent, R, T)
    chk.on_gpu()
    d = ConvDesc(R, T, C, W, _dtype_code(x), int(bool(silu)), HRS_TREE if parent is not None else HRS_CHAIN, par_p)
    st = lib.conv1d_verify_span_nocapture(ctypes.byref(d), _ptr(x), _ptr(w), _ptr(conv_state), _ptr(y),
                                          _stream(stream))
    _check(st, "conv1d_verify_span_nocapture")


def conv_state_advance(x, conv_state, path, accept_len, status=None, stream=None):
    """x [L,R,T,C]; conv_state [L,R,W-1,C]; path [R,T], accept_len [R] int32 (device)."""
    L, R, T, C = x.shape
    dt = _in_dtypes("x", x)
    chk = _Checks()
    chk("x", x, None, dt)
    chk("conv_state", conv_state, None, dt)
    chk("conv_state", conv_state, (L, R, conv_state.shape[2], C), dt)
    chk("path", path, (R, T), _i32t())
    chk("accept_len", accept_len, (R,), _i32t())
    chk.status(status)
    chk.on_gpu()
    d = ConvAdvanceDesc(L, R, T, C, conv_state.shape[2] + 1, _dtype_code(x))
    st = lib.conv_state_advance(ctypes.byref(d), _ptr(x), _ptr(conv_state), _ptr(path), _ptr(accept_len),
                                _ptr(status), _stream(stream))
    _check(st, "conv_state_advance")


def conv1d_verify_span(x, w, conv_state, conv_ckpt, y, parent=None, silu: bool = False, stream=None):
    """x [R,T,C]; w [C,W]; conv_state [R,W-1,C]; conv_ckpt [R,T,W-1,C] or None
    (same dtype as x); y [R,T,C] f32. parent: None (chain) or host [R,T]/[T]."""
    R, T, C = x.shape
    dt = _in_dtypes("x", x)
    chk = _Checks()
    chk("x", x, None, dt)
    chk("w", w, None, dt)
    W = w.shape[1] if w.dim() == 2 else 0
    chk("w", w, (C, W), dt)
    chk("conv_state", conv_state, (R, W - 1, C), dt)
    chk("conv_ckpt", conv_ckpt, (R, T, W - 1, C), dt, optional=True)
    chk("y", y, (R, T, C), _f32())
    par, par_p = _parent_array(parent, R, T)
    chk.on_gpu()
    d = ConvDesc(R, T, C, W, _dtype_code(x), int(bool(silu)),
                 HRS_TREE if parent is not None else HRS_CHAIN, par_p)
    st = lib.conv1d_verify_span(ctypes.byref(d), _ptr(x), _ptr(w), _ptr(conv_state), _ptr(conv_ckpt),
                                _ptr(y), _stream(stream))
    _check(st, "conv1d_verify_span")


def accept_desc(n_req: int, n_pos: int, vocab: int, logit_dtype: int, parent=None):
    par, par_p = _parent_array(parent, n_req, n_pos)
    d = AcceptDesc(n_req, n_pos, vocab, logit_dtype, HRS_TREE if parent is not None else HRS_CHAIN, par_p)
    return d, par


def accept_greedy_workspace_bytes(n_req: int, n_pos: int, vocab: int, logit_dtype: int = HRS_BF16,
                                  parent=None) -> int:
    d, _keep = accept_desc(n_req, n_pos, vocab, logit_dtype, parent)
    return int(lib.accept_greedy_workspace_bytes(ctypes.byref(d)))


def accept_greedy(logits, tokens, argmax, accept_node, accept_len, path, bonus, workspace,
                  parent=None, stream=None):
    """logits [R,T,V]; tokens [R,T] int32; outputs int32 device tensors
    argmax [R,T], accept_node [R], accept_len [R], path [R,T], bonus [R];
    workspace: device tensor of at least accept_greedy_workspace_bytes."""
    R, T, V = logits.shape
    chk = _Checks()
    chk("logits", logits, None, _in_dtypes("logits", logits))
    for name, t, shape in (("tokens", tokens, (R, T)), ("argmax", argmax, (R, T)), ("accept_node", accept_node, (R,)),
                           ("accept_len", accept_len, (R,)), ("path", path, (R, T)), ("bonus", bonus, (R,))):
        chk(name, t, shape, _i32t())
    chk("workspace", workspace)
    d, _keep = accept_desc(R, T, V, _dtype_code(logits), parent)
    chk.on_gpu()
    nbytes = workspace.numel() * workspace.element_size()
    st = lib.accept_greedy(ctypes.byref(d), _ptr(logits), _ptr(tokens), _ptr(argmax), _ptr(accept_node),
                           _ptr(accept_len), _ptr(path), _ptr(bonus), _ptr(workspace), nbytes,
                           _stream(stream))
    _check(st, "accept_greedy")


ACCEPT_NOALLOC_MAX_BYTES = 1 << 20


def accept_greedy_noalloc(logits, tokens, argmax, accept_node, accept_len, path, bonus, parent=None, stream=None):
    """accept_greedy without a workspace: the library keeps the keys in a
    fixed device array of ACCEPT_NOALLOC_MAX_BYTES per GPU (no allocation in
    the call). Overlapping calls on one GPU share that array and race."""
    R, T, V = logits.shape
    chk = _Checks()
    chk("logits", logits, None, _in_dtypes("logits", logits))
    for name, t, shape in (("tokens", tokens, (R, T)), ("argmax", argmax, (R, T)), ("accept_node", accept_node, (R,)),
                           ("accept_len", accept_len, (R,)), ("path", path, (R, T)), ("bonus", bonus, (R,))):
        chk(name, t, shape, _i32t())
    d, _keep = accept_desc(R, T, V, _dtype_code(logits), parent)
    chk.on_gpu()
    st = lib.accept_greedy_noalloc(ctypes.byref(d), _ptr(logits), _ptr(tokens), _ptr(argmax), _ptr(accept_node),
                                   _ptr(accept_len), _ptr(path), _ptr(bonus), _stream(stream))
    _check(st, "accept_greedy_noalloc")


def rollback_restore(ckpt, state, conv_ckpt, conv_state, accept_node, status, stream=None):
    """ckpt [L,R,T,Hv,dv,dk] f32 -> state [L,R,Hv,dv,dk]; conv_ckpt
    [L,R,T,W-1,C] -> conv_state [L,R,W-1,C] (both None to skip);
    accept_node [R] int32 device; status [>=1] int32 device."""
    L, R, T, Hv, dv, dk = ckpt.shape
    chk = _Checks()
    chk("ckpt", ckpt, None, _f32())
    chk("state", state, (L, R, Hv, dv, dk), _f32())
    chk("accept_node", accept_node, (R,), _i32t())
    chk.status(status, optional=False)
    if (conv_ckpt is None) != (conv_state is None):
        raise ValueError("conv_ckpt and conv_state go together")
    if conv_ckpt is not None:
        cdt_t = _in_dtypes("conv_ckpt", conv_ckpt)
        chk("conv_ckpt", conv_ckpt, None, cdt_t)
        if conv_ckpt.dim() != 5 or tuple(conv_ckpt.shape[:3]) != (L, R, T):
            raise ValueError(f"conv_ckpt: shape {tuple(conv_ckpt.shape)}, expected ({L}, {R}, {T}, W-1, C)")
        C, W1 = conv_ckpt.shape[4], conv_ckpt.shape[3]
        chk("conv_state", conv_state, (L, R, W1, C), cdt_t)
        cdt = _dtype_code(conv_ckpt)
    else:
        C, W1, cdt = 0, 0, HRS_F32
    chk.on_gpu()
    d = RollbackDesc(L, R, T, Hv, dk, dv, C, W1 + 1 if conv_ckpt is not None else 0, cdt)
    st = lib.rollback_restore(ctypes.byref(d), _ptr(ckpt), _ptr(state), _ptr(conv_ckpt), _ptr(conv_state),
                              _ptr(accept_node), _ptr(status), _stream(stream))
    _check(st, "rollback_restore")


def _ring_desc(ring, packed, runs: Sequence[tuple]):
    n_rings, S, D = ring.shape
    dt = _in_dtypes("ring", ring)
    chk = _Checks()
    chk("ring", ring, None, dt)
    chk("packed", packed, None, dt)
    if packed.dim() != 2 or packed.shape[1] != D:
        raise ValueError(f"packed: shape {tuple(packed.shape)}, expected (rows, {D})")
    chk.on_gpu()
    n_packed_rows = packed.shape[0]
    arr = (RingRun * max(1, len(runs)))(*[RingRun(*map(int, r)) for r in runs])
    d = RingDesc(n_rings, S, D, _dtype_code(ring), n_packed_rows, len(runs), arr)
    return d, arr


def ring_set_2d(ring, packed, runs, stream=None):
    """ring [n_rings,S,D]; packed [N,D]; runs: (ring_id, start_pos, n_rows, packed_row)."""
    d, _keep = _ring_desc(ring, packed, runs)
    _check(lib.ring_set_2d(ctypes.byref(d), _ptr(ring), _ptr(packed), _stream(stream)), "ring_set_2d")


def ring_get_2d(ring, packed, runs, stream=None):
    d, _keep = _ring_desc(ring, packed, runs)
    _check(lib.ring_get_2d(ctypes.byref(d), _ptr(ring), _ptr(packed), _stream(stream)), "ring_get_2d")


# --- full-attention layers and sampling --------------------------------------

def _current_stream(device: int) -> int:
    """Raw handle of the current stream. torch's own raw getter where it has
    one: building a Stream object takes 2.5 us, more than the call's checks
    and half of a small launch."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device) if raw is not None else torch.cuda.current_stream().cuda_stream


class PreparedCall:
    """One call of an entry point with its checks done and its arguments laid
    out. Calling it launches on ``stream`` (torch stream or raw handle;
    default: the current one) and reads whatever the same tensors hold by
    then; it keeps them alive. The tensors must not be moved or resized."""

    __slots__ = ("_name", "_fn", "_args", "_keep", "_device")

    def __init__(self, name, args, keep, tensors):
        self._name, self._fn, self._args = name, getattr(lib, name), args
        self._keep, self._device = (keep, tensors), tensors[0].device

    def __call__(self, stream=None) -> None:
        cuda = _torch().cuda
        device = cuda.current_device()
        if device != self._device.index:
            raise ValueError(f"{self._name}: tensors are on {self._device}, the current device is cuda:{device}")
        st = self._fn(*self._args, _current_stream(device) if stream is None else _stream(stream))
        if st != HRS_OK:
            raise HrsError(st, self._name)


class _SpanChecks(_Checks):
    """_Checks with span tensors that may be views of a wider projection, and
    one device for every tensor of the call."""

    def strided(self, name: str, t, shape, dtypes) -> int:
        """Elements from one position to the next of t [..., heads, d]: the
        heads of a position are contiguous and all positions equally far
        apart."""
        if t is None:
            raise ValueError(f"{name} is required")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
        h, d = t.shape[-2:]
        if t.stride(-1) != 1 or (h > 1 and t.stride(-2) != d):
            raise ValueError(f"{name}: the heads of a position must be contiguous")
        stride, n = None, 1
        for size, st in zip(reversed(t.shape[:-2]), reversed(t.stride()[:-2])):
            if size > 1:
                if stride is None:
                    stride = st // n
                if st != stride * n:
                    raise ValueError(f"{name}: positions must be equally far apart")
            n *= size
        stride = h * d if stride is None else stride
        if stride < h * d or stride % 8 != 0:
            raise ValueError(f"{name}: positions {stride} elements apart (at least {h * d}, a multiple of 8)")
        self.seen.append((name, t))
        return stride

    def written(self, *names: str) -> None:
        """The tensors of these names share no byte with any other tensor of
        the call: blocks write them while others read."""
        spans = []
        for name, t in self.seen:
            at = t.data_ptr()
            if t.is_contiguous():
                spans.append((at, at + t.nbytes, name))
            else:
                last = sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
                spans.append((at, at + (last + 1) * t.element_size(), name))
        spans.sort()
        top = 0        # where the last of the spans before ends
        for i, (start, end, name) in enumerate(spans):
            if start < top:
                for _, e, other in spans[:i]:
                    if start < e and (name in names or other in names):
                        raise ValueError(f"{name} overlaps {other}")
            top = max(top, end)

    def on_gpu(self) -> None:
        super().on_gpu()
        dev = self.seen[0][1].device
        for name, t in self.seen:
            if t.device != dev:
                raise ValueError(f"{name} is on {t.device}, {self.seen[0][0]} on {dev}")

    def call(self, name, args, *keep) -> PreparedCall:
        return PreparedCall(name, args, keep, [t for _, t in self.seen])


def _rank(name: str, t, n: int) -> None:
    if t is None or t.dim() != n:
        raise ValueError(f"{name}: {'required' if t is None else f'{t.dim()} dimensions'}, expected {n} dimensions")


def _cache_code(dtype, span_dtype, name: str) -> int:
    torch = _torch()
    ok = (torch.float32,) if span_dtype == torch.float32 else (torch.bfloat16, torch.float8_e4m3fn)
    if dtype not in ok:
        raise TypeError(f"{name}: dtype {dtype}, expected {' or '.join(str(d) for d in ok)} beside {span_dtype} spans")
    return {torch.float32: HRS_F32, torch.bfloat16: HRS_BF16}.get(dtype, HRS_F8E4M3)


def _topo(parent) -> int:
    return HRS_TREE if parent is not None else HRS_CHAIN


def _data(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _scales(chk, shape, cache_code: int, **scales) -> None:
    for name, t in scales.items():
        if t is not None and cache_code != HRS_F8E4M3:
            raise ValueError(f"{name} goes with float8_e4m3fn caches only")
        chk(name, t, shape, _f32(), optional=True)


def qk_norm_rope_call(q, k, q_weight, k_weight, freq, seq_len, q_out, k_out, parent=None, eps: float = 1e-6,
                      weight_offset: float = 0.0, interleaved: bool = False) -> PreparedCall:
    """The PreparedCall of qk_norm_rope (same arguments, without the stream)."""
    _rank("q", q, 4)
    _rank("k", k, 4)
    R, T, Hq, D = q.shape
    Hkv = k.shape[2]
    dt = _in_dtypes("q", q)
    chk = _SpanChecks()
    qs = chk.strided("q", q, (R, T, Hq, D), dt)
    ks = chk.strided("k", k, (R, T, Hkv, D), dt)
    chk("q_weight", q_weight, (D,), dt, optional=True)
    chk("k_weight", k_weight, (D,), dt, optional=True)
    if freq is not None:
        _rank("freq", freq, 1)
    chk("freq", freq, None, (_torch().float64,), optional=True)
    chk("seq_len", seq_len, (R,), _i32t())
    chk("q_out", q_out, (R, T, Hq, D), dt)
    chk("k_out", k_out, (R, T, Hkv, D), dt)
    # In place where that side is dense; blocks still read everything else.
    written = []
    for name, out, x in (("q", q_out, q), ("k", k_out, k)):
        in_place = out.data_ptr() == x.data_ptr() and x.is_contiguous()
        if in_place:
            chk.seen = [(n, y) for n, y in chk.seen if n != f"{name}_out"]
        written.append(name if in_place else f"{name}_out")
    chk.written(*written)
    par, par_p = _parent_array(parent, R, T)
    chk.on_gpu()
    rot = 0 if freq is None else 2 * freq.shape[0]
    d = QkDesc(R, T, Hq, Hkv, D, rot, _dtype_code(q), qs, ks, float(eps), float(weight_offset),
               int(bool(interleaved)), _topo(parent), par_p)
    return chk.call("qk_norm_rope", (ctypes.byref(d), _data(q), _data(k), _data(q_weight), _data(k_weight),
                                     _data(freq) if rot else None, _data(seq_len), _data(q_out), _data(k_out)),
                    d, par)


def qk_norm_rope(q, k, q_weight, k_weight, freq, seq_len, q_out, k_out, parent=None, eps: float = 1e-6,
                 weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """RMS norm of every head of q [R,T,Hq,D] and k [R,T,Hkv,D] (weights [D]
    or None) and the rotation of its first 2 * len(freq) elements by the
    position seq_len[r] + depth(t); freq: float64 radians per position, or
    None for no rotation. q and k may be views of one projection's rows;
    q_out, k_out are dense (q_out may be q itself where q is)."""
    qk_norm_rope_call(q, k, q_weight, k_weight, freq, seq_len, q_out, k_out, parent, eps, weight_offset,
                      interleaved)(stream)


def attn_verify_span_workspace_bytes(n_req: int, n_pos: int, n_heads: int, n_kvheads: int, d: int) -> int:
    """Device workspace bytes attn_verify_span needs for these sizes."""
    a = AttnDesc(n_req, n_pos, n_heads, n_kvheads, d, HRS_BF16, 0, 0, 0, 1.0, 0, CacheDesc(1, 16, 1, HRS_BF16),
                 HRS_CHAIN, None)
    return int(lib.attn_verify_span_workspace_bytes(ctypes.byref(a)))


def _attn_checks(q, k, v, k_cache, v_cache, page_table, seq_len, out, workspace, parent, scale, window, k_scale,
                 v_scale, status):
    """Checks and descriptor of the attention calls: (checks, AttnDesc, what it points to)."""
    _rank("q", q, 4)
    _rank("k", k, 4)
    _rank("k_cache", k_cache, 4)
    _rank("page_table", page_table, 2)
    R, T, Hq, D = q.shape
    Hkv = k.shape[2]
    N, _, S, _ = k_cache.shape
    dt = _in_dtypes("q", q)
    code = _cache_code(k_cache.dtype, q.dtype, "k_cache")
    chk = _SpanChecks()
    qs = chk.strided("q", q, (R, T, Hq, D), dt)
    ks = chk.strided("k", k, (R, T, Hkv, D), dt)
    vs = chk.strided("v", v, (R, T, Hkv, D), dt)
    chk("k_cache", k_cache, (N, Hkv, S, D), (k_cache.dtype,))
    chk("v_cache", v_cache, (N, Hkv, S, D), (k_cache.dtype,))
    chk("page_table", page_table, (R, page_table.shape[1]), _i32t())
    chk("seq_len", seq_len, (R,), _i32t())
    chk("out", out, (R, T, Hq, D), dt)
    chk("workspace", workspace)
    _scales(chk, (Hkv,), code, k_scale=k_scale, v_scale=v_scale)
    chk.status(status)
    par, par_p = _parent_array(parent, R, T)
    cache = CacheDesc(N, S, page_table.shape[1], code)
    d = AttnDesc(R, T, Hq, Hkv, D, _dtype_code(q), qs, ks, vs, float(D ** -0.5 if scale is None else scale),
                 int(window), cache, _topo(parent), par_p)
    return chk, d, par


def attn_verify_span_call(q, k, v, k_cache, v_cache, page_table, seq_len, out, workspace, parent=None, scale=None,
                          window: int = 0, k_scale=None, v_scale=None, status=None) -> PreparedCall:
    """The PreparedCall of attn_verify_span (same arguments, without the stream)."""
    chk, d, par = _attn_checks(q, k, v, k_cache, v_cache, page_table, seq_len, out, workspace, parent, scale, window,
                               k_scale, v_scale, status)
    chk.written("out", "workspace", "status")
    chk.on_gpu()
    nbytes = workspace.numel() * workspace.element_size()
    return chk.call("attn_verify_span",
                    (ctypes.byref(d), _data(q), _data(k), _data(v), _data(k_cache), _data(v_cache), _data(page_table),
                     _data(seq_len), _data(k_scale), _data(v_scale), _data(out), _data(status), _data(workspace),
                     nbytes), d, par)


def attn_verify_span(q, k, v, k_cache, v_cache, page_table, seq_len, out, workspace, parent=None, scale=None,
                     window: int = 0, k_scale=None, v_scale=None, status=None, stream=None):
    """Attention of the span q [R,T,Hq,D] over the paged context (k_cache,
    v_cache [pages,Hkv,slots,D], page_table [R,P], seq_len [R]) and the span's
    own rows k, v [R,T,Hkv,D] along each position's root path. parent: None
    (chain) or host ints [R,T] / [T] (tree). scale: default D ** -0.5. window:
    0 = everything. k_scale, v_scale [Hkv] f32: float8_e4m3fn caches."""
    attn_verify_span_call(q, k, v, k_cache, v_cache, page_table, seq_len, out, workspace, parent, scale, window,
                          k_scale, v_scale, status)(stream)


def attn_verify_shared_workspace_bytes(n_req: int, n_pos: int, n_heads: int, n_kvheads: int, d: int) -> int:
    """Device workspace bytes attn_verify_shared needs for these sizes."""
    a = AttnDesc(n_req, n_pos, n_heads, n_kvheads, d, HRS_BF16, 0, 0, 0, 1.0, 0, CacheDesc(1, 16, 1, HRS_BF16),
                 HRS_CHAIN, None)
    return int(lib.attn_verify_shared_workspace_bytes(ctypes.byref(a)))


def attn_verify_shared_call(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table, seq_len, out, workspace,
                            parent=None, scale=None, window: int = 0, k_scale=None, v_scale=None,
                            status=None) -> PreparedCall:
    """The PreparedCall of attn_verify_shared (same arguments, without the stream)."""
    chk, d, par = _attn_checks(q, k, v, k_cache, v_cache, page_table, seq_len, out, workspace, parent, scale, window,
                               k_scale, v_scale, status)
    _rank("prefix_table", prefix_table, 1)
    chk("prefix_table", prefix_table, None, _i32t())
    chk("prefix_len", prefix_len, (1,), _i32t())
    chk.written("out", "workspace", "status")
    chk.on_gpu()
    nbytes = workspace.numel() * workspace.element_size()
    return chk.call("attn_verify_shared",
                    (ctypes.byref(d), prefix_table.shape[0], _data(q), _data(k), _data(v), _data(k_cache),
                     _data(v_cache), _data(prefix_table), _data(prefix_len), _data(page_table), _data(seq_len),
                     _data(k_scale), _data(v_scale), _data(out), _data(status), _data(workspace), nbytes), d, par)


def attn_verify_shared(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table, seq_len, out, workspace,
                       parent=None, scale=None, window: int = 0, k_scale=None, v_scale=None, status=None, stream=None):
    """attn_verify_span of requests that share a prefix: slots below
    prefix_len [1] are read through prefix_table [n], once for all requests,
    the others through each one's page_table row (seq_len counts both).
    workspace of at least attn_verify_shared_workspace_bytes."""
    attn_verify_shared_call(q, k, v, k_cache, v_cache, prefix_table, prefix_len, page_table, seq_len, out, workspace,
                            parent, scale, window, k_scale, v_scale, status)(stream)


def kv_cache_append_call(k, v, k_cache, v_cache, page_table, seq_len, accept_len, seq_len_out=None, path=None,
                         k_scale=None, v_scale=None, status=None) -> PreparedCall:
    """The PreparedCall of kv_cache_append (same arguments, without the stream)."""
    _rank("k", k, 5)
    _rank("k_cache", k_cache, 5)
    _rank("page_table", page_table, 2)
    L, R, T, Hkv, D = k.shape
    N, S = k_cache.shape[1], k_cache.shape[3]
    dt = _in_dtypes("k", k)
    code = _cache_code(k_cache.dtype, k.dtype, "k_cache")
    chk = _SpanChecks()
    ks = chk.strided("k", k, (L, R, T, Hkv, D), dt)
    vs = chk.strided("v", v, (L, R, T, Hkv, D), dt)
    chk("k_cache", k_cache, (L, N, Hkv, S, D), (k_cache.dtype,))
    chk("v_cache", v_cache, (L, N, Hkv, S, D), (k_cache.dtype,))
    chk("page_table", page_table, (R, page_table.shape[1]), _i32t())
    chk("seq_len", seq_len, (R,), _i32t())
    chk("accept_len", accept_len, (R,), _i32t())
    chk("path", path, (R, T), _i32t(), optional=True)
    _scales(chk, (L, Hkv), code, k_scale=k_scale, v_scale=v_scale)
    chk.status(status)
    chk("seq_len_out", seq_len_out, (R,), _i32t(), optional=True)
    in_place = seq_len_out is not None and seq_len_out.data_ptr() == seq_len.data_ptr()
    if in_place:
        chk.seen.pop()
    chk.written("k_cache", "v_cache", "seq_len" if in_place else "seq_len_out", "status")
    chk.on_gpu()
    d = AppendDesc(L, R, T, Hkv, D, _dtype_code(k), ks, vs, CacheDesc(N, S, page_table.shape[1], code))
    return chk.call("kv_cache_append",
                    (ctypes.byref(d), _data(k), _data(v), _data(k_cache), _data(v_cache), _data(page_table),
                     _data(seq_len), _data(accept_len), _data(path), _data(k_scale), _data(v_scale),
                     _data(seq_len_out), _data(status)), d)


def kv_cache_append(k, v, k_cache, v_cache, page_table, seq_len, accept_len, seq_len_out=None, path=None,
                    k_scale=None, v_scale=None, status=None, stream=None):
    """Rows path[r][0..accept_len[r]] (path None: 0..accept_len[r]) of the
    span's k, v [L,R,T,Hkv,D] into slots seq_len[r] ... of every layer's pages
    (k_cache, v_cache [L,pages,Hkv,slots,D]); seq_len_out [R] (seq_len itself,
    a buffer apart from all others, or None) receives the new lengths."""
    kv_cache_append_call(k, v, k_cache, v_cache, page_table, seq_len, accept_len, seq_len_out, path, k_scale,
                         v_scale, status)(stream)


def sample_desc(n_req: int, n_pos: int, vocab: int, logit_dtype: int, draft_dtype: int = HRS_F32, parent=None):
    par, par_p = _parent_array(parent, n_req, n_pos)
    return SampleDesc(n_req, n_pos, vocab, logit_dtype, draft_dtype, _topo(parent), par_p), par


def accept_sample_workspace_bytes(n_req: int, n_pos: int, vocab: int) -> int:
    """Device workspace bytes accept_sample needs for these sizes."""
    d, _keep = sample_desc(n_req, n_pos, vocab, HRS_BF16)
    return int(lib.accept_sample_workspace_bytes(ctypes.byref(d)))


def _sample_checks(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace, draft_probs,
                   temperature, status, **limits):
    _rank("logits", logits, 3)
    R, T, V = logits.shape
    chk = _SpanChecks()
    chk("logits", logits, None, _in_dtypes("logits", logits))
    chk("tokens", tokens, (R, T), _i32t())
    chk("uniforms", uniforms, (R, T), _f32())
    chk("token_prob", token_prob, (R, T), _f32())
    for name, t, shape in (("accept_node", accept_node, (R,)), ("accept_len", accept_len, (R,)), ("path", path, (R, T)),
                           ("bonus", bonus, (R,))):
        chk(name, t, shape, _i32t())
    chk("workspace", workspace)
    if draft_probs is not None:
        chk("draft_probs", draft_probs, (R, T, V), _in_dtypes("draft_probs", draft_probs))
    chk("temperature", temperature, (R,), _f32(), optional=True)
    for name, t in limits.items():
        chk(name, t, (R,), _i32t() if name == "top_k" else _f32(), optional=True)
    chk.status(status)
    chk.written("token_prob", "accept_node", "accept_len", "path", "bonus", "workspace", "status")
    return chk


def accept_sample_call(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                       draft_probs=None, temperature=None, parent=None, status=None) -> PreparedCall:
    """The PreparedCall of accept_sample (same arguments, without the stream)."""
    chk = _sample_checks(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                         draft_probs, temperature, status)
    R, T, V = logits.shape
    d, par = sample_desc(R, T, V, _dtype_code(logits), HRS_F32 if draft_probs is None else _dtype_code(draft_probs),
                         parent)
    chk.on_gpu()
    nbytes = workspace.numel() * workspace.element_size()
    return chk.call("accept_sample",
                    (ctypes.byref(d), _data(logits), _data(tokens), _data(uniforms), _data(draft_probs),
                     _data(temperature), _data(token_prob), _data(accept_node), _data(accept_len), _data(path),
                     _data(bonus), _data(status), _data(workspace), nbytes), d, par)


def accept_sample(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                  draft_probs=None, temperature=None, parent=None, status=None, stream=None):
    """Acceptance of one draft block per request by sampling. logits [R,T,V];
    tokens [R,T] int32; uniforms [R,T] f32 in [0, 1) (column 0 draws the
    bonus token); draft_probs [R,T,V] (row t: what token t + 1 was drawn
    from; chains) or None (drafts were picked); temperature [R] f32 or None;
    outputs token_prob [R,T] f32 and int32 accept_node [R], accept_len [R],
    path [R,T], bonus [R]."""
    accept_sample_call(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                       draft_probs, temperature, parent, status)(stream)


def accept_sample_filtered_workspace_bytes(n_req: int, n_pos: int, vocab: int) -> int:
    """Device workspace bytes accept_sample_filtered needs for these sizes."""
    d, _keep = sample_desc(n_req, n_pos, vocab, HRS_BF16)
    return int(lib.accept_sample_filtered_workspace_bytes(ctypes.byref(d)))


def accept_sample_filtered_call(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                                top_k=None, top_p=None, min_p=None, draft_probs=None, temperature=None, parent=None,
                                status=None) -> PreparedCall:
    """The PreparedCall of accept_sample_filtered (same arguments, without the stream)."""
    chk = _sample_checks(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                         draft_probs, temperature, status, top_k=top_k, top_p=top_p, min_p=min_p)
    R, T, V = logits.shape
    d, par = sample_desc(R, T, V, _dtype_code(logits), HRS_F32 if draft_probs is None else _dtype_code(draft_probs),
                         parent)
    chk.on_gpu()
    nbytes = workspace.numel() * workspace.element_size()
    return chk.call("accept_sample_filtered",
                    (ctypes.byref(d), _data(logits), _data(tokens), _data(uniforms), _data(draft_probs),
                     _data(temperature), _data(top_k), _data(top_p), _data(min_p), _data(token_prob),
                     _data(accept_node), _data(accept_len), _data(path), _data(bonus), _data(status),
                     _data(workspace), nbytes), d, par)


def accept_sample_filtered(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                           top_k=None, top_p=None, min_p=None, draft_probs=None, temperature=None, parent=None,
                           status=None, stream=None):
    """accept_sample from the target's probabilities after top_k [R] int32 (0:
    none), top_p [R] f32 (1: none) and min_p [R] f32 (0: none), each or None;
    workspace of at least accept_sample_filtered_workspace_bytes. One position
    a request (T = 1): plain sampling, the token in bonus."""
    accept_sample_filtered_call(logits, tokens, uniforms, token_prob, accept_node, accept_len, path, bonus, workspace,
                                top_k, top_p, min_p, draft_probs, temperature, parent, status)(stream)


def _hold_checks(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages, page_size, held_node,
                 temperature):
    """Checks, descriptor and pointers of the accept_hold calls."""
    _rank("path", path, 2)
    _rank("page_table", page_table, 2)
    R, T = path.shape
    chk = _SpanChecks()
    for name, t, shape in (("path", path, (R, T)), ("page_table", page_table, (R, page_table.shape[1])),
                           ("seq_len", seq_len, (R,)), ("accept_node", accept_node, (R,)),
                           ("accept_len", accept_len, (R,)), ("bonus", bonus, (R,)), ("held", held, (R,)),
                           ("last_node", last_node, (R,))):
        chk(name, t, shape, _i32t())
    chk("held_node", held_node, (R,), _i32t(), optional=True)
    chk("temperature", temperature, (R,), _f32(), optional=True)
    chk.written("accept_node", "accept_len", "path", "bonus", "held", "last_node", "held_node")
    chk.on_gpu()
    d = HoldDesc(R, T, n_pages, page_size, page_table.shape[1])
    return chk, d, (_data(page_table), _data(seq_len), _data(temperature), _data(accept_node), _data(accept_len),
                    _data(path), _data(bonus), _data(held), _data(last_node), _data(held_node))


def accept_hold_call(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages: int,
                     page_size: int, held_node=None, temperature=None) -> PreparedCall:
    """The PreparedCall of accept_hold (same arguments, without the stream)."""
    chk, d, ptrs = _hold_checks(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages,
                                page_size, held_node, temperature)
    return chk.call("accept_hold", (ctypes.byref(d), *ptrs), d)


def accept_hold(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages: int,
                page_size: int, held_node=None, temperature=None, stream=None):
    """Requests that cannot go on taken out of an acceptance (accept_node,
    accept_len, bonus [R] and path [R,T] become -1, held [R] 1): pages of
    page_table [R,P] missing or full behind seq_len [R], a temperature [R]
    that is negative or NaN, or held before. The others' accept_node goes to
    last_node [R]; a newly held request's last_node to held_node [R]."""
    accept_hold_call(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages, page_size,
                     held_node, temperature)(stream)


def accept_hold_behind_call(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages: int,
                            page_size: int, prefix_len: int, held_node=None, temperature=None) -> PreparedCall:
    """The PreparedCall of accept_hold_behind (same arguments, without the stream)."""
    chk, d, ptrs = _hold_checks(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages,
                                page_size, held_node, temperature)
    return chk.call("accept_hold_behind", (ctypes.byref(d), prefix_len, *ptrs), d)


def accept_hold_behind(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages: int,
                       page_size: int, prefix_len: int, held_node=None, temperature=None, stream=None):
    """accept_hold of requests behind a prefix that all of them read: those
    with a seq_len below prefix_len are held as well."""
    accept_hold_behind_call(page_table, seq_len, accept_node, accept_len, path, bonus, held, last_node, n_pages, page_size,
                            prefix_len, held_node, temperature)(stream)


# --- page lists -----------------------------------------------------------------

def kv_pages_workspace_bytes(n_req: int) -> int:
    """Device workspace bytes kv_pages_reserve and kv_pages_release need."""
    return int(lib.kv_pages_workspace_bytes(ctypes.byref(PagesDesc(n_req, 1, 1, 16, 1, 0))))


def _pages_checks(page_table, n_held, free_pages, n_free, workspace, status, **lens):
    _rank("page_table", page_table, 2)
    _rank("free_pages", free_pages, 1)
    R, P = page_table.shape
    chk = _SpanChecks()
    for name, t in lens.items():
        chk(name, t, (R,), _i32t(), optional=name in ("n_new", "skip"))
    for name, t, shape in (("page_table", page_table, (R, P)), ("n_held", n_held, (R,)),
                           ("free_pages", free_pages, None), ("n_free", n_free, (1,))):
        chk(name, t, shape, _i32t())
    chk("workspace", workspace)
    chk.status(status)
    return chk, R, P


def _reserve_call(fn, seq_len, page_table, n_held, free_pages, n_free, workspace, page_size, n_pos, n_new, prefix_table,
                  slot_map, status, skip=None) -> PreparedCall:
    chk, R, P = _pages_checks(page_table, n_held, free_pages, n_free, workspace, status, seq_len=seq_len, n_new=n_new,
                              skip=skip)
    if prefix_table is not None:
        _rank("prefix_table", prefix_table, 1)
    chk("prefix_table", prefix_table, None, _i32t(), optional=True)
    if slot_map is not None:
        _rank("slot_map", slot_map, 2)
        n_pos = n_pos or slot_map.shape[1]
    chk("slot_map", slot_map, (R, n_pos), (_torch().int64,), optional=True)
    chk.written("page_table", "n_held", "n_free", "slot_map", "workspace", "status")
    chk.on_gpu()
    d = PagesDesc(R, n_pos, free_pages.shape[0], page_size, P, 0 if prefix_table is None else prefix_table.shape[0])
    nbytes = workspace.numel() * workspace.element_size()
    first = (_data(seq_len), _data(n_new)) + ((_data(skip),) if fn == "kv_pages_reserve_step" else ())
    return chk.call(fn,
                    (ctypes.byref(d), *first, _data(prefix_table) if d.n_prefix else None, _data(page_table),
                     _data(n_held), _data(free_pages), _data(n_free), _data(slot_map), _data(status), _data(workspace),
                     nbytes), d)


def kv_pages_reserve_call(seq_len, page_table, n_held, free_pages, n_free, workspace, page_size: int, n_pos: int = 0,
                          n_new=None, prefix_table=None, slot_map=None, status=None) -> PreparedCall:
    """The PreparedCall of kv_pages_reserve (same arguments, without the stream)."""
    return _reserve_call("kv_pages_reserve", seq_len, page_table, n_held, free_pages, n_free, workspace, page_size, n_pos,
                         n_new, prefix_table, slot_map, status)


def kv_pages_reserve(seq_len, page_table, n_held, free_pages, n_free, workspace, page_size: int, n_pos: int = 0,
                     n_new=None, prefix_table=None, slot_map=None, status=None, stream=None):
    """Pages for slots up to seq_len[r] + n_new[r] (None: n_pos) of every
    request, from the stack free_pages [n_pages], n_free [1] into page_table
    [R,P], n_held [R]; prefix_table: the shared leading entries of every table.
    slot_map [R,n_pos] int64: where the new positions lie. int32 device tensors
    but for slot_map; workspace of at least kv_pages_workspace_bytes."""
    kv_pages_reserve_call(seq_len, page_table, n_held, free_pages, n_free, workspace, page_size, n_pos, n_new,
                          prefix_table, slot_map, status)(stream)


def kv_pages_reserve_step_call(seq_len, page_table, n_held, free_pages, n_free, workspace, page_size: int, n_pos: int = 0,
                               n_new=None, prefix_table=None, slot_map=None, status=None, skip=None) -> PreparedCall:
    """The PreparedCall of kv_pages_reserve_step (same arguments, without the stream)."""
    return _reserve_call("kv_pages_reserve_step", seq_len, page_table, n_held, free_pages, n_free, workspace, page_size,
                         n_pos, n_new, prefix_table, slot_map, status, skip)


def kv_pages_reserve_step(seq_len, page_table, n_held, free_pages, n_free, workspace, page_size: int, n_pos: int = 0,
                          n_new=None, prefix_table=None, slot_map=None, status=None, skip=None, stream=None):
    """kv_pages_reserve up to the end of a request's table, where that refuses
    the request, and without the requests that skip [R] int32 names (any value
    but 0)."""
    kv_pages_reserve_step_call(seq_len, page_table, n_held, free_pages, n_free, workspace, page_size, n_pos, n_new,
                               prefix_table, slot_map, status, skip)(stream)


def kv_pages_release_call(keep_len, page_table, n_held, free_pages, n_free, workspace, page_size: int,
                          n_prefix: int = 0, status=None) -> PreparedCall:
    """The PreparedCall of kv_pages_release (same arguments, without the stream)."""
    chk, R, P = _pages_checks(page_table, n_held, free_pages, n_free, workspace, status, keep_len=keep_len)
    chk.written("page_table", "n_held", "free_pages", "n_free", "workspace", "status")
    chk.on_gpu()
    d = PagesDesc(R, 1, free_pages.shape[0], page_size, P, n_prefix)
    nbytes = workspace.numel() * workspace.element_size()
    return chk.call("kv_pages_release",
                    (ctypes.byref(d), _data(keep_len), _data(page_table), _data(n_held), _data(free_pages),
                     _data(n_free), _data(status), _data(workspace), nbytes), d)


def kv_pages_release(keep_len, page_table, n_held, free_pages, n_free, workspace, page_size: int, n_prefix: int = 0,
                     status=None, stream=None):
    """Pages behind slot keep_len[r] of every request (and the n_prefix
    leading ones) back from page_table [R,P], n_held [R] onto the stack
    free_pages [n_pages], n_free [1]; their entries become -1."""
    kv_pages_release_call(keep_len, page_table, n_held, free_pages, n_free, workspace, page_size, n_prefix,
                          status)(stream)

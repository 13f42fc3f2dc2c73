"""Full-attention layer of the verify span: the oracle (test infrastructure only).

The hybrid target's remaining layers are full attention over a paged cache:
queries and keys are normed per head and rotated by position, the span attends
to the cached context and to its own root paths, and the accepted rows enter
the cache (openinfer PR #626, file table: batched Q/K norm and RoPE, paged
causal-window attention; What Changed: the hybrid state includes the attention
layers' cache; lucebox PR #533, Verification: DDTree).

Definitions, one request, float64 throughout:
  norm_rope   n = x / sqrt(mean(x^2) + eps) * (offset + w); the pair (a, b) of
              angle f turned by (length + depth) * freq[f]
  attn_span   softmax over the visible slots of scale * q . k, times v. Visible
              from position t: context slots in [length + depth - window + 1,
              length) (window 0: all), span positions on t's root path less
              than `window` levels up. Slots of absent pages do not count; no
              visible slot gives zeros.
  append      accepted rows into slots length, length + 1, ... of the pages

Readings: tokens of the context sit at positions 0 .. length - 1 and a span
position at length + depth; a page entry outside [0, pages) is a page that is
not there; e4m3 is the 8-bit format with 4 exponent bits (bias 7), 3 mantissa
bits, no infinities, NaN at 0x7f and 0xff.

Pins (tests/test_oracle_attn.py): rotation by complex numbers and by exact
quarter turns; a one-slot softmax; uniform scores give the mean; a tree node
equals the chain over its root path; the e4m3 table against torch's type.
"""
from __future__ import annotations

from typing import List, Optional

import numpy as np

from .common import widen


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 e4m3 patterns."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            v = np.nan
        elif e == 0:
            v = m * 2.0 ** -9
        else:
            v = (8 + m) * 2.0 ** (e - 10)
        out[b] = -v if b & 128 else v
    return out


def widen_cache(x) -> np.ndarray:
    x = np.asarray(x)
    return e4m3_table()[x] if x.dtype == np.uint8 else widen(x)


def depths(parent) -> List[int]:
    out: List[int] = []
    for p in parent:
        out.append(0 if p < 0 else out[int(p)] + 1)
    return out


def chain(n: int) -> List[int]:
    return list(range(-1, n - 1))


def norm_rope(x, weight, freq, length: int, depth, eps: float, offset: float = 0.0, interleaved: bool = False):
    """x [T, H, d] -> [T, H, d]; weight [d] or None; depth [T]."""
    y = widen(x).copy()
    if weight is not None:
        ms = np.mean(y * y, axis=-1, keepdims=True)
        y = y / np.sqrt(ms + float(np.float32(eps))) * (float(np.float32(offset)) + widen(weight))
    half = len(freq)
    for t in range(y.shape[0]):
        for f in range(half):
            a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
            ang = (length + depth[t]) * float(freq[f])
            c, s = np.cos(ang), np.sin(ang)
            na, nb = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a], y[t, :, b] = na * c - nb * s, nb * c + na * s
    return y


def attn_span(q, k, v, k_cache, v_cache, pages, length: int, parent=None, scale: Optional[float] = None,
              window: int = 0, k_scale=None, v_scale=None, want_bound: bool = False):
    """q [T, Hq, d], k, v [T, Hkv, d]; caches [N, Hkv, S, d]; pages [P].

    want_bound: also sum_j w_j |v_j| [T, Hq, d], the largest scale * |q| . |k|
    over the visible slots and their number ([T, Hq] each), from which the
    tests derive what rounding may do."""
    q, k, v = widen(q), widen(k), widen(v)
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    N, _, S, _ = k_cache.shape
    scale = d ** -0.5 if scale is None else scale
    parent = chain(T) if parent is None else parent
    dep = depths(parent)
    out = np.zeros((T, Hq, d))
    absv, reach, count = np.zeros((T, Hq, d)), np.zeros((T, Hq)), np.zeros((T, Hq), dtype=int)
    slots = [j for j in range(length) if 0 <= int(pages[j // S]) < N]
    at = np.array([int(pages[j // S]) for j in slots], dtype=int)
    off = np.array([j % S for j in slots], dtype=int)
    slots = np.array(slots, dtype=int)
    for g in range(Hkv):
        kc = widen_cache(k_cache[at, g, off]) * (1.0 if k_scale is None else float(k_scale[g]))
        vc = widen_cache(v_cache[at, g, off]) * (1.0 if v_scale is None else float(v_scale[g]))
        for t in range(T):
            seen = slots >= (length + dep[t] - window + 1 if window else 0)
            path, a = [], t
            while a >= 0 and (window == 0 or dep[t] - dep[a] < window):
                path.append(a)
                a = int(parent[a])
            kk = np.concatenate([kc[seen].reshape(-1, d), k[path, g]])
            vv = np.concatenate([vc[seen].reshape(-1, d), v[path, g]])
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                if not len(kk):
                    continue
                s = scale * (kk @ q[t, h])
                w = np.exp(s - np.max(s))
                w /= np.sum(w)
                out[t, h] = w @ vv
                absv[t, h] = w @ np.abs(vv)
                reach[t, h] = np.max(abs(scale) * (np.abs(kk) @ np.abs(q[t, h])))
                count[t, h] = len(kk)
    return (out, absv, reach, count) if want_bound else out


def append(rows, cache, pages, length: int, path, n: int) -> None:
    """rows [T, H, d] -> cache [N, H, S, d] in place, bit patterns as they are."""
    N, _, S, _ = cache.shape
    for i in range(n):
        j = length + i
        p = int(pages[j // S])
        if 0 <= p < N:
            cache[p, :, j % S] = rows[i if path is None else int(path[i])]


def quantize_e4m3(x, scale) -> np.ndarray:
    """float64 values to e4m3 patterns: x / scale in float32, limited to
    +-448, nearest, ties to the even pattern; x [..., H, d], scale [H] or None."""
    y = np.asarray(x, dtype=np.float32)
    if scale is not None:
        y = (y / np.asarray(scale, dtype=np.float32)[:, None]).astype(np.float32)
    y = y.astype(np.float64)
    grid = e4m3_table()[:127]          # 0 .. 448, increasing
    mag = np.minimum(np.abs(y), 448.0)
    with np.errstate(invalid="ignore"):
        hi = np.clip(np.searchsorted(grid, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - grid[lo], grid[hi] - mag
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(np.isnan(y), 127, pick)
    return (pick + np.where(np.signbit(y), 128, 0)).astype(np.uint8)

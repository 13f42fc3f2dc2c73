"""attn_verify_span on the GPU where a block runs many tiles, through several
heads and requests: the ring of tiles is used again, the reference moves
between tiles, pages are read a tile ahead, runs are cut inside heads.

Two checks of every block shape:
  coverage: queries of zero weigh every slot that counts alike, values are
    small whole numbers, so all sums are exact and a result is S / n after a
    reciprocal, a product and the rounding to the output's type: a slot that
    is left out or taken twice shows.
  peaked: scores with a deviation of 6 whose size grows or falls along the
    context, against the formula in 64 bits under the bound of
    test_gpu_attn.py.
"""
import numpy as np
import pytest

from oracle import attn as oa
from oracle.common import widen
from tests.gpu_util import say
from tests.test_gpu_attn import KINDS, OUT, U, Attn, cast, host, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hrs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import hybrid_recurrent_state_amd as m
    return m


def block_shape(cache, d, rows):
    """(rows of a block, slots of a tile, blocks, tiles of the ring) of a
    launch, worked out here for the inputs' sake: that they give a block more
    tiles than its ring holds is asserted below."""
    wide, esz = d == 256, {"f32": 4, "bf16": 2, "f8": 1}[cache]
    cls = 4 if cache == "f8" and not wide and 64 < rows <= 96 else 0 if rows <= 16 else 1 if rows <= 32 else 2 if rows <= 64 else 3
    rt = 3 if cls == 4 else 1 if cls < 3 or wide else 2
    wr = {0: 1, 1: 2, 4: 2, 2: 4}.get(cls, 8 if wide else 4)
    wk = (2 if wide else 4) if cls < 2 else 2 if cls in (2, 4) else 1
    ss = (16 if cls == 0 else (32 if d * esz <= 128 else 16) if cls == 1 else (16 if wide else 32) if cls == 2
          else 16 if cache == "f32" and d == 128 else 32)
    per_cu = 2 if cls >= 3 and not wide else 1
    return 16 * rt * wr, ss * wk, 256 * per_cu, min(3, 131072 // per_cu // (2 * ss * wk * d * esz))


def total_units(cache, d, T, G, Hkv, lens, window):
    rows, ts, blocks, ring = block_shape(cache, d, T * G)
    tiles = lambda n: -(-n // ts) - min(max(n + 1 - window, 0) // ts if window else 0, -(-n // ts))
    per_head = [tiles(n) + -(-T // ts) + 4 for n in lens]
    return sum(per_head) * Hkv * -(-T * G // rows), blocks, ring


class Runs(Attn):
    """Whole small numbers as values, keys whose size changes along the
    context, in place of Attn's (whose 8-bit caches take long to make)."""

    def __init__(self, R, T, G, Hkv, d, S, lens, dtype, cache, tree, window, seed):
        rng = np.random.default_rng(seed)
        self.shape = (R, T, G * Hkv, Hkv, d, S)
        self.lens, self.dtype, self.cache, self.window, self.scale = list(lens), dtype, cache, window, 6.0 * d ** -0.5
        P = max(1, -(-max(lens) // S))
        self.P, self.N = P, R * P + 3
        self.pages = rng.permutation(self.N)[:R * P].reshape(R, P).astype(np.int32)
        f = lambda *s: rng.standard_normal(s, dtype=np.float32)
        whole = lambda *s: rng.integers(-8, 9, s).astype(np.float32)
        self.q, self.k, self.v = cast(f(R, T, G * Hkv, d), dtype), cast(f(R, T, Hkv, d), dtype), cast(whole(R, T, Hkv, d), dtype)
        self.ks = self.vs = None
        # slot j of request r: keys 0.5 to 1 times a normal number, larger with j or smaller
        gain = np.ones((self.N, S), dtype=np.float32)
        for r in range(R):
            ramp = np.linspace(0.5, 1.0, P * S, dtype=np.float32)
            gain[self.pages[r]] = (ramp if r % 2 == 0 else ramp[::-1]).reshape(P, S)
        size = (self.N, Hkv, S, d)
        if cache == "f8":
            table = oa.quantize_e4m3(np.concatenate([rng.standard_normal(4096) * g * 50 for g in np.linspace(0.5, 1, 8)]), None)
            level = np.rint((gain - 0.5) * 14).astype(np.int32)[:, None, :, None]
            self.kc = table[level * 4096 + rng.integers(0, 4096, size, dtype=np.int32)]
            self.vc = oa.quantize_e4m3(np.arange(-8.0, 9.0), None)[rng.integers(0, 17, size)]
            self.ks = rng.uniform(0.018, 0.022, Hkv).astype(np.float32)
            self.vs = np.full(Hkv, 0.25, dtype=np.float32)
            self.v = cast(widen(self.v) * 0.25, dtype)
        else:
            self.kc, self.vc = cast(f(*size) * gain[:, None, :, None], cache), cast(whole(*size), cache)
        self.parent = np.stack([random_tree(rng, T) for _ in range(R)]) if tree else None

    def counted(self, r, t):
        """Whether position t counts each slot of the context, and its path."""
        T, S = self.shape[1], self.shape[5]
        par = oa.chain(T) if self.parent is None else self.parent[r]
        dep, j = oa.depths(par), np.arange(self.lens[r])
        pg = self.pages[r][j // S]
        seen = (pg >= 0) & (pg < self.N)
        if self.window:
            seen &= j > self.lens[r] + dep[t] - self.window
        path, x = [], t
        while x >= 0 and (not self.window or dep[t] - dep[x] < self.window):
            path.append(x)
            x = int(par[x])
        return seen, path

    def head(self, r, g):
        """Keys and values of the context and the span, in 64 bits."""
        S = self.shape[5]
        j = np.arange(self.lens[r])
        pg = np.where((self.pages[r][j // S] >= 0) & (self.pages[r][j // S] < self.N), self.pages[r][j // S], 0)
        out = []
        for c, s, x in ((self.kc, self.ks, self.k), (self.vc, self.vs, self.v)):
            y = oa.widen_cache(c[pg, g, j % S])
            out.append(np.concatenate([y if s is None else y * float(s[g]), widen(x)[r, :, g]]))
        return out

    def check_runs(self, got, r, g, flat):
        R, T, Hq, Hkv, d, S = self.shape
        G = Hq // Hkv
        k, v = self.head(r, g)
        n = self.lens[r]
        mask = np.zeros((T, n + T), dtype=bool)
        for t in range(T):
            seen, path = self.counted(r, t)
            mask[t, :n] = seen
            mask[t, [n + x for x in path]] = True
        out = widen(host(got[r, :, g * G:(g + 1) * G]))                      # [T, G, d]
        assert not np.isnan(out).any(), (r, g)
        if flat:
            want = ((mask @ v) / mask.sum(1)[:, None])[:, None, :]
            # A weight's lower part is 2^-40 of it where the upper one is all
            # of it: lost beside a sum that is not zero, 2^-40 of values up to
            # 8 where it is.
            tol = (3 * U + OUT[self.dtype] * (1 + 3 * U)) * np.abs(want) + 2.0 ** -37
            assert np.all(np.abs(out - want) <= tol), (r, g, float(np.max(np.abs(out - want) / (tol + 1e-300))))
            return
        q = widen(self.q)[r, :, g * G:(g + 1) * G].reshape(T * G, d)
        m = np.repeat(mask, G, axis=0)
        s = np.where(m, self.scale * (q @ k.T), -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        reach = np.max(np.where(m, self.scale * (np.abs(q) @ np.abs(k).T), 0), 1)
        rel = (2 * (2 * (d + 4) * U) * reach + (2 * m.sum(1) + 16) * U + (2.0 ** -8 if self.dtype == "bf16" else 0))[:, None]
        want, absv = w @ v, w @ np.abs(v)
        e = rel * absv
        if self.cache == "f8":
            # float16 weights end at 2^-25 beside a largest one of 2^7 at
            # least: 2^-32 of it for every slot, of values up to the largest.
            e = e + (m.sum(1) * 2.0 ** -32)[:, None] * np.abs(v).max()
        tol = e + OUT[self.dtype] * (np.abs(want) + e)
        err = np.abs(out.reshape(T * G, d) - want)
        assert np.all(err <= tol), (r, g, float(np.max(err / (tol + 1e-300))))


ROWS = [(3, 4), (7, 4), (9, 6), (9, 8), (17, 6), (23, 8)]     # positions, group: 12, 28, 54, 72, 102 and 184 rows a key head


def check_both(hrs, a, head):
    import torch
    R = a.shape[0]
    q = a.q
    for flat in (True, False):
        a.q = np.zeros_like(q) if flat else q
        got = a.run(hrs)
        for r in range(R) if R <= 8 else range(0, R, 7):
            a.check_runs(got, r, head(r), flat)
        assert torch.equal(a.run(hrs), got)


# The shorter runs at one head size.
MANY = [(d, rows, ratio) for d in (64, 128, 256) for rows in ROWS for ratio in (1.5, 3, 8) if ratio == 8 or d == 128]


@pytest.mark.parametrize("d,rows,ratio", MANY, ids=[f"d{d}rows{T * G}x{ratio}" for d, (T, G), ratio in MANY])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_runs_of_many_tiles(hrs, dtype, cache, d, rows, ratio):
    """Four ragged requests, one of them without a context, three key heads:
    1.5, 3 and 8 units a block. Chains and trees, with and without a window,
    absent pages."""
    T, G = rows
    tree, windowed = (ROWS.index(rows) // 2 + d // 128) % 2 == 1, (ROWS.index(rows) + d // 128) % 2 == 1
    Hkv, S = 3, 32 if d == 128 else 64
    shape = block_shape(cache, d, T * G)
    top = int(ratio * shape[2] * shape[1] / (Hkv * -(-T * G // shape[0]) * 2.08)) + 70
    lens = [top, int(0.37 * top) + 1, 0, int(0.71 * top) // S * S]
    window = lens[3] if windowed else 0
    if windowed:
        lens[0] += lens[3] // 3
    units, blocks, ring = total_units(cache, d, T, G, Hkv, lens, window)
    assert 0.85 * ratio < units / blocks < 1.4 * ratio, (units, blocks)
    if ratio == 8:
        assert units / blocks > ring + 1
    a = Runs(4, T, G, Hkv, d, S, lens, dtype, cache, tree, window, seed=T * G + d)
    for r, at in ((0, 0.4), (0, 0.41), (3, 0.9)):
        a.pages[r, int(at * lens[r]) // S] = -1 - r
    a.pages[1, 1] = a.N
    check_both(hrs, a, lambda r: (r + T) % 3)
    say(f"  runs {a.shape} {cache}: {units} units on {blocks} blocks")


@pytest.mark.parametrize("rows", ROWS, ids=lambda x: f"rows{x[0] * x[1]}")
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_runs_through_several_heads_and_requests(hrs, dtype, cache, rows):
    """Sixty-four requests of 16 key heads with contexts of a few tiles at
    most: a block takes several whole heads, of more than one request."""
    T, G = rows
    rng = np.random.default_rng(T)
    lens = [int(x) for x in rng.integers(0, 130, 64)]
    units, blocks, _ = total_units(cache, 64, T, G, 16, lens, 0)
    assert units / blocks > 11
    a = Runs(64, T, G, 16, 64, 16, lens, dtype, cache, tree=T % 2 == 1 and G < 8, window=0, seed=T * G)
    check_both(hrs, a, lambda r: (r + T) % 16)

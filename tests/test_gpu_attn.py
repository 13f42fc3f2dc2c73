"""qk_norm_rope, attn_verify_span and kv_cache_append on the GPU against the
float64 oracle.

Tolerances count roundings (u = 2^-24 for float32 sums and products, 2^-8 for
one rounding to bf16, the largest relative error of each):
  norm_rope: an element is x * r * w of a sum of d squares (every lane adds 8
    terms, then 5 levels), one reciprocal root, then two products and a sum
    with a sine good to 2 ulp and a turn rounded to float32 (3.2 u at most):
    under 32 u of |n_a| + |n_b|, plus one rounding to the output's type.
  attention: a score is a sum of d products (2 (d + 4) u of scale |q| . |k|,
    in any order), a weight's relative error is at most twice the largest
    score error plus 8 u, the sums over n visible slots add 2 n u; a bf16 span
    rounds each weight (2^-8). All relative to sum w |v|. Plus one rounding to
    the output's type. Cached e4m3 values times their scale: two more u each.
"""
import numpy as np
import pytest

from oracle import attn as oa
from oracle.common import widen
from synth import bf16_bits
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
OUT = {"f32": U, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def hrs():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import hybrid_recurrent_state_amd as m
    return m


def cast(x, dtype):
    x = np.ascontiguousarray(x, dtype=np.float32)
    return x if dtype == "f32" else bf16_bits(x)


def dev(x):
    """float32, bf16 bits (uint16), e4m3 bits (uint8) or integers on the GPU."""
    import torch
    x = np.ascontiguousarray(x)
    if x.dtype == np.uint16:
        return torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)
    if x.dtype == np.uint8:
        return torch.from_numpy(x).cuda().view(torch.float8_e4m3fn)
    return torch.from_numpy(x).cuda()


def host(t):
    import torch
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).cpu().numpy()
    return t.cpu().numpy()


def random_tree(rng, T):
    return np.array([-1] + [int(rng.integers(max(0, t - 9), t)) for t in range(1, T)], dtype=np.int32)


# --- qk_norm_rope -----------------------------------------------------------

ROPE = [
    # R, T, Hq, Hkv, d, rot, dtype, tree, interleaved, packed, weights, offset, lengths
    (1, 1, 24, 4, 256, 64, "bf16", False, False, True, True, 0.0, [98304]),
    (3, 17, 8, 2, 128, 128, "bf16", False, False, False, True, 1.0, [0, 7, 262144]),
    (2, 23, 6, 3, 64, 32, "f32", True, False, True, True, 1.0, [1000, 5]),
    (2, 5, 4, 4, 64, 64, "f32", False, True, False, True, 0.0, [1, 999999]),
    (1, 64, 1, 1, 16, 16, "f32", True, True, False, False, 0.0, [31]),
    (2, 9, 3, 1, 96, 48, "bf16", False, False, True, True, 0.0, [4095, 12]),
    (1, 700, 5, 2, 80, 0, "f32", False, False, False, True, 0.0, [3]),
    (1, 601, 5, 1, 208, 112, "bf16", False, True, True, False, 0.0, [77]),
    (70, 64, 2, 1, 64, 32, "bf16", True, False, False, True, 0.0, list(range(70))),   # several launches
]


@pytest.mark.parametrize("case", ROPE, ids=lambda c: f"R{c[0]}T{c[1]}h{c[2]}-{c[3]}d{c[4]}r{c[5]}{c[6]}{'t' if c[7] else ''}{'i' if c[8] else ''}")
def test_norm_rope(hrs, case):
    import torch
    R, T, Hq, Hkv, d, rot, dt, tree, inter, packed, weights, offset, lens = case
    rng = np.random.default_rng(R * 1000 + T + d)
    pre, post = (8, 16) if packed else (0, 0)          # other columns of the projection, kept out
    qkv = cast(rng.standard_normal((R, T, pre + (Hq + Hkv) * d + post)) * 3, dt)
    full = dev(qkv)
    q = full[..., pre:pre + Hq * d].unflatten(-1, (Hq, d))
    k = full[..., pre + Hq * d:pre + (Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    w = [cast(1 - offset + 0.3 * rng.standard_normal(d), dt) if weights else None for _ in range(2)]
    freq = 1e6 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    par = np.stack([random_tree(rng, T) for _ in range(R)]) if tree else None
    qo, ko = torch.full((R, T, Hq, d), 77.0, dtype=q.dtype, device="cuda"), torch.full((R, T, Hkv, d), 77.0, dtype=q.dtype, device="cuda")
    hrs.qk_norm_rope(q, k, *[None if x is None else dev(x) for x in w], dev(freq) if rot else None,
                     dev(np.array(lens, dtype=np.int32)), qo, ko, parent=par, eps=1e-6, weight_offset=offset,
                     interleaved=inter)
    half = rot // 2
    for x, wt, got in ((q, w[0], host(qo)), (k, w[1], host(ko))):
        src, got = host(x), widen(got)
        for r in range(R):
            dep = oa.depths(par[r]) if tree else list(range(T))
            ref = oa.norm_rope(src[r], wt, freq, lens[r], dep, 1e-6, offset, inter)
            mag = np.abs(oa.norm_rope(src[r], wt, [], lens[r], dep, 1e-6, offset))
            size = mag.copy()
            for f in range(half):
                a, b = (2 * f, 2 * f + 1) if inter else (f, f + half)
                size[..., a] = size[..., b] = mag[..., a] + mag[..., b]
            err = np.abs(got[r] - ref)
            tol = 32 * U * size + OUT[dt] * np.abs(ref) + 32 * U * OUT[dt] * size
            assert np.all(err <= tol), (r, float(np.max(err / (tol + 1e-300))))


def test_norm_rope_in_place_and_guard(hrs):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 3, 4, 64, generator=g, device="cuda")
    k = torch.randn(2, 3, 2, 64, generator=g, device="cuda")
    freq = torch.tensor([0.5, 0.25, 0.1, 0.01, 1, 2, 3, 4], dtype=torch.float64, device="cuda")
    n = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    buf = torch.full((2 * 3 * 4 * 64 + 128,), 5.0, device="cuda")
    qo = buf[64:-64].view(2, 3, 4, 64)
    ko = torch.empty_like(k)
    hrs.qk_norm_rope(q, k, None, None, freq, n, qo, ko)
    assert bool((buf[:64] == 5).all()) and bool((buf[-64:] == 5).all())
    hrs.qk_norm_rope(q, k, None, None, freq, n, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


# --- attn_verify_span ---------------------------------------------------------

class Attn:
    """One attention problem: host arrays in the kernel layouts."""

    def __init__(self, R, T, Hq, Hkv, d, S, lens, dtype="bf16", cache="bf16", tree=False, window=0, seed=0, gain=1.0,
                 table_len=None, scale=None):
        rng = np.random.default_rng(seed + 17 * R + T + d)
        self.shape = (R, T, Hq, Hkv, d, S)
        self.lens, self.dtype, self.cache, self.window, self.scale = list(lens), dtype, cache, window, scale
        P = table_len or max(1, -(-max(lens) // S))
        self.P, self.N = P, R * P + 3
        self.pages = rng.permutation(self.N)[:R * P].reshape(R, P).astype(np.int32)
        f = lambda *s: rng.standard_normal(s, dtype=np.float32) * np.float32(gain)
        self.q, self.k, self.v = (cast(f(R, T, h, d), dtype) for h in (Hq, Hkv, Hkv))
        self.ks = self.vs = None
        if cache == "f8":
            self.ks, self.vs = (rng.uniform(0.01, 0.03, Hkv).astype(np.float32) for _ in range(2))
            self.kc, self.vc = (oa.quantize_e4m3(f(self.N, Hkv, S, d) * 50, None) for _ in range(2))
        else:
            self.kc, self.vc = (cast(f(self.N, Hkv, S, d), cache) for _ in range(2))
        self.parent = np.stack([random_tree(rng, T) for _ in range(R)]) if tree else None

    def run(self, hrs, out=None, status=None, stream=None, ws=None):
        import torch
        R, T, Hq, Hkv, d, S = self.shape
        n = hrs.attn_verify_span_workspace_bytes(R, T, Hq, Hkv, d)
        assert n > 0
        if ws is None:
            ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")     # contents must not matter: NaNs
        q = dev(self.q)
        if out is None:
            out = torch.full((R, T, Hq, d), 77.0, dtype=q.dtype, device="cuda")
        opt = lambda x: None if x is None else dev(x)
        hrs.attn_verify_span(q, dev(self.k), dev(self.v), dev(self.kc), dev(self.vc), dev(self.pages),
                             dev(np.array(self.lens, dtype=np.int32)), out, ws, parent=self.parent, scale=self.scale,
                             window=self.window, k_scale=opt(self.ks), v_scale=opt(self.vs), status=status,
                             stream=stream)
        return out

    def check(self, got, requests=None, what=""):
        R, T, Hq, Hkv, d, S = self.shape
        got = widen(host(got))
        worst = 0.0
        for r in range(R) if requests is None else requests:
            ref, absv, reach, n = oa.attn_span(
                self.q[r], self.k[r], self.v[r], self.kc, self.vc, self.pages[r], self.lens[r],
                None if self.parent is None else self.parent[r], self.scale, self.window, self.ks, self.vs, want_bound=True)
            rel = 2 * (2 * (d + 4) * U) * reach + (2 * n + 16) * U + (2.0 ** -8 if self.dtype == "bf16" else 0)
            tol = rel[..., None] * absv + OUT[self.dtype] * (np.abs(ref) + rel[..., None] * absv)
            err = np.abs(got[r] - ref)
            assert not np.isnan(got[r]).any(), (what, r, "NaN")
            assert np.all(err <= tol), (what, r, float(np.max(err / (tol + 1e-300))))
            worst = max(worst, float(np.max(err / (tol + 1e-300))))
        say(f"  attn {what} {self.shape} {self.dtype}/{self.cache}: largest error {worst:.2f} of its bound")


GRID = [
    # R, T, Hq, Hkv, d, S, lens, dtype, cache, tree, window
    (1, 1, 1, 1, 64, 16, [0], "f32", "f32", False, 0),
    (1, 1, 1, 1, 64, 16, [1], "bf16", "bf16", False, 0),
    (1, 1, 24, 4, 256, 64, [1000], "bf16", "bf16", False, 0),
    (2, 1, 8, 8, 128, 16, [0, 333], "bf16", "bf16", False, 0),
    (1, 17, 24, 4, 256, 64, [517], "bf16", "bf16", False, 0),
    (3, 9, 4, 4, 64, 32, [200, 0, 31], "f32", "f32", False, 0),
    (2, 23, 32, 8, 128, 16, [300, 127], "bf16", "bf16", True, 0),
    (1, 64, 16, 2, 64, 128, [700], "bf16", "bf16", True, 0),
    (2, 64, 8, 1, 128, 16, [65, 64], "bf16", "f8", True, 0),
    (1, 33, 12, 2, 256, 16, [129], "bf16", "f8", False, 0),
    (2, 3, 5, 1, 64, 1024, [1025, 63], "bf16", "f8", False, 0),
    (1, 7, 6, 2, 256, 32, [95], "f32", "f32", True, 0),
    (1, 64, 8, 2, 128, 16, [90], "f32", "f32", False, 0),
    (2, 17, 4, 2, 128, 16, [400, 20], "bf16", "bf16", True, 50),
    (1, 17, 4, 2, 64, 16, [400], "f32", "f32", False, 1),
    (1, 40, 6, 1, 128, 64, [333], "bf16", "bf16", True, 3),
    (1, 5, 64, 1, 64, 16, [257], "bf16", "bf16", False, 100),
    (5, 2, 3, 3, 64, 16, [0, 1, 16, 17, 2049], "bf16", "bf16", False, 0),
    (1, 1, 8, 2, 128, 64, [20000], "bf16", "bf16", False, 0),
    (1, 4, 8, 2, 128, 64, [9001], "bf16", "f8", False, 2048),
    (1, 2, 4, 2, 64, 32, [6007], "f32", "f32", False, 0),
    (2, 17, 8, 2, 128, 16, [517, 40], "bf16", "f8", False, 0),
    (1, 20, 4, 1, 128, 64, [1500], "bf16", "f8", True, 77),
    (3, 11, 6, 1, 64, 32, [0, 64, 799], "bf16", "f8", True, 0),
    (1, 64, 6, 6, 256, 16, [300], "f32", "f32", True, 0),
    (1, 29, 4, 2, 256, 64, [1100], "bf16", "f8", False, 500),
    (1, 8, 12, 2, 128, 16, [222], "bf16", "f8", True, 0),
    (1, 12, 2, 1, 256, 32, [130], "f32", "f32", False, 9),
    (1, 64, 16, 1, 256, 16, [120], "bf16", "bf16", True, 0),
]


@pytest.mark.parametrize("case", GRID, ids=lambda c: f"R{c[0]}T{c[1]}h{c[2]}-{c[3]}d{c[4]}p{c[5]}n{max(c[6])}{c[7]}{c[8]}{'t' if c[9] else ''}w{c[10]}")
def test_attn_vs_oracle(hrs, case):
    R, T, Hq, Hkv, d, S, lens, dt, ct, tree, window = case
    a = Attn(R, T, Hq, Hkv, d, S, lens, dt, ct, tree, window)
    a.check(a.run(hrs), what="grid")


def test_attn_many_requests_over_several_launches(hrs):
    rng = np.random.default_rng(3)
    a = Attn(130, 25, 2, 1, 64, 16, [int(x) for x in rng.integers(0, 120, 130)], tree=True)
    a.check(a.run(hrs), what="130 trees")


def test_attn_strided_views_of_one_projection(hrs):
    import torch
    a = Attn(2, 5, 6, 2, 64, 16, [40, 99], "bf16", "bf16")
    R, T, Hq, Hkv, d, S = a.shape
    full = torch.cat([dev(a.q).flatten(2), dev(a.k).flatten(2), dev(a.v).flatten(2)], -1)
    cut = lambda lo, h: full[..., lo * d:(lo + h) * d].unflatten(-1, (h, d))
    ws = torch.empty(hrs.attn_verify_span_workspace_bytes(*a.shape[:5]), dtype=torch.uint8, device="cuda")
    out = torch.empty(R, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    hrs.attn_verify_span(cut(0, Hq), cut(Hq, Hkv), cut(Hq + Hkv, Hkv), dev(a.kc), dev(a.vc), dev(a.pages),
                         dev(np.array(a.lens, dtype=np.int32)), out, ws)
    assert torch.equal(out, a.run(hrs))


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")])
@pytest.mark.parametrize("tree", [False, True])
def test_attn_what_does_not_count_has_no_influence(hrs, dtype, cache, tree):
    """NaN and infinities in every slot behind the length, in every page that
    no table names, and, in turn, in every span row that is off one node's
    path: that node's result stays the same, bit for bit."""
    import torch
    a = Attn(2, 9, 4, 2, 64, 16, [37, 90], dtype, cache, tree)
    clean = a.run(hrs)
    bad = {"f32": np.float32(np.nan), "bf16": np.uint16(0x7FC0), "f8": np.uint8(0x7F)}
    inf = {"f32": np.float32(np.inf), "bf16": np.uint16(0xFF80), "f8": np.uint8(0xFF)}
    used = np.zeros((a.N, 16), dtype=bool)
    for r, n in enumerate(a.lens):
        for j in range(n):
            used[a.pages[r][j // 16], j % 16] = True
    for c, fill in ((a.kc, inf), (a.vc, bad)):
        c.transpose(0, 2, 1, 3)[~used] = fill[cache]
    assert torch.equal(a.run(hrs), clean)
    k0, v0 = a.k.copy(), a.v.copy()
    for node in (0, 4, 8):
        a.k, a.v = k0.copy(), v0.copy()
        for r in range(2):
            par = a.parent[r] if tree else oa.chain(9)
            path, x = set(), node
            while x >= 0:
                path.add(x)
                x = int(par[x])
            off = [t for t in range(9) if t not in path]
            a.k[r, off], a.v[r, off] = bad[dtype], inf[dtype]
        got = a.run(hrs)
        assert torch.equal(got[:, node], clean[:, node]), node


KINDS = [("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")]


@pytest.mark.parametrize("group", [1, 3, 7, 8, 12])       # 9 to 108 rows a key head: every class of blocks
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_attn_odd_values_at_every_block_shape(hrs, dtype, cache, d, group):
    """Infinities and NaN in places that count come through exactly where the
    formula has them, in places that do not count they change nothing: a
    context of three requests (one a whole number of tiles, one that ends inside
    one, one without), a tree, an absent page."""
    import torch
    a = Attn(3, 9, 2 * group, 2, d, 16, [37, 256, 0], dtype, cache, tree=True, seed=d + group)
    a.pages[1, 3] = -7
    clean = a.run(hrs)
    a.check(clean, what="clean")
    bad = {"f32": np.float32(np.nan), "bf16": np.uint16(0x7FC0), "f8": np.uint8(0x7F)}
    pos = {"f32": np.float32(np.inf), "bf16": np.uint16(0x7F80), "f8": np.uint8(0x7F)}
    neg = {"f32": np.float32(-np.inf), "bf16": np.uint16(0xFF80), "f8": np.uint8(0xFF)}
    used = np.zeros((a.N, 16), dtype=bool)
    for r, n in enumerate(a.lens):
        for j in range(n):
            if 0 <= a.pages[r][j // 16] < a.N:
                used[a.pages[r][j // 16], j % 16] = True
    for c, fill in ((a.kc, neg), (a.vc, bad)):
        c.transpose(0, 2, 1, 3)[~used] = fill[cache]
    assert torch.equal(a.run(hrs), clean)
    def put(r, j, col, x):                                # a value of a cached slot, second key head
        a.vc[a.pages[r][j // 16], 1, j % 16, col] = x[cache]
    put(0, 5, 3, pos)
    put(0, 36, 7, neg)
    put(0, 5, 11, pos)
    put(0, 36, 11, neg)
    put(1, 250, 2, neg)
    put(1, 17, d - 1, bad)
    a.v[2, 4, 0, 20] = pos[dtype]
    a.v[1, 8, 1, 21] = bad[dtype]
    got = widen(host(a.run(hrs)))
    for r in range(3):
        with np.errstate(invalid="ignore"):
            ref, absv, reach, n = oa.attn_span(a.q[r], a.k[r], a.v[r], a.kc, a.vc, a.pages[r], a.lens[r], a.parent[r],
                                               None, 0, a.ks, a.vs, want_bound=True)
            assert np.array_equal(np.isnan(got[r]), np.isnan(ref)), r
            assert np.array_equal(got[r][np.isinf(ref)], ref[np.isinf(ref)]), r
            rel = 2 * (2 * (d + 4) * U) * reach + (2 * n + 16) * U + (2.0 ** -8 if dtype == "bf16" else 0)
            tol = rel[..., None] * absv + OUT[dtype] * (np.abs(ref) + rel[..., None] * absv)
            fin = np.isfinite(ref)
            assert np.all(np.abs(got[r] - ref)[fin] <= tol[fin]), r
    assert np.isnan(got).any()


def test_attn_two_streams_at_once(hrs):
    """Two calls on two streams, each with a workspace of its own."""
    import torch
    cases = [Attn(2, 17, 8, 2, 128, 16, [3000, 900], "bf16", "bf16", seed=1),
             Attn(1, 5, 4, 2, 256, 32, [5000], "bf16", "f8", seed=2)]
    want = [c.run(hrs) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    calls, outs = [], []
    for c, w in zip(cases, want):
        R, T, Hq, Hkv, d, S = c.shape
        ws = torch.empty(hrs.attn_verify_span_workspace_bytes(R, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
        outs.append(torch.zeros_like(w))
        opt = lambda x: None if x is None else dev(x)
        calls.append(hrs.attn_verify_span_call(dev(c.q), dev(c.k), dev(c.v), dev(c.kc), dev(c.vc), dev(c.pages),
                                               dev(np.array(c.lens, dtype=np.int32)), outs[-1], ws,
                                               k_scale=opt(c.ks), v_scale=opt(c.vs)))
    torch.cuda.synchronize()
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for call, st in zip(calls, streams):
            call(st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_attn_nan_that_counts_is_seen(hrs):
    import torch
    a = Attn(1, 3, 2, 1, 64, 16, [20], "f32", "f32")
    a.v[0, 1, 0, 5] = np.nan
    got = a.run(hrs)
    assert not torch.isnan(got[0, 0]).any()
    assert torch.isnan(got[0, 1:, :, 5]).all() and int(torch.isnan(got).sum()) == 4


def test_attn_absent_pages(hrs):
    """Pages that are not there do not count; a query that nothing counts for
    cannot come about from them alone (its own row counts), so the window and
    the pages together leave just that row."""
    a = Attn(2, 4, 4, 2, 64, 16, [100, 64], "bf16", "bf16")
    a.pages[0, [0, 3]] = [-1, a.N]
    a.pages[1, :] = [2 ** 31 - 1, -2 ** 31, -5, a.N + 1, 0, 0, 0][:a.P]
    got = a.run(hrs)
    a.check(got, what="absent pages")
    b = Attn(1, 2, 2, 2, 128, 16, [70], "f32", "f32", window=1)
    b.check(b.run(hrs), what="window 1")


def test_attn_bad_lengths_are_left_alone_and_counted(hrs):
    import torch
    a = Attn(4, 3, 4, 2, 64, 16, [30, 40, 50, 64], "bf16", "bf16", table_len=4)
    a.lens = [30, -1, 65, 64]
    status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    got = a.run(hrs, status=status)
    assert status.tolist() == [2, 9, 9, 9]
    assert bool((got[1:3] == 77).all())
    a.check(got, requests=[0, 3], what="beside bad lengths")


@pytest.mark.parametrize("gain", [1e-3, 30.0])
def test_attn_flat_and_peaked_scores(hrs, gain):
    a = Attn(1, 6, 4, 1, 128, 32, [500], "f32", "f32", gain=gain, seed=5)
    a.check(a.run(hrs), what=f"gain {gain}")


def test_attn_negative_scale_and_large_scores(hrs):
    a = Attn(1, 6, 4, 2, 64, 32, [300], "f32", "f32", scale=-0.3)
    a.check(a.run(hrs), what="negative scale")
    a = Attn(1, 6, 4, 2, 64, 32, [300], "bf16", "bf16", scale=0.0)
    a.check(a.run(hrs), what="zero scale")


def test_attn_repeat_is_bit_identical_and_guarded(hrs):
    import torch
    a = Attn(3, 17, 8, 2, 128, 16, [1500, 3, 700], "bf16", "bf16", tree=True)
    first = a.run(hrs)
    for _ in range(3):
        assert torch.equal(a.run(hrs), first)
    buf = torch.full((first.numel() + 256,), 3.0, dtype=torch.bfloat16, device="cuda")
    n = hrs.attn_verify_span_workspace_bytes(*a.shape[:5])
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    a.run(hrs, out=buf[128:-128].view(first.shape), ws=ws[256:-256])
    assert torch.equal(buf[128:-128].view(first.shape), first)
    assert bool((buf[:128] == 3).all()) and bool((buf[-128:] == 3).all())
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[-256:] == 0xA5).all())


def test_attn_pages_behind_2_31_elements(hrs):
    """A cache whose last pages start beyond 2^31 elements and 2^32 bytes."""
    import torch
    N, H, S, d = 70000, 4, 64, 128          # 2.3e9 elements a side, 4.6 GB
    a = Attn(1, 2, 4, 4, d, S, [150], "bf16", "bf16")
    big = [torch.zeros(N, H, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far = np.array([[69999, 40000, 69998]], dtype=np.int32)
    for b, c in zip(big, (a.kc, a.vc)):
        b[torch.from_numpy(far[0]).long().cuda()] = dev(c[a.pages[0]])
    out = torch.empty(1, 2, 4, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(hrs.attn_verify_span_workspace_bytes(1, 2, 4, 4, d), dtype=torch.uint8, device="cuda")
    hrs.attn_verify_span(dev(a.q), dev(a.k), dev(a.v), big[0], big[1], dev(far), dev(np.array([150], dtype=np.int32)), out,
                         ws)
    a.check(out, what="far pages")


def test_attn_own_stream_and_graph_replays(hrs):
    """A captured call replays on changed lengths and inputs; eager calls with
    another workspace run between the replays."""
    import torch
    a = Attn(2, 9, 8, 2, 128, 16, [200, 77], "bf16", "bf16", tree=True)
    R, T, Hq, Hkv, d, S = a.shape
    q, k, v, kc, vc, pages = map(dev, (a.q, a.k, a.v, a.kc, a.vc, a.pages))
    n = dev(np.array(a.lens, dtype=np.int32))
    ws = torch.empty(hrs.attn_verify_span_workspace_bytes(R, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    out = torch.empty(R, T, Hq, d, dtype=torch.bfloat16, device="cuda")
    call = hrs.attn_verify_span_call(q, k, v, kc, vc, pages, n, out, ws, parent=a.parent)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for lens in ([200, 77], [0, 208], [31, 32], [200, 77]):
        a.lens = lens
        n.copy_(dev(np.array(lens, dtype=np.int32)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a.run(hrs)), lens
        a.check(out, what=f"replay {lens}")


# --- kv_cache_append -----------------------------------------------------------

@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")])
@pytest.mark.parametrize("L,R,T,H,d,S,tree,apart", [(1, 1, 1, 1, 16, 16, False, True), (3, 4, 17, 4, 128, 16, True, True),
                                                    (2, 3, 9, 3, 80, 32, False, False), (1, 2, 64, 2, 256, 64, True, False),
                                                    (2, 1, 300, 1, 64, 16, False, True), (1, 300, 2, 1, 64, 16, False, False)])
def test_append(hrs, dtype, cache, L, R, T, H, d, S, tree, apart):
    import torch
    rng = np.random.default_rng(L + R + T + d)
    lens = rng.integers(0, 3 * S, R).astype(np.int32)
    P = int(max(lens) + T + S - 1) // S + 1
    N = R * P + 2
    pages = rng.permutation(N)[:R * P].reshape(R, P).astype(np.int32)
    rows = [cast(rng.standard_normal((L, R, T, H, d)) * 4, dtype) for _ in range(2)]
    if dtype == "bf16":
        rows[0][0, 0, 0, 0, :4] = [0x7FC0, 0x7F80, 0xFF80, 0x4700]       # NaN, inf, -inf, 32768
    mk = lambda: (rng.integers(0, 255, (L, N, H, S, d)).astype(np.uint8) if cache == "f8"
                  else cast(rng.standard_normal((L, N, H, S, d)), cache))
    caches = [mk(), mk()]
    scales = [rng.uniform(0.005, 0.03, (L, H)).astype(np.float32) if cache == "f8" else None for _ in range(2)]
    alen = rng.integers(0, T, R).astype(np.int32)
    alen[0] = T - 1
    path = None
    if tree:
        path = np.full((R, T), -1, dtype=np.int32)
        for r in range(R):
            path[r, :alen[r] + 1] = np.sort(rng.permutation(T)[:alen[r] + 1])
    if R > 2:
        pages[1, int(lens[1]) // S] = -3                                  # a page that is not there
        alen[2] = T                                                       # refused
    n_dev, k_dev, v_dev = dev(lens), dev(caches[0]), dev(caches[1])
    out = torch.full((R,), -9, dtype=torch.int32, device="cuda") if apart else n_dev
    status = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    hrs.kv_cache_append(dev(rows[0]), dev(rows[1]), k_dev, v_dev, dev(pages), n_dev, dev(alen), seq_len_out=out,
                        path=None if path is None else dev(path), k_scale=None if scales[0] is None else dev(scales[0]),
                        v_scale=None if scales[1] is None else dev(scales[1]), status=status)
    ok = [0 <= alen[r] < T for r in range(R)]
    assert out.tolist() == [int(lens[r] + (alen[r] + 1 if ok[r] else 0)) for r in range(R)]
    assert status.tolist() == [sum(not x for x in ok), 7, 7, 7]
    for x, c, s, got in zip(rows, caches, scales, (k_dev, v_dev)):
        for l in range(L):
            for r in range(R):
                if ok[r]:
                    src = oa.quantize_e4m3(widen(x[l, r]), s[l]) if cache == "f8" else x[l, r]
                    oa.append(src, c[l], pages[r], int(lens[r]), None if path is None else path[r], int(alen[r]) + 1)
        g = host(got)
        if cache == "f8":     # any NaN pattern of the same sign bit's byte
            assert np.array_equal(np.where((g & 127) == 127, 127, g), np.where((c & 127) == 127, 127, c))
        else:
            assert np.array_equal(g.view(np.uint32 if cache == "f32" else np.uint16), c.view(np.uint32 if cache == "f32" else np.uint16))


def test_append_refuses_bad_requests_on_the_device(hrs):
    import torch
    L, R, T, H, d, S, P = 1, 6, 4, 1, 16, 16, 2
    k = torch.ones(L, R, T, H, d, device="cuda")
    kc, vc = (torch.zeros(L, R * P, H, S, d, device="cuda") for _ in range(2))
    pages = torch.arange(R * P, dtype=torch.int32, device="cuda").view(R, P)
    n = dev(np.array([28, 29, -1, 0, 0, 2 ** 31 - 1], dtype=np.int32))      # 29 + 4 slots do not fit in 32
    alen = dev(np.array([3, 3, 0, -1, 1, 3], dtype=np.int32))
    path = np.tile(np.arange(T, dtype=np.int32), (R, 1))
    path[4, 1] = T
    out = torch.zeros(R, dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    hrs.kv_cache_append(k, k, kc, vc, pages, n, alen, seq_len_out=out, path=dev(path), status=status)
    assert out.tolist() == [32, 29, -1, 0, 0, 2 ** 31 - 1] and int(status[0]) == 5
    assert int((kc != 0).sum()) == 4 * d and bool((kc[0, 1, 0, 12:] == 1).all())


def test_append_graph_replay_advances_in_place(hrs):
    import torch
    L, R, T, H, d, S, P = 2, 3, 5, 2, 64, 16, 6
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(L, R, T, H, d, generator=g, device="cuda") for _ in range(2))
    kc, vc = (torch.zeros(L, R * P, H, S, d, device="cuda") for _ in range(2))
    pages = torch.randperm(R * P, generator=g, device="cuda").to(torch.int32).view(R, P)
    n = torch.zeros(R, dtype=torch.int32, device="cuda")
    alen = torch.zeros(R, dtype=torch.int32, device="cuda")
    call = hrs.kv_cache_append_call(k, v, kc, vc, pages, n, alen, seq_len_out=n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    want = [[] for _ in range(R)]
    for step in range(4):
        k.normal_(generator=g)
        v.normal_(generator=g)
        alen.copy_(torch.tensor([step, 4, 0], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for r, a in enumerate(alen.tolist()):
            want[r].append(v[:, r, :a + 1].clone())
    for r in range(R):
        rows = torch.cat(want[r], 1)
        assert int(n[r]) == rows.shape[1]
        got = vc[:, pages[r].long()].permute(0, 1, 3, 2, 4).reshape(L, P * S, H, d)
        assert torch.equal(got[:, :rows.shape[1]], rows) and not bool(got[:, rows.shape[1]:].any())


# --- the operators of one attention layer and step together -----------------------

@pytest.mark.parametrize("tree,cache", [(False, "bf16"), (True, "bf16"), (True, "f8")])
def test_steps_of_an_attention_layer_with_sampled_acceptance(hrs, tree, cache):
    """Three verify steps of a two-layer model as they are used: norm and
    rotation, attention over the pages and the draft, acceptance by sampling,
    accepted rows into the pages, lengths advanced on the device. Every step
    is compared with the oracle run on the same history."""
    import torch
    from oracle import sample as osm
    rng = np.random.default_rng(11)
    L, R, T, Hq, Hkv, d, S, P, V = 2, 3, 7, 4, 2, 64, 16, 4, 96
    kc, vc = (torch.zeros(L, R * P, Hkv, S, d, dtype=torch.uint8 if cache == "f8" else torch.bfloat16, device="cuda") for _ in range(2))
    if cache == "f8":
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    sc = [np.full((L, Hkv), 0.02, np.float32) if cache == "f8" else None for _ in range(2)]
    scd = [None if x is None else dev(x) for x in sc]
    pages = rng.permutation(R * P).reshape(R, P).astype(np.int32)
    n = torch.zeros(R, dtype=torch.int32, device="cuda")
    freq = 100.0 ** (-np.arange(16) / 16.0)
    qw, kw = (cast(1 + 0.1 * rng.standard_normal(d), "bf16") for _ in range(2))
    ws = torch.empty(hrs.attn_verify_span_workspace_bytes(R, T, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    sws = torch.empty(hrs.accept_sample_workspace_bytes(R, T, V), dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    for step in range(3):
        par = np.stack([random_tree(rng, T) for _ in range(R)]) if tree else None
        lens = n.tolist()
        x = [cast(rng.standard_normal((L, R, T, h, d)), "bf16") for h in (Hq, Hkv, Hkv)]
        qo = torch.empty(L, R, T, Hq, d, dtype=torch.bfloat16, device="cuda")
        ko = torch.empty(L, R, T, Hkv, d, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(L, R, T, Hq, d, dtype=torch.bfloat16, device="cuda")
        q, k, v = map(dev, x)
        for l in range(L):
            hrs.qk_norm_rope(q[l], k[l], dev(qw), dev(kw), dev(freq), n, qo[l], ko[l], parent=par)
            hrs.attn_verify_span(qo[l], ko[l], v[l], kc[l], vc[l], dev(pages), n, out[l], ws, parent=par,
                                 k_scale=None if scd[0] is None else scd[0][l], v_scale=None if scd[1] is None else scd[1][l])
        logits, tok, u = cast(rng.standard_normal((R, T, V)) * 2, "bf16"), rng.integers(0, 6, (R, T)).astype(np.int32), rng.random((R, T), dtype=np.float32) * np.float32(0.1)
        prob, node, alen, path, bonus = torch.zeros(R, T, device="cuda"), i32(R), i32(R), i32(R, T), i32(R)
        hrs.accept_sample(dev(logits), dev(tok), dev(u), prob, node, alen, path, bonus, sws, parent=par)
        before = [host(c).copy() for c in (kc, vc)]
        hrs.kv_cache_append(ko, v, kc, vc, dev(pages), n, alen, seq_len_out=n, path=path, k_scale=scd[0], v_scale=scd[1])
        kh = host(ko)
        for l in range(L):
            for r in range(R):
                a = Attn(1, T, Hq, Hkv, d, S, [lens[r]], "bf16", cache)
                a.q, a.k, a.v = host(qo)[l, r][None], kh[l, r][None], x[2][l, r][None]
                a.kc, a.vc, a.N, a.pages = before[0][l], before[1][l], R * P, pages[r][None]
                a.ks, a.vs = (None if s is None else s[l] for s in sc)
                a.parent = None if par is None else par[r][None]
                a.check(out[l, r][None], what=f"step {step}")
        for r in range(R):
            ref = osm.accept(logits[r], tok[r], u[r], parent=None if par is None else par[r])
            assert np.array_equal(host(path)[r], ref.path) and int(bonus[r]) == ref.bonus
            assert int(n[r]) == lens[r] + ref.accept_len + 1
            for l in range(L):
                for rows, c, s, b in ((kh, kc, sc[0], before[0]), (x[2], vc, sc[1], before[1])):
                    src = oa.quantize_e4m3(widen(rows[l, r]), s[l]) if cache == "f8" else rows[l, r]
                    oa.append(src, b[l], pages[r], lens[r], ref.path, ref.accept_len + 1)
        for c, b in zip((kc, vc), before):
            assert np.array_equal(host(c), b)

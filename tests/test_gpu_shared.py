"""attn_verify_shared on the GPU against the float64 oracle of attention, fed
every request's slots one by one (prefix below prefix_len, its own pages from
there on).

Tolerances as in test_gpu_attn.py: a bf16 span rounds each weight (2^-8 for a
bf16 cache, which covers the 16 bits that short batches keep; weights beside
e4m3 values are good to 2^-11), all relative to sum w |v|.
"""
import numpy as np
import pytest

from oracle import attn as oa
from oracle.common import widen
from tests.gpu_util import say
from tests.test_gpu_attn import OUT, U, cast, dev, host, hrs, random_tree  # noqa: F401

pytestmark = pytest.mark.gpu


class Shared:
    def __init__(self, R, T, Hq, Hkv, d, S, prefix, own, dtype="bf16", cache="bf16", tree=False, window=0, seed=0, gain=1.0,
                 scale=None):
        rng = np.random.default_rng(seed + 17 * R + T + d)
        self.shape = (R, T, Hq, Hkv, d, S)
        self.prefix, self.lens = prefix, [x for x in own]
        self.dtype, self.cache, self.window, self.scale = dtype, cache, window, scale
        PP = -(-prefix // S) + 1
        P = max(1, -(-max(self.lens) // S))
        self.N = R * P + PP + 3
        order = rng.permutation(self.N).astype(np.int32)
        self.ptable, self.pages = order[:PP], order[PP:PP + R * P].reshape(R, P).copy()
        f = lambda *s: rng.standard_normal(s, dtype=np.float32) * np.float32(gain)
        self.q, self.k, self.v = (cast(f(R, T, h, d), dtype) for h in (Hq, Hkv, Hkv))
        self.ks = self.vs = None
        if cache == "f8":
            self.ks, self.vs = (rng.uniform(0.01, 0.03, Hkv).astype(np.float32) for _ in range(2))
            self.kc, self.vc = (oa.quantize_e4m3(f(self.N, Hkv, S, d) * 50, None) for _ in range(2))
        else:
            self.kc, self.vc = (cast(f(self.N, Hkv, S, d), cache) for _ in range(2))
        self.parent = np.stack([random_tree(rng, T) for _ in range(R)]) if tree else None

    def tensors(self, hrs, out=None, ws=None):
        import torch
        R, T, Hq, Hkv, d, S = self.shape
        n = hrs.attn_verify_shared_workspace_bytes(R, T, Hq, Hkv, d)
        if ws is None:
            ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")     # contents must not matter: NaNs
        q = dev(self.q)
        if out is None:
            out = torch.full((R, T, Hq, d), 77.0, dtype=q.dtype, device="cuda")
        opt = lambda x: None if x is None else dev(x)
        return dict(q=q, k=dev(self.k), v=dev(self.v), k_cache=dev(self.kc), v_cache=dev(self.vc),
                    prefix_table=dev(self.ptable), prefix_len=dev(np.array([self.prefix], np.int32)),
                    page_table=dev(self.pages), seq_len=dev(np.array(self.lens, np.int32)), out=out, workspace=ws,
                    parent=self.parent, scale=self.scale, window=self.window, k_scale=opt(self.ks), v_scale=opt(self.vs))

    def run(self, hrs, out=None, ws=None, status=None, stream=None):
        a = self.tensors(hrs, out, ws)
        hrs.attn_verify_shared(**a, status=status, stream=stream)
        return a["out"]

    def slots(self, r):
        """Request r's keys and values slot by slot, and which are there."""
        S, n = self.shape[5], self.lens[r]
        page = [int(self.ptable[j // S] if j < self.prefix else self.pages[r, j // S]) for j in range(n)]
        at = np.array([p if 0 <= p < self.N else 0 for p in page], dtype=int)
        row = np.arange(n) % S
        there = np.array([j if 0 <= p < self.N else -1 for j, p in enumerate(page)] + [-1], dtype=np.int64)
        return self.kc[at, :, row][:, :, None], self.vc[at, :, row][:, :, None], there

    def reference(self, r):
        kc, vc, there = self.slots(r)
        return oa.attn_span(self.q[r], self.k[r], self.v[r], kc, vc, there, self.lens[r],
                            None if self.parent is None else self.parent[r], self.scale, self.window, self.ks, self.vs,
                            want_bound=True)

    def tolerance(self, ref, absv, reach, n):
        d = self.shape[4]
        rel = 2 * (2 * (d + 4) * U) * reach + (2 * n + 16) * U + (2.0 ** -8 if self.dtype == "bf16" else 0)
        return rel[..., None] * absv + OUT[self.dtype] * (np.abs(ref) + rel[..., None] * absv)

    def check(self, got, requests=None, what=""):
        got = widen(host(got))
        worst = 0.0
        for r in range(self.shape[0]) if requests is None else requests:
            ref, *bound = self.reference(r)
            tol = self.tolerance(ref, *bound)
            err = np.abs(got[r] - ref)
            assert not np.isnan(got[r]).any(), (what, r, "NaN")
            assert np.all(err <= tol), (what, r, float(np.max(err / (tol + 1e-300))))
            worst = max(worst, float(np.max(err / (tol + 1e-300))))
        say(f"  shared {what} {self.shape} {self.dtype}/{self.cache}: largest error {worst:.2f} of its bound")


GRID = [
    # R, T, Hq, Hkv, d, S, prefix, lengths, dtype, cache, tree, window
    (1, 1, 1, 1, 64, 16, 0, [0], "f32", "f32", False, 0),
    (1, 1, 1, 1, 64, 16, 1, [1], "bf16", "bf16", False, 0),
    (2, 1, 4, 2, 128, 16, 127, [127, 300], "bf16", "bf16", False, 0),
    (2, 1, 4, 2, 128, 16, 128, [128, 129], "bf16", "bf16", False, 0),
    (3, 1, 24, 4, 256, 64, 1000, [1003, 1400, 1000], "bf16", "bf16", False, 0),
    (16, 1, 12, 2, 256, 64, 515, [520 + 7 * i for i in range(16)], "bf16", "bf16", False, 0),
    (5, 17, 12, 2, 256, 64, 700, [700, 705, 900, 1100, 764], "bf16", "bf16", False, 0),
    (3, 17, 24, 4, 256, 16, 517, [600, 517, 530], "bf16", "f8", False, 0),
    (4, 9, 4, 4, 64, 32, 300, [301, 400, 300, 555], "f32", "f32", False, 0),
    (6, 23, 8, 2, 128, 16, 391, [391, 400, 410, 600, 900, 393], "bf16", "bf16", True, 0),
    (6, 23, 8, 2, 128, 16, 391, [391, 400, 410, 600, 900, 393], "bf16", "f8", True, 0),
    (3, 64, 8, 1, 128, 128, 1030, [1030, 1500, 1033], "bf16", "bf16", True, 0),
    (3, 30, 8, 1, 64, 128, 1030, [1030, 1500, 1033], "bf16", "f8", False, 0),
    (2, 33, 6, 2, 256, 32, 650, [700, 651], "f32", "f32", True, 0),
    (4, 5, 6, 2, 64, 16, 500, [20, 500, 700, 260], "bf16", "bf16", False, 0),          # shorter than the prefix
    (3, 4, 6, 2, 64, 16, 500, [0, 600, 700], "bf16", "bf16", False, 0),                # and empty
    (4, 17, 4, 2, 128, 16, 800, [900, 850, 820, 1000], "bf16", "bf16", False, 500),    # windows that start in the prefix
    (4, 17, 16, 1, 128, 16, 800, [900, 850, 820, 1000], "bf16", "f8", True, 480),
    (2, 7, 4, 2, 64, 16, 800, [1200, 900], "f32", "f32", False, 150),                  # one behind it, one in it
    (2, 3, 4, 2, 64, 16, 300, [900, 800], "bf16", "bf16", False, 1),
    (70, 2, 4, 1, 128, 16, 260, [260 + i for i in range(70)], "bf16", "bf16", False, 0),
    (70, 2, 4, 1, 64, 16, 260, [260 + i for i in range(70)], "f32", "f32", False, 0),
    (2, 2, 64, 1, 64, 1024, 1500, [1500, 1501], "bf16", "f8", False, 0),
    (9, 19, 2, 2, 64, 16, 4000, [4100 - i for i in range(9)], "bf16", "bf16", False, 0),
]


@pytest.mark.parametrize("case", GRID, ids=lambda c: f"R{c[0]}T{c[1]}h{c[2]}-{c[3]}d{c[4]}p{c[5]}n{c[6]}{c[8]}{c[9]}{'t' if c[10] else ''}w{c[11]}")
def test_shared_vs_oracle(hrs, case):
    R, T, Hq, Hkv, d, S, prefix, lens, dt, ct, tree, window = case
    a = Shared(R, T, Hq, Hkv, d, S, prefix, lens, dt, ct, tree, window)
    a.check(a.run(hrs), what="grid")


KINDS = [("bf16", "bf16"), ("bf16", "f8"), ("f32", "f32")]


@pytest.mark.parametrize("rows", [3, 20, 50, 90, 120, 130, 300, 500])      # of a key head, over all requests
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_shared_at_every_block_shape(hrs, dtype, cache, d, rows):
    """Row counts of every class, absent pages in the prefix and behind it, values that are not finite where they count
    and where they do not."""
    T = 5 if rows >= 20 else 1
    R = -(-rows // (2 * T))
    lens = [660 + (37 * r) % 200 for r in range(R)]
    a = Shared(R, T, 4, 2, d, 16, 650, lens, dtype, cache, tree=T > 1, seed=rows)
    a.ptable[[3, 17]] = [-1, a.N]
    a.pages[R // 2, 42] = -7
    pick = sorted({0, R // 2, R - 1})
    clean = a.run(hrs)
    a.check(clean, pick, what=f"{rows} rows")
    bad = {"f32": np.float32(np.nan), "bf16": np.uint16(0x7FC0), "f8": np.uint8(0x7F)}
    pos = {"f32": np.float32(np.inf), "bf16": np.uint16(0x7F80), "f8": np.uint8(0x7F)}
    used = np.zeros((a.N, 16), dtype=bool)
    for r in range(R):
        for j in range(lens[r]):
            p = a.ptable[j // 16] if j < 650 else a.pages[r, j // 16]
            if 0 <= p < a.N:
                used[p, j % 16] = True
    import torch
    for c in (a.kc, a.vc):
        c.transpose(0, 2, 1, 3)[~used] = bad[cache]
    assert torch.equal(a.run(hrs), clean)
    a.vc[a.ptable[200 // 16], 1, 200 % 16, 5] = pos[cache]       # counts for all
    a.vc[a.ptable[649 // 16], 0, 649 % 16, 7] = bad[cache]
    a.vc[a.pages[0, 655 // 16], 1, 655 % 16, 9] = pos[cache]     # for the first request
    got = widen(host(a.run(hrs)))
    for r in pick:
        with np.errstate(invalid="ignore"):
            ref, *bound = a.reference(r)
            tol = a.tolerance(ref, *bound)
            assert np.array_equal(np.isnan(got[r]), np.isnan(ref)), r
            assert np.array_equal(got[r][np.isinf(ref)], ref[np.isinf(ref)]), r
            fin = np.isfinite(ref)
            assert np.all(np.abs(got[r] - ref)[fin] <= tol[fin]), r


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("gain", [1e-3, 8.0])
def test_shared_flat_and_peaked_scores(hrs, dtype, cache, gain):
    a = Shared(9, 9, 8, 2, 128, 32, 900, [901 + 3 * r for r in range(9)], dtype, cache, gain=gain if cache != "f8" else 1.0,
               scale=None if cache != "f8" else gain)
    a.check(a.run(hrs), [0, 8], what=f"gain {gain}")


@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_shared_scales(hrs, dtype, cache, scale):
    a = Shared(9, 9, 8, 2, 64, 32, 600, [601 + 3 * r for r in range(9)], dtype, cache, scale=scale)
    a.check(a.run(hrs), [0, 8], what=f"scale {scale}")


def test_shared_many_requests_over_several_launches(hrs):
    rng = np.random.default_rng(3)
    a = Shared(300, 3, 2, 1, 64, 16, 200, [int(x) for x in rng.integers(150, 300, 300)])
    a.check(a.run(hrs), range(0, 300, 23), what="300 requests")
    a = Shared(130, 25, 2, 1, 64, 16, 256, [int(x) for x in rng.integers(256, 300, 130)], tree=True)
    a.check(a.run(hrs), range(0, 130, 17), what="130 trees")


def test_shared_strided_views_of_one_projection(hrs):
    import torch
    a = Shared(7, 5, 12, 2, 64, 16, 300, [340 + r for r in range(7)])
    t = a.tensors(hrs)
    full = torch.cat([t["q"].flatten(2), t["k"].flatten(2), t["v"].flatten(2)], -1)
    cut = lambda lo, h: full[..., lo * 64:(lo + h) * 64].unflatten(-1, (h, 64))
    t.update(q=cut(0, 12), k=cut(12, 2), v=cut(14, 2))
    hrs.attn_verify_shared(**t)
    assert torch.equal(t["out"], a.run(hrs))


def test_shared_bad_lengths_are_left_alone_and_counted(hrs):
    import torch
    a = Shared(5, 30, 4, 2, 64, 16, 200, [230, 240, 250, 256, 210])
    status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    a.lens = [230, -1, 257, 256, -2 ** 31]
    got = a.run(hrs, status=status)
    assert status.tolist() == [3, 9, 9, 9]
    assert bool((got[[1, 2, 4]] == 77).all())
    a.check(got, [0, 3], what="beside bad lengths")
    for p in (-1, len(a.ptable) * 16 + 1, 2 ** 31 - 1):
        a.prefix, a.lens = p, [230, 240, 250, 256, 210]
        assert bool((a.run(hrs, status=status) == 77).all()) and status.tolist() == [5, 9, 9, 9]


def test_shared_repeat_is_bit_identical_and_guarded(hrs):
    import torch
    for case in (Shared(9, 17, 8, 2, 128, 16, 1500, [1501 + 9 * r for r in range(9)], tree=True),
                 Shared(3, 2, 8, 2, 128, 16, 1500, [1501 + 9 * r for r in range(3)], cache="f8")):
        first = case.run(hrs)
        for _ in range(3):
            assert torch.equal(case.run(hrs), first)
        buf = torch.full((first.numel() + 256,), 3.0, dtype=torch.bfloat16, device="cuda")
        n = hrs.attn_verify_shared_workspace_bytes(*case.shape[:5])
        ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        case.run(hrs, out=buf[128:-128].view(first.shape), ws=ws[256:-256])
        assert torch.equal(buf[128:-128].view(first.shape), first)
        assert bool((buf[:128] == 3).all()) and bool((buf[-128:] == 3).all())
        assert bool((ws[:256] == 0xA5).all()) and bool((ws[-256:] == 0xA5).all())


def test_shared_as_attn_verify_span(hrs):
    """The same slots through one table: the two agree to rounding."""
    import torch
    a = Shared(6, 9, 8, 2, 128, 16, 640, [700 + 11 * r for r in range(6)], "f32", "f32", tree=True)
    a.pages[:, :40] = a.ptable[:40]
    t = a.tensors(hrs)
    hrs.attn_verify_shared(**t)
    span = {k: v for k, v in t.items() if not k.startswith("prefix")}
    span["out"] = torch.empty_like(t["out"])
    span["workspace"] = torch.empty(hrs.attn_verify_span_workspace_bytes(*a.shape[:5]), dtype=torch.uint8, device="cuda")
    hrs.attn_verify_span(**span)
    assert torch.allclose(span["out"], t["out"], rtol=0, atol=1e-4 * float(t["out"].abs().max()))


def test_shared_two_streams_at_once(hrs):
    import torch
    cases = [Shared(9, 17, 8, 2, 128, 16, 3000, [3001 + r for r in range(9)], seed=1),
             Shared(2, 5, 4, 2, 256, 32, 5000, [5100, 5200], cache="f8", seed=2)]
    want = [c.run(hrs) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w) for w in want]
    calls = [hrs.attn_verify_shared_call(**c.tensors(hrs, out=o)) for c, o in zip(cases, outs)]
    torch.cuda.synchronize()
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for call, st in zip(calls, streams):
            call(st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_shared_graph_replays_on_other_lengths(hrs):
    """A captured call on changed lengths and prefixes, eager calls with another workspace in between."""
    import torch
    a = Shared(9, 9, 8, 2, 128, 16, 500, [560 + r for r in range(9)], tree=True)
    t = a.tensors(hrs)
    call = hrs.attn_verify_shared_call(**t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for prefix, lens in ((500, [560 + r for r in range(9)]), (0, [100] * 9), (130, [400, 3] + [200] * 7), (512, [512] * 9)):
        a.prefix, a.lens = prefix, lens
        t["prefix_len"].copy_(dev(np.array([prefix], np.int32)))
        t["seq_len"].copy_(dev(np.array(lens, np.int32)))
        t["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t["out"], a.run(hrs)), lens
        a.check(t["out"], [0, 1, 8], what=f"replay {prefix}")


def test_shared_pages_behind_2_31_elements(hrs):
    import torch
    N, H, S, d = 70000, 4, 64, 128          # 2.3e9 elements a side, 4.6 GB
    a = Shared(40, 2, 8, 4, d, S, 256, [260 + r % 60 for r in range(40)])
    big = [torch.zeros(N, H, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far = (np.arange(a.N) * 7 + 69999 - 7 * (a.N - 1)).astype(np.int32)
    for b, c in zip(big, (a.kc, a.vc)):
        b[torch.from_numpy(far).long().cuda()] = dev(c)
    t = a.tensors(hrs)
    t.update(k_cache=big[0], v_cache=big[1], prefix_table=dev(far[a.ptable]), page_table=dev(far[a.pages]))
    hrs.attn_verify_shared(**t)
    a.check(t["out"], [0, 39], what="far pages")


# Batches with more than 256 rows of a key head, whose weights over the prefix
# are rounded once, and the rounded ones summed: out = sum w (1 + e) v /
# sum w (1 + e) is off by sum w e (v - out) / sum w, |e| <= 2^-8, which is at
# most 2^-8 (sum w |v| + |out|).
class Large(Shared):
    def tolerance(self, ref, absv, reach, n):
        return super().tolerance(ref, absv, reach, n) + 2.0 ** -8 * np.abs(ref)


WIDE = [("bf16", "bf16"), ("bf16", "f8")]


@pytest.mark.parametrize("dtype,cache", WIDE)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("gain,scale", [(1e-3, None), (8.0, None), (700.0, None), (1.0, -0.3), (1.0, 0.0)])
def test_shared_large_scores(hrs, dtype, cache, d, gain, scale):
    a = Large(9, 9, 8, 2, d, 16, 900, [901 + 3 * r for r in range(9)], dtype, cache, gain=gain if cache != "f8" else 1.0,
              scale=scale if scale is not None or cache != "f8" else min(gain, 20.0))
    a.check(a.run(hrs), [0, 8], what=f"large, gain {gain} scale {scale}")


@pytest.mark.parametrize("dtype,cache", WIDE)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [257, 577])
def test_shared_large_rows(hrs, dtype, cache, d, rows):
    """Blocks that end inside a tile of rows and waves without any."""
    a = Large(rows, 1, 2, 2, d, 32, 300, [300 + r % 30 for r in range(rows)], dtype, cache)
    a.check(a.run(hrs), [0, 192, rows - 1], what=f"large, {rows} rows")


@pytest.mark.parametrize("dtype,cache", WIDE)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_shared_large_prefixes(hrs, dtype, cache, d):
    """A captured call on prefixes of every number of tiles a run may have, with eager calls in between."""
    import torch
    a = Large(40, 2, 16, 2, d, 16, 2000, [2000 + r for r in range(40)], dtype, cache)
    t = a.tensors(hrs)
    call = hrs.attn_verify_shared_call(**t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for prefix in (0, 1, 127, 128, 129, 384, 640, 1999, 2000):
        a.prefix, a.lens = prefix, [prefix + r for r in range(40)]
        a.ptable[5] = -1 if prefix == 1999 else abs(int(a.ptable[5]))
        t["prefix_table"].copy_(dev(a.ptable))
        t["prefix_len"].copy_(dev(np.array([prefix], np.int32)))
        t["seq_len"].copy_(dev(np.array(a.lens, np.int32)))
        t["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t["out"], a.run(hrs)), prefix
        a.check(t["out"], [39], what=f"large, prefix {prefix}")


def test_shared_large_two_streams_at_once(hrs):
    import torch
    cases = [Large(20, 17, 8, 2, 128, 16, 3000, [3001 + r for r in range(20)], cache=c, seed=1) for c in ("bf16", "f8")]
    cases.append(Large(20, 17, 12, 2, 256, 32, 2000, [2100 + r for r in range(20)], seed=2))
    want = [c.run(hrs) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w) for w in want]
    calls = [hrs.attn_verify_shared_call(**c.tensors(hrs, out=o)) for c, o in zip(cases, outs)]
    torch.cuda.synchronize()
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for call, st in zip(calls, streams):
            call(st)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("dtype,cache", WIDE)
@pytest.mark.parametrize("d,S,tree,window", [(64, 16, True, 700), (128, 64, False, 500), (256, 128, False, 333)])
def test_shared_large_windows(hrs, dtype, cache, d, S, tree, window):
    """Windows that start in the prefix: the shared slots begin behind its start."""
    a = Large(20, 17, 4, 2, d, S, 1000, [1000 + 9 * r for r in range(20)], dtype, cache, tree=tree, window=window)
    a.ptable[len(a.ptable) // 2] = -1
    a.check(a.run(hrs), [0, 10, 19], what=f"large, window {window}")

"""Measured cases of the attention-layer and sampling operators of the verify step.

Four operators, used one after another when a draft block is verified: norm and
rotation of queries and keys (qk_norm_rope), attention of a draft chain or tree
over a paged cache (attn_verify_span), the accepted rows' way into the cache
(kv_cache_append) and acceptance by sampling (accept_sample). ``run`` computes
the plain form with elementary torch operations, or calls the library where
``own`` is true; ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f8": F8}
SIZE = {"bf16": 2, "f32": 4, "f8": 1}


# --- cases ------------------------------------------------------------------

def listed():
    return [
        # One decoded token of one request far into its context: launch latency.
        dict(name="rope-decode", op="rope", R=1, T=1, Hq=24, Hkv=4, D=256, rot=64, dtype="bf16", ctx=98304,
             tree=False, interleaved=False, packed=True),
        # A prefill chunk: every byte read and written once.
        dict(name="rope-prefill-4096", op="rope", R=1, T=4096, Hq=24, Hkv=4, D=256, rot=64, dtype="bf16", ctx=26758,
             tree=False, interleaved=False, packed=True),
        # Plain decoding of one request with a short context.
        dict(name="attn-decode-1000", op="attn", R=1, T=1, Hq=24, Hkv=4, D=256, dtype="bf16", cache="bf16", ctx=1000,
             page=64, tree=False, window=0),
        # A 16-draft chain of one request behind a long prompt.
        dict(name="attn-chain-26758", op="attn", R=1, T=17, Hq=24, Hkv=4, D=256, dtype="bf16", cache="bf16",
             ctx=26758, page=64, tree=False, window=0),
        # Sixteen requests with draft trees and ragged contexts, small pages.
        dict(name="attn-tree-r16", op="attn", R=16, T=23, Hq=32, Hkv=8, D=128, dtype="bf16", cache="bf16", ctx=8191,
             page=16, tree=True, window=0),
        # One very long context with an 8-bit cache.
        dict(name="attn-long-f8", op="attn", R=1, T=17, Hq=32, Hkv=8, D=128, dtype="bf16", cache="f8", ctx=262144,
             page=64, tree=False, window=0),
        # The small float32 configuration, draft model's window.
        dict(name="attn-f32-window", op="attn", R=3, T=9, Hq=4, Hkv=4, D=64, dtype="f32", cache="f32", ctx=5000,
             page=32, tree=False, window=2048),
        # Acceptance by sampling, one request, 16 drafts with their probabilities.
        dict(name="sample-chain-1", op="sample", R=1, T=17, V=151936, dtype="bf16", tree=False, drafts=True),
        # Sixteen concurrent requests.
        dict(name="sample-chain-r16", op="sample", R=16, T=17, V=151936, dtype="bf16", tree=False, drafts=True),
        # Draft trees of top tokens (no draft probabilities), float32 logits.
        dict(name="sample-tree-r4", op="sample", R=4, T=23, V=151936, dtype="f32", tree=True, drafts=False),
        # Accepted rows of a 16-layer stack into the pages: one request's tree.
        dict(name="append-tree-1", op="append", L=16, R=1, T=23, Hkv=4, D=256, dtype="bf16", cache="bf16", page=64,
             ctx=100, tree=True),
        # Sixteen chains into an 8-bit cache.
        dict(name="append-chain-r16-f8", op="append", L=16, R=16, T=17, Hkv=8, D=128, dtype="bf16", cache="f8",
             page=64, ctx=100, tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "attn", "sample", "sample", "append"])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    cache = rng.choice(["bf16", "f8"]) if dtype == "bf16" else "f32"
    tree = rng.random() < 0.5
    if op == "rope":
        T = rng.randint(2, 64) if tree else _log(rng, 1, 4096)
        R = _log(rng, 1, max(1, 8192 // T))
        return dict(op=op, R=min(R, 64), T=T, Hq=Hkv * rng.randint(1, 6), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2, D // 4]), dtype=dtype, ctx=_log(rng, 1, 262144), tree=tree,
                    interleaved=rng.random() < 0.3, packed=rng.random() < 0.5)
    if op == "attn":
        T = rng.randint(2, 64) if tree else rng.choice([1, rng.randint(2, 17), rng.randint(18, 64)])
        R = rng.choice([1, 1, rng.randint(2, 16)])
        G = rng.randint(1, 8)
        # at most the largest listed case's products and bytes
        most = min(262144, int(4.5e8 / (2 * Hkv * D * SIZE[cache] * R)), int(7e7 / (T * G * Hkv * R * D / 128)))
        if dtype == "f32":
            most //= 4
        return dict(op=op, R=R, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, cache=cache, ctx=_log(rng, 1, max(2, most)),
                    page=rng.choice([16, 32, 64, 128]), tree=tree,
                    window=rng.choice([0, 0, _log(rng, 1, 4096)]))
    if op == "sample":
        T = rng.choice([1, rng.randint(2, 17), rng.randint(18, 64)])
        return dict(op=op, R=rng.randint(1, max(1, min(16, 272 // T))), T=T, V=8 * _log(rng, 16, 18992), dtype=dtype,
                    tree=tree and T > 1, drafts=not tree and rng.random() < 0.7)
    T = rng.randint(2, 64) if tree else _log(rng, 1, 64)
    return dict(op=op, L=rng.randint(1, 16), R=rng.randint(1, 16), T=T, Hkv=Hkv, D=D, dtype=dtype, cache=cache,
                page=rng.choice([16, 32, 64, 128]), ctx=_log(rng, 1, 500), tree=tree)


# --- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lengths(case):
    """Ragged context lengths, fixed by the case: the longest first, the shortest about half of it."""
    return [case["ctx"] - (r * 7919) % (case["ctx"] // 2 + 1) for r in range(case["R"])]


def _parents(case, seed):
    """Draft trees in topological order: depth at most 8, at most 3 children."""
    R, T = case["R"], case["T"]
    if not case["tree"]:
        return [[t - 1 for t in range(T)] for _ in range(R)]
    rnd = torch.Generator().manual_seed(int(seed) * 3 + 1)
    rows = []
    for _ in range(R):
        par, depth, kids = [-1], [0], [0]
        for t in range(1, T):
            free = [i for i in range(t) if depth[i] < 8 and kids[i] < 3]
            p = free[int(torch.randint(len(free), (1,), generator=rnd))]
            par.append(p)
            depth.append(depth[p] + 1)
            kids.append(0)
            kids[p] += 1
        rows.append(par)
    return rows


def _depths(par):
    out = []
    for p in par:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def _fill(shape, g, dtype, gain=1.0):
    """Normal values in a type, made in slices so that a large buffer needs little more than itself."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(torch.uint8).reshape(-1) if dtype == F8 else out.reshape(-1)
    n, step = flat.numel(), 1 << 26
    for i in range(0, n, step):
        x = torch.randn(min(step, n - i), generator=g, device="cuda") * gain
        x = x.to(dtype)
        flat[i:i + step] = x.view(torch.uint8) if dtype == F8 else x
    return out


def _pages(case, g, tokens):
    """Shuffled page table rows that hold `tokens` slots each."""
    per = (tokens + case["page"] - 1) // case["page"]
    n = case["R"] * per
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    return order.reshape(case["R"], per).contiguous(), n


def _inputs(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    R, T = case["R"], case["T"]
    dt = DTYPES[case["dtype"]]
    s["parent"] = _parents(case, seed)
    s["depth"] = torch.tensor([_depths(p) for p in s["parent"]], device="cuda")
    if op == "rope":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        if case["packed"]:      # q | k | v as one projection wrote them
            qkv = _fill((R, T, (Hq + 2 * Hkv) * D), g, dt, 2.0)
            s["q"] = qkv[..., :Hq * D].unflatten(-1, (Hq, D))
            s["k"] = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        else:
            s["q"], s["k"] = _fill((R, T, Hq, D), g, dt, 2.0), _fill((R, T, Hkv, D), g, dt, 2.0)
        s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["freq"] = 10000000.0 ** (-2.0 * i / case["rot"])
        s["seq_len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        s["q_out"] = torch.empty(R, T, Hq, D, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(R, T, Hkv, D, dtype=dt, device="cuda")
    elif op == "attn":
        Hq, Hkv, D, S = case["Hq"], case["Hkv"], case["D"], case["page"]
        s["q"], s["k"] = _fill((R, T, Hq, D), g, dt), _fill((R, T, Hkv, D), g, dt)
        s["v"] = _fill((R, T, Hkv, D), g, dt)
        s["table"], n = _pages(case, g, case["ctx"])
        ct = DTYPES[case["cache"]]
        gain = 64.0 if ct == F8 else 1.0
        s["kc"], s["vc"] = _fill((n, Hkv, S, D), g, ct, gain), _fill((n, Hkv, S, D), g, ct, gain)
        s["ks"] = s["vs"] = None
        if ct == F8:
            s["ks"] = (1 + 0.1 * torch.rand(Hkv, generator=g, device="cuda")) / 64
            s["vs"] = (1 + 0.1 * torch.rand(Hkv, generator=g, device="cuda")) / 64
        s["seq_len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(R, T, Hq, D, dtype=dt, device="cuda")
        # root path and window of every span position
        anc = [[[False] * T for _ in range(T)] for _ in range(R)]
        for r in range(R):
            dep = _depths(s["parent"][r])
            for t in range(T):
                a = t
                while a >= 0 and (case["window"] == 0 or dep[t] - dep[a] < case["window"]):
                    anc[r][t][a] = True
                    a = s["parent"][r][a]
        s["anc"] = torch.tensor(anc, device="cuda")
    elif op == "sample":
        V = case["V"]
        z = torch.randn(R, T, V, generator=g, device="cuda") * 2.5
        s["logits"] = z.to(dt)
        s["tau"] = (0.7 + 0.6 * torch.rand(R, generator=g, device="cuda")).float()
        noise = -torch.log(-torch.log(torch.rand(R, T, V, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
        s["dq"] = None
        tok = torch.zeros(R, T, dtype=torch.int64, device="cuda")
        if case["drafts"]:
            # the draft's distribution is near the target's, and its tokens are drawn from it
            y = z / s["tau"].view(-1, 1, 1) + 0.5 * torch.randn(R, T, V, generator=g, device="cuda")
            s["dq"] = torch.softmax(y, -1)
            pick = (y + noise).argmax(-1)
            tok[:, 1:] = pick[:, :-1]
        else:
            top = (z / s["tau"].view(-1, 1, 1) + 0.3 * noise).topk(3, -1).indices   # siblings: three distinct likely tokens
            seen = [[0] * T for _ in range(R)]
            pos, nth = [], []
            for r in range(R):
                for t in range(1, T):
                    p = s["parent"][r][t]
                    pos.append((r, t, p))
                    nth.append(seen[r][p])
                    seen[r][p] += 1
            if pos:
                ix = torch.tensor(pos, device="cuda")
                tok[ix[:, 0], ix[:, 1]] = top[ix[:, 0], ix[:, 2], torch.tensor(nth, device="cuda")]
        s["tokens"] = tok.to(torch.int32)
        s["u"] = torch.rand(R, T, generator=g, device="cuda")
        e = lambda *shape, d=torch.int32: torch.zeros(shape, dtype=d, device="cuda")
        s["token_prob"], s["node"], s["len"], s["path"], s["bonus"] = e(R, T, d=torch.float32), e(R), e(R), e(R, T), e(R)
    else:
        L, Hkv, D = case["L"], case["Hkv"], case["D"]
        s["k"], s["v"] = _fill((L, R, T, Hkv, D), g, dt), _fill((L, R, T, Hkv, D), g, dt)
        s["table"], n = _pages(case, g, case["ctx"] + T)
        ct = DTYPES[case["cache"]]
        s["kc"], s["vc"] = (torch.zeros(L, n, Hkv, case["page"], D, dtype=torch.uint8 if ct == F8 else ct,
                                        device="cuda") for _ in range(2))
        if ct == F8:
            s["kc"], s["vc"] = s["kc"].view(F8), s["vc"].view(F8)
        s["ks"] = s["vs"] = None
        if ct == F8:
            s["ks"] = (1 + 0.1 * torch.rand(L, Hkv, generator=g, device="cuda")) / 64
            s["vs"] = (1 + 0.1 * torch.rand(L, Hkv, generator=g, device="cuda")) / 64
        s["seq_len"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        path = torch.full((R, T), -1, dtype=torch.int32)
        alen = torch.zeros(R, dtype=torch.int32)
        rnd = torch.Generator().manual_seed(int(seed) * 5 + 2)
        for r in range(R):
            par = s["parent"][r]
            a = int(torch.randint(T, (1,), generator=rnd))
            if not case["tree"]:
                a = max(a, T // 2)
            root = []
            while a >= 0:
                root.append(a)
                a = par[a]
            root.reverse()
            path[r, :len(root)] = torch.tensor(root, dtype=torch.int32)
            alen[r] = len(root) - 1
        s["path"], s["alen"] = path.cuda(), alen.cuda()
        s["new_len"] = torch.zeros(R, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import numpy as np

        import hybrid_recurrent_state_amd as hrs
        par = np.asarray(s["parent"], dtype=np.int32) if case["tree"] else None
        op = case["op"]
        if op == "rope":
            s["call"] = hrs.qk_norm_rope_call(s["q"], s["k"], s["qw"], s["kw"], s["freq"], s["seq_len"], s["q_out"],
                                              s["k_out"], parent=par, eps=1e-6, interleaved=case["interleaved"])
        elif op == "attn":
            n = hrs.attn_verify_span_workspace_bytes(case["R"], case["T"], case["Hq"], case["Hkv"], case["D"])
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            s["call"] = hrs.attn_verify_span_call(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["seq_len"],
                                                  s["out"], ws, parent=par, window=case["window"], k_scale=s["ks"],
                                                  v_scale=s["vs"])
        elif op == "sample":
            n = hrs.accept_sample_workspace_bytes(case["R"], case["T"], case["V"])
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            s["call"] = hrs.accept_sample_call(s["logits"], s["tokens"], s["u"], s["token_prob"], s["node"], s["len"],
                                               s["path"], s["bonus"], ws, draft_probs=s["dq"], temperature=s["tau"],
                                               parent=par)
        else:
            s["call"] = hrs.kv_cache_append_call(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["seq_len"], s["alen"],
                                                 seq_len_out=s["new_len"], path=s["path"] if case["tree"] else None,
                                                 k_scale=s["ks"], v_scale=s["vs"])
    return s


# --- one pass ---------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        state["call"]()
    else:
        _PLAIN[case["op"]](state)
    return _outputs(state)


def _outputs(s):
    op = s["case"]["op"]
    if op == "rope":
        return s["q_out"], s["k_out"]
    if op == "attn":
        return s["out"]
    if op == "sample":
        return s["token_prob"], s["node"], s["len"], s["path"], s["bonus"]
    return s["kc"], s["vc"], s["new_len"]


def _plain_rope(s):
    case = s["case"]
    rot, D = case["rot"], case["D"]
    pos = s["seq_len"].double().view(-1, 1) + s["depth"]
    ang = pos[..., None, None] * s["freq"]                       # 64 bits: far positions
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    for x, w, out in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        z = y.clone()
        if case["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z[..., 0:rot:2], z[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z[..., :rot // 2], z[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
        out.copy_(z)


def _context(s, cache, scale):
    """The pages of every request in a row, in 32 bits: [R, Hkv, slots, D]."""
    x = cache.view(torch.uint8)[s["table"].long()].view(F8) if cache.dtype == F8 else cache[s["table"].long()]
    R, P, H, S, D = x.shape
    x = x.permute(0, 2, 1, 3, 4).reshape(R, H, P * S, D).float()
    return x if scale is None else x * scale.view(1, H, 1, 1)


def _plain_attn(s):
    case = s["case"]
    R, T, Hq, Hkv, D = case["R"], case["T"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    k = torch.cat([_context(s, s["kc"], s["ks"]), s["k"].float().transpose(1, 2)], 2)
    n = k.shape[2]
    j = torch.arange(n - T, device="cuda")
    length = s["seq_len"].view(R, 1, 1)
    seen = (j < length).expand(R, T, n - T)
    if case["window"]:
        seen = seen & (j > (length + s["depth"].view(R, T, 1) - case["window"]))
    mask = torch.cat([seen, s["anc"]], 2)                        # [R, T, slots]
    q = s["q"].float().view(R, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * T, D)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()) / math.sqrt(D)
    del k
    score = score.view(R, Hkv, G, T, n).masked_fill_(~mask[:, None, None], -math.inf)
    score = score - score.amax(-1, keepdim=True)
    p = torch.exp_(score)
    p = (p / p.sum(-1, keepdim=True)).view(R, Hkv, G * T, n)
    v = torch.cat([_context(s, s["vc"], s["vs"]), s["v"].float().transpose(1, 2)], 2)
    o = torch.matmul(p, v)
    s["out"].copy_(o.view(R, Hkv, G, T, D).permute(0, 3, 1, 2, 4).reshape(R, T, Hq, D))


def _children(s):
    """Every position's parent on the card, once per pass as a program with new trees does."""
    return torch.tensor(s["parent"], device="cuda")


def _plain_sample(s):
    case = s["case"]
    R, T, V = case["R"], case["T"], case["V"]
    tok, u = s["tokens"].long(), s["u"].double()
    x = s["logits"].float() / s["tau"].view(R, 1, 1)
    top = x.amax(-1, keepdim=True)
    total = torch.exp(x - top).sum(-1, dtype=torch.float64)                            # [R, T]
    par = _children(s).clamp(min=0)
    prob = torch.ones(R, T, dtype=torch.float64, device="cuda")
    prow = torch.arange(R, device="cuda").view(R, 1).expand(R, T)
    own_p = torch.exp((x[prow, par, tok] - top[prow, par, 0]).double()) / total[prow, par]
    prob[:, 1:] = own_p[:, 1:]
    s["token_prob"].copy_(prob)
    if case["drafts"]:
        ok = u[:, 1:] * s["dq"][prow, par, tok].double()[:, 1:] < prob[:, 1:]
        n = torch.cumprod(ok.long(), 1).sum(1)
        node = n
        taken = [[] for _ in range(R)]
        steps = torch.arange(T, device="cuda")
        s["path"].copy_(torch.where(steps <= n.view(R, 1), steps, -1))
        s["node"].copy_(n)
        s["len"].copy_(n)
    else:
        ph, uh = prob.tolist(), u.tolist()       # the walk of a tree is a program on the host
        th = tok.tolist()
        nodes, taken = [], []
        for r in range(R):
            at, route, gone = 0, [0], []
            while True:
                kids = [t for t in range(at + 1, T) if s["parent"][r][t] == at]
                left, gone, nxt = 1.0, [], None
                for t in kids:
                    if th[r][t] in gone:
                        continue
                    if uh[r][t] * left < ph[r][t]:
                        nxt = t
                        break
                    left -= ph[r][t]
                    gone.append(th[r][t])
                if nxt is None:
                    break
                at = nxt
                route.append(at)
            nodes.append(at)
            taken.append(gone)
            s["path"][r].copy_(torch.tensor(route + [-1] * (T - len(route))))
            s["len"][r] = len(route) - 1
        node = torch.tensor(nodes, device="cuda")
        s["node"].copy_(node)
    rows = torch.arange(R, device="cuda")
    y = s["logits"][rows, node].double() / s["tau"].double().view(R, 1)                # 64 bits: the borders of a long sum
    w = torch.exp(y - y.amax(-1, keepdim=True))
    if case["drafts"]:
        rest = torch.clamp(w / w.sum(-1, keepdim=True) - s["dq"][rows, node].double(), min=0)
        rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
        w = torch.where((node < T - 1).view(R, 1), rest, w)
    for r in range(R):
        if taken[r]:
            w[r, torch.tensor(taken[r], device="cuda")] = 0
    c = torch.cumsum(w, -1)
    s["bonus"].copy_((c <= u[:, :1] * c[:, -1:]).sum(-1).clamp(max=V - 1))


def _plain_append(s):
    case = s["case"]
    R, T, S = case["R"], case["T"], case["page"]
    step = torch.arange(T, device="cuda").expand(R, T)
    keep = step <= s["alen"].view(R, 1)
    slot = s["seq_len"].view(R, 1) + step
    r = torch.arange(R, device="cuda").view(R, 1).expand(R, T)[keep]
    src = (s["path"] if case["tree"] else step)[keep].long()
    slot = slot[keep].long()
    page = s["table"][r, slot // S].long()
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        rows = x[:, r, src].float()                              # [L, n, Hkv, D]
        if scale is not None:
            rows = (rows / scale.view(scale.shape[0], 1, -1, 1)).clamp_(-448, 448)
        rows = rows.to(cache.dtype)
        if cache.dtype == F8:
            cache.view(torch.uint8)[:, page, :, slot % S] = rows.view(torch.uint8).transpose(0, 1)
        else:
            cache[:, page, :, slot % S] = rows.transpose(0, 1)
    s["new_len"].copy_(s["seq_len"] + s["alen"] + 1)


_PLAIN = {"rope": _plain_rope, "attn": _plain_attn, "sample": _plain_sample, "append": _plain_append}


# --- what a pass cannot do without --------------------------------------------

def work(case):
    R, T = case["R"], case["T"]
    op = case["op"]
    if op == "rope":
        n = R * T * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 2 * n * SIZE[case["dtype"]], "flops": 8 * n}
    if op == "attn":
        Hq, Hkv, D, W = case["Hq"], case["Hkv"], case["D"], case["window"]
        slots = sum(min(n, W) if W else n for n in _lengths(case))
        span = R * T * (2 * Hq + 2 * Hkv) * D * SIZE[case["dtype"]]
        return {"bytes": 2 * slots * Hkv * D * SIZE[case["cache"]] + span,
                "flops": 4 * D * Hq * T * (slots + R * (T + 1) / 2)}
    if op == "sample":
        n = R * T * case["V"]
        row = R * case["V"] * 4 if case["drafts"] else 0         # one row of draft probabilities a request
        return {"bytes": n * SIZE[case["dtype"]] + row, "flops": 4 * n}
    rows = R * (0.75 * T if not case["tree"] else min(T, 5))     # about the accepted rows
    n = rows * case["L"] * 2 * case["Hkv"] * case["D"]
    return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["cache"]]), "flops": n}


# --- the definition in 64 bits --------------------------------------------------

def exact(case, seed):
    if case["op"] == "attn" and case["R"] * case["T"] * case["Hq"] * case["ctx"] > 2.5e8:
        return None
    s = _inputs(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "sample": _exact_sample, "append": _exact_append}[case["op"]](s)


def _exact_rope(s):
    case = s["case"]
    rot, D, R, T = case["rot"], case["D"], case["R"], case["T"]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        n = torch.linalg.vector_norm(x.double(), dim=-1, keepdim=True)
        y = x.double() / torch.sqrt(n ** 2 / D + 1e-6) * w.double()
        # each pair as one complex number, turned by its angle
        first = torch.arange(rot // 2, device="cuda") * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else rot // 2)
        z = torch.complex(y[..., first], y[..., second])
        where = (s["seq_len"].double()[:, None] + s["depth"].double())[:, :, None, None]
        z = z * torch.polar(torch.ones_like(s["freq"]).expand(R, T, 1, -1), where * s["freq"])
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_attn(s):
    case = s["case"]
    R, T, Hq, Hkv, D, S, W = (case[x] for x in ("R", "T", "Hq", "Hkv", "D", "page", "window"))
    out = torch.zeros(R, T, Hq, D, dtype=torch.float64, device="cuda")
    for r in range(R):
        n = int(s["seq_len"][r])
        at = torch.arange(n, device="cuda")
        pages = s["table"][r][at // S].long()
        place = [n + d for d in _depths(s["parent"][r])]
        for h in range(Hkv):
            k, v = [], []
            for cache, scale, span, into in ((s["kc"], s["ks"], s["k"], k), (s["vc"], s["vs"], s["v"], v)):
                raw = cache[:, h].view(torch.uint8) if cache.dtype == F8 else cache[:, h]
                rows = raw[pages, at % S]
                rows = (rows.view(F8).float() if cache.dtype == F8 else rows).double()
                into.append(rows if scale is None else rows * scale[h].double())
                into.append(span[r, :, h].double())
            k, v = torch.cat(k), torch.cat(v)
            for t in range(T):
                route, a = [], t
                while a >= 0:
                    route.append(a)
                    a = s["parent"][r][a]
                if W:
                    route = [a for a in route if place[t] - place[a] < W]
                first = max(0, place[t] - W + 1) if W else 0
                pick = torch.cat([at[min(first, n):], torch.tensor(route, device="cuda") + n])
                q = s["q"][r, t, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
                w = torch.softmax(q @ k[pick].t() / math.sqrt(D), -1)
                out[r, t, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = w @ v[pick]
    return out


def _exact_sample(s):
    case = s["case"]
    R, T, V = case["R"], case["T"], case["V"]
    prob = torch.ones(R, T, dtype=torch.float64)
    node, length, bonus = (torch.zeros(R, dtype=torch.int32) for _ in range(3))
    path = torch.full((R, T), -1, dtype=torch.int32)
    for r in range(R):
        p = torch.softmax(s["logits"][r].double() / s["tau"][r].double(), -1)
        tok, u, par = s["tokens"][r].tolist(), s["u"][r].double().tolist(), s["parent"][r]
        for t in range(1, T):
            prob[r, t] = p[par[t], tok[t]]
        route, rest, going = [0], p[0].clone(), True
        while going:
            going, at = False, route[-1]
            rest = p[at].clone()
            for t in range(at + 1, T):
                if par[t] != at:
                    continue
                if case["drafts"]:
                    q = s["dq"][r, at].double()
                    going = u[t] * float(q[tok[t]]) < float(p[at, tok[t]])
                    if not going:
                        rest = torch.relu(p[at] - q)
                        if float(rest.sum()) == 0:
                            rest = p[at].clone()
                else:
                    going = u[t] * float(rest.sum()) < float(rest[tok[t]])
                    if not going:
                        rest[tok[t]] = 0
                if going:
                    route.append(t)
                    break
        node[r], length[r] = route[-1], len(route) - 1
        path[r, :len(route)] = torch.tensor(route, dtype=torch.int32)
        c = torch.cumsum(rest, 0)
        bonus[r] = min(V - 1, int(torch.searchsorted(c, (u[0] * c[-1]).reshape(1), right=True)))
    return prob, node, length, path, bonus


def _exact_append(s):
    case = s["case"]
    S = case["page"]
    out = []
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        c = cache.float().double()
        for r in range(case["R"]):
            for i in range(int(s["alen"][r]) + 1):
                at = int(s["seq_len"][r]) + i
                t = int(s["path"][r, i]) if case["tree"] else i
                row = x[:, r, t].double()
                if scale is not None:
                    row = torch.clamp(row / scale.double()[:, :, None], -448.0, 448.0)
                c[:, int(s["table"][r, at // S]), :, at % S] = row
        out.append(c)
    return out[0], out[1], s["seq_len"] + s["alen"] + 1

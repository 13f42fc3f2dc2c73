"""Measured cases of serving many sampled requests behind one prompt.

Three operators around a verify step: pages for the new positions of every
request (kv_pages_reserve, kv_pages_release), attention of the requests' spans
over a prefix that all of them share and over their own contexts
(attn_verify_shared), and acceptance by sampling from the target's probabilities
after top-k, top-p and min-p (accept_sample_filtered). ``run`` computes the plain
form with elementary torch operations, or calls the library where ``own`` is
true; ``exact`` is the definition in 64 bits.
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
        # Plain decoding of sixteen requests behind one system prompt.
        dict(name="shared-decode-r16", op="attn", R=16, T=1, Hq=24, Hkv=4, D=256, dtype="bf16", cache="bf16",
             prefix=4096, ctx=300, page=64, tree=False, window=0),
        # Sixteen chains of 16 drafts behind one long document.
        dict(name="shared-chain-r16", op="attn", R=16, T=17, Hq=24, Hkv=4, D=256, dtype="bf16", cache="bf16",
             prefix=26758, ctx=1000, page=64, tree=False, window=0),
        # Thirty-two draft trees over an 8-bit cache, small pages.
        dict(name="shared-tree-f8-r32", op="attn", R=32, T=23, Hq=32, Hkv=8, D=128, dtype="bf16", cache="f8",
             prefix=8191, ctx=500, page=16, tree=True, window=0),
        # The small float32 configuration with a draft model's window.
        dict(name="shared-f32-window", op="attn", R=3, T=9, Hq=4, Hkv=4, D=64, dtype="f32", cache="f32", prefix=1000,
             ctx=700, page=32, tree=False, window=2048),
        # The next token of one request: launch latency.
        dict(name="filter-decode-1", op="sample", R=1, T=1, V=151936, dtype="bf16", tree=False, drafts=False,
             k=20, p=0.95, m=0.0, mixed=False, flat=False),
        # Sixteen chains with their drafts' probabilities, the usual settings.
        dict(name="filter-chain-r16", op="sample", R=16, T=17, V=151936, dtype="bf16", tree=False, drafts=True,
             k=20, p=0.95, m=0.0, mixed=False, flat=False),
        # Even distributions cut by top-p alone: tens of thousands of tokens stay.
        dict(name="filter-flat-r8", op="sample", R=8, T=9, V=151936, dtype="bf16", tree=False, drafts=True,
             k=0, p=0.9, m=0.0, mixed=False, flat=True),
        # Draft trees, float32 logits, another setting for every request.
        dict(name="filter-tree-r4", op="sample", R=4, T=23, V=151936, dtype="f32", tree=True, drafts=False,
             k=50, p=0.9, m=0.05, mixed=True, flat=False),
        # Pages for one verify step of sixteen requests, two of them new.
        dict(name="pages-step-r16", op="pages", R=16, new=17, page=64, ctx=8192, prefix=64, fresh=8, short=False),
        # Pages for the prompts of 256 new requests.
        dict(name="pages-prompt-r256", op="pages", R=256, new=32768, page=16, ctx=1, prefix=32, fresh=1, short=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "sample", "sample", "pages"])
    tree = rng.random() < 0.4
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "attn":
        cache = rng.choice(["bf16", "f8"]) if dtype == "bf16" else "f32"
        Hkv, D, G = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.randint(1, 8)
        T = rng.randint(2, 64) if tree else rng.choice([1, rng.randint(2, 17), rng.randint(18, 64)])
        R = _log(rng, 1, 64)
        # at most the largest listed case's products
        most = int((3e9 if dtype == "f32" else 3e10) / (R * T * G * Hkv * D))
        return dict(op=op, R=R, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, cache=cache,
                    prefix=_log(rng, 1, max(2, min(32768, most))), ctx=_log(rng, 1, max(2, min(4096, most // 2))),
                    page=rng.choice([16, 32, 64, 128]), tree=tree, window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]))
    if op == "sample":
        T = rng.choice([1, rng.randint(2, 17), rng.randint(18, 64)])
        R = rng.randint(1, max(1, min(64, 200 // T)))
        return dict(op=op, R=R, T=T, V=8 * _log(rng, 16, 18992), dtype=dtype, tree=tree and T > 1,
                    drafts=not tree and rng.random() < 0.6, k=rng.choice([0, _log(rng, 1, 2000)]),
                    p=rng.choice([1.0, rng.uniform(0.3, 0.99)]), m=rng.choice([0.0, rng.uniform(0.01, 0.3)]),
                    mixed=rng.random() < 0.5, flat=rng.random() < 0.3)
    page = rng.choice([16, 32, 64, 128])
    return dict(op=op, R=_log(rng, 1, 256), new=rng.choice([1, 17, _log(rng, 2, 8192)]), page=page,
                ctx=_log(rng, 1, 16384), prefix=rng.choice([0, rng.randint(1, 64)]), fresh=rng.randint(1, 8),
                short=rng.random() < 0.3)


# --- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


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


def _own_lengths(case):
    """Ragged own contexts behind the prefix, fixed by the case."""
    return [case["ctx"] - (r * 7919) % (case["ctx"] // 2 + 1) for r in range(case["R"])]


def _inputs_attn(case, seed):
    g = _gen(seed)
    R, T, Hq, Hkv, D, S, P = (case[x] for x in ("R", "T", "Hq", "Hkv", "D", "page", "prefix"))
    s = dict(case=case, parent=_parents(case, seed))
    dt, ct = DTYPES[case["dtype"]], DTYPES[case["cache"]]
    depth = [_depths(p) for p in s["parent"]]
    s["depth"] = torch.tensor(depth, device="cuda")
    s["q"], s["k"], s["v"] = (_fill((R, T, h, D), g, dt) for h in (Hq, Hkv, Hkv))
    # A shared page list for the prefix, then every request's own pages; a
    # page that the prefix ends in is the request's own copy.
    whole, total = P // S, (P + case["ctx"] + T + S - 1) // S
    n = (P + S - 1) // S + R * (total - whole)
    order = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    s["prefix_table"] = order[:(P + S - 1) // S].contiguous()
    rest = order[(P + S - 1) // S:].reshape(R, total - whole)
    s["table"] = torch.cat([order[:whole].expand(R, whole), rest], 1).contiguous()
    gain = 64.0 if ct == F8 else 1.0
    s["kc"], s["vc"] = (_fill((n, Hkv, S, D), g, ct, gain) for _ in range(2))
    s["ks"] = s["vs"] = None
    if ct == F8:
        s["ks"], s["vs"] = ((1 + 0.1 * torch.rand(Hkv, generator=g, device="cuda")) / 64 for _ in range(2))
    s["seq_len"] = torch.tensor([P + x for x in _own_lengths(case)], dtype=torch.int32, device="cuda")
    s["prefix_len"] = torch.tensor([P], dtype=torch.int32, device="cuda")
    s["out"] = torch.empty(R, T, Hq, D, dtype=dt, device="cuda")
    anc = [[[False] * T for _ in range(T)] for _ in range(R)]        # root path and window of every span position
    for r in range(R):
        for t in range(T):
            a = t
            while a >= 0 and (case["window"] == 0 or depth[r][t] - depth[r][a] < case["window"]):
                anc[r][t][a] = True
                a = s["parent"][r][a]
    s["anc"] = torch.tensor(anc, device="cuda")
    return s


def _inputs_sample(case, seed):
    g = _gen(seed)
    R, T, V = case["R"], case["T"], case["V"]
    s = dict(case=case, parent=_parents(case, seed))
    if case["flat"]:
        z = torch.randn(R, T, V, generator=g, device="cuda") * 2.5
    else:
        # A few likely tokens above a wide floor, as a language model's rows look.
        z = torch.randn(R, T, V, generator=g, device="cuda") * 2.0
        head = torch.randint(V, (R, T, 40), generator=g, device="cuda")
        z.scatter_reduce_(2, head, 14 + 2.5 * torch.randn(R, T, 40, generator=g, device="cuda"), "amax")
    s["logits"] = z.to(DTYPES[case["dtype"]])
    s["tau"] = (0.7 + 0.6 * torch.rand(R, generator=g, device="cuda")).float()
    which = torch.arange(R, device="cuda") % 4 if case["mixed"] else torch.full((R,), -1, device="cuda")
    s["top_k"] = torch.where(which == 0, 0, case["k"]).to(torch.int32)
    s["top_p"] = torch.where(which == 1, 1.0, case["p"]).float()
    s["min_p"] = torch.where(which == 2, 0.0, case["m"]).float()
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
    return s


def _inputs_pages(case, seed):
    """A step's pages: every fresh-th request has ended and another one starts behind the prefix in its place."""
    R, S, new, pre = case["R"], case["page"], case["new"], case["prefix"]
    rnd = torch.Generator().manual_seed(int(seed) * 7 + 3)
    grow = torch.randint(0, 4, (R,), generator=rnd)
    lens = torch.tensor([pre * S + max(0, x - i) for x, i in zip(_own_lengths(case), grow.tolist())])
    ended = torch.arange(R) % case["fresh"] == 0
    asked = torch.where(ended, torch.randint(max(1, new // 2), new + 1, (R,), generator=rnd), new)
    held = torch.where(ended & (case["ctx"] == 1), pre, (lens + S - 1) // S)
    start = torch.where(ended, pre * S, lens)                       # what a request has behind it in this step
    most = pre + (case["ctx"] + new + S - 1) // S + 1
    want = (start + asked + S - 1) // S - torch.where(ended, pre, held)
    freed = torch.where(ended, held - pre, 0)
    spare = int(want.sum() - freed.sum()) if not case["short"] else int(want.sum() * 0.6 - freed.sum())
    spare = max(0, spare) + (0 if case["short"] else 1000)
    n = pre + R * (most - pre) + 1000                                # some are in use elsewhere
    order = torch.randperm(n, generator=rnd).to(torch.int32)
    table = torch.full((R, most), -1, dtype=torch.int32)
    table[:, :pre] = order[:pre]
    mine = (torch.arange(most)[None] >= pre) & (torch.arange(most)[None] < held[:, None])
    table[mine] = order[pre:pre + int(mine.sum())]
    spare = min(spare, n - pre - int(mine.sum()))
    free = torch.full((n,), -1, dtype=torch.int32)
    free[:spare] = order[n - spare:]
    i32 = lambda x: x.to(torch.int32).cuda()
    return dict(case=case, n_pages=n, prefix_table=i32(order[:pre]) if pre else None, table=table.cuda(), held=i32(held),
                free=free.cuda(), n_free=torch.tensor([spare], dtype=torch.int32, device="cuda"),
                keep=i32(torch.where(ended, 0, lens)), seq_len=i32(start), n_new=i32(asked),
                slots=torch.zeros(R, new, dtype=torch.int64, device="cuda"))


_INPUTS = {"attn": _inputs_attn, "sample": _inputs_sample, "pages": _inputs_pages}


def prepare(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    if own:
        import numpy as np

        import hybrid_recurrent_state_amd as hrs
        bytes_ = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
        par = np.asarray(s["parent"], dtype=np.int32) if case.get("tree") else None
        if case["op"] == "attn":
            ws = bytes_(hrs.attn_verify_shared_workspace_bytes(case["R"], case["T"], case["Hq"], case["Hkv"], case["D"]))
            s["calls"] = [hrs.attn_verify_shared_call(
                s["q"], s["k"], s["v"], s["kc"], s["vc"], s["prefix_table"], s["prefix_len"], s["table"], s["seq_len"],
                s["out"], ws, parent=par, window=case["window"], k_scale=s["ks"], v_scale=s["vs"])]
        elif case["op"] == "sample":
            ws = bytes_(hrs.accept_sample_filtered_workspace_bytes(case["R"], case["T"], case["V"]))
            s["calls"] = [hrs.accept_sample_filtered_call(
                s["logits"], s["tokens"], s["u"], s["token_prob"], s["node"], s["len"], s["path"], s["bonus"], ws,
                top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], draft_probs=s["dq"], temperature=s["tau"],
                parent=par)]
        else:
            ws = bytes_(hrs.kv_pages_workspace_bytes(case["R"]))
            s["calls"] = [
                hrs.kv_pages_release_call(s["keep"], s["table"], s["held"], s["free"], s["n_free"], ws,
                                          page_size=case["page"], n_prefix=case["prefix"]),
                hrs.kv_pages_reserve_call(s["seq_len"], s["table"], s["held"], s["free"], s["n_free"], ws,
                                          page_size=case["page"], n_new=s["n_new"], prefix_table=s["prefix_table"],
                                          slot_map=s["slots"])]
    return s


# --- one pass ---------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        for call in state["calls"]:
            call()
    else:
        _PLAIN[op](state)
    if op == "attn":
        return state["out"]
    if op == "sample":
        return state["token_prob"], state["node"], state["len"], state["path"], state["bonus"]
    return state["table"], state["held"], state["free"], state["n_free"], state["slots"]


def _slots_of(cache, table, scale):
    """Pages in a row, in 32 bits: table [..., P] -> [..., Hkv, slots, D]."""
    x = cache.view(torch.uint8)[table.long()].view(F8) if cache.dtype == F8 else cache[table.long()]
    x = x.float().transpose(-4, -3)                                  # [..., Hkv, P, S, D]
    x = x.flatten(-3, -2)
    return x if scale is None else x * scale.view(-1, 1, 1)


def _plain_attn(s):
    case = s["case"]
    R, T, Hq, Hkv, D, S, P = (case[x] for x in ("R", "T", "Hq", "Hkv", "D", "page", "prefix"))
    G, W = Hq // Hkv, case["window"]
    length = s["seq_len"].view(R, 1, 1)
    first = length + s["depth"].view(R, T, 1) - W + 1 if W else torch.zeros_like(length)
    q = s["q"].float().view(R, T, Hkv, G, D).permute(2, 0, 3, 1, 4)                   # [Hkv, R, G, T, D]
    # the prefix: one product for the rows of all requests
    k = _slots_of(s["kc"], s["prefix_table"], s["ks"])[:, :P]
    n = k.shape[1]
    j = torch.arange(n, device="cuda")
    a = torch.matmul(q.reshape(Hkv, R * G * T, D), k.transpose(1, 2).contiguous()) / math.sqrt(D)
    a = a.view(Hkv, R, G, T, n).masked_fill_(~((j < length) & (j >= first)).view(1, R, 1, -1, n), -math.inf)
    # the requests' own contexts and spans
    whole = P // S
    k = torch.cat([_slots_of(s["kc"], s["table"][:, whole:], s["ks"]), s["k"].float().transpose(1, 2)], 2)
    m = k.shape[2]
    j = whole * S + torch.arange(m - T, device="cuda")
    seen = ((j >= P) & (j < length) & (j >= first)).expand(R, T, m - T)
    mask = torch.cat([seen, s["anc"]], 2).view(R, 1, 1, T, m)
    b = torch.matmul(q.permute(1, 0, 2, 3, 4).reshape(R, Hkv, G * T, D), k.transpose(2, 3).contiguous()) / math.sqrt(D)
    b = b.view(R, Hkv, G, T, m).masked_fill_(~mask, -math.inf)
    top = torch.maximum(a.amax(-1).transpose(0, 1), b.amax(-1))                        # [R, Hkv, G, T]
    a = torch.exp_(a.sub_(top.transpose(0, 1)[..., None]))
    b = torch.exp_(b.sub_(top[..., None]))
    total = a.sum(-1).transpose(0, 1) + b.sum(-1)
    v = _slots_of(s["vc"], s["prefix_table"], s["vs"])[:, :P]
    o = torch.matmul(a.view(Hkv, R * G * T, n), v).view(Hkv, R, G, T, D).transpose(0, 1)
    v = torch.cat([_slots_of(s["vc"], s["table"][:, whole:], s["vs"]), s["v"].float().transpose(1, 2)], 2)
    o = o + torch.matmul(b.view(R, Hkv, G * T, m), v).view(R, Hkv, G, T, D)
    o = o / total[..., None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(R, T, Hq, D))


def _plain_sample(s):
    case = s["case"]
    R, T, V = case["R"], case["T"], case["V"]
    tok, u = s["tokens"].long(), s["u"].double()
    per = lambda x: x.view(R, 1, 1)
    # 64 bits: borders of cumulative sums decide which tokens stay
    z, order = torch.sort(s["logits"].float(), dim=-1, descending=True, stable=True)
    w = torch.exp((z - z[..., :1]).double() / per(s["tau"].double()))
    rank = torch.arange(V, device="cuda")
    k = per(torch.where((s["top_k"] <= 0) | (s["top_k"] > V), V, s["top_k"]))
    w = torch.where(rank < k, w, 0.0)
    c = torch.cumsum(w, -1)
    p = per(s["top_p"].double())
    w = torch.where((p >= 1) | (c - w < p * c[..., -1:]) | (rank == 0), w, 0.0)
    w = torch.where(w >= per(s["min_p"].double()), w, 0.0)
    w = torch.zeros_like(w).scatter_(-1, order, w / w.sum(-1, keepdim=True))           # p, by token
    par = torch.tensor(s["parent"], device="cuda")
    prow = torch.arange(R, device="cuda").view(R, 1).expand(R, T)
    up = par.clamp(min=0)
    prob = torch.where(par < 0, 1.0, w[prow, up, tok])
    s["token_prob"].copy_(prob)
    rows = torch.arange(R, device="cuda")
    need = u * s["dq"][prow, up, tok].double() if case["drafts"] else u
    # positions in index order: a node's children come after it, in the order in which they are tried
    node = torch.zeros(R, dtype=torch.int64, device="cuda")
    depth = torch.zeros_like(node)
    left = torch.ones(R, dtype=torch.float64, device="cuda")
    path = torch.full((R, T), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    out = torch.zeros(R, T, dtype=torch.bool, device="cuda")         # rejected children of the node
    for t in range(1, T):
        again = (out & (tok == tok[:, t:t + 1])).any(1)
        tried = (par[:, t] == node) & ~again
        ok = tried & (need[:, t] * left < prob[:, t])
        bad = tried & ~ok
        left = torch.where(ok, 1.0, torch.where(bad, left - prob[:, t], left))
        out[:, t] |= bad
        out &= ~ok.view(R, 1)
        node = torch.where(ok, t, node)
        depth = depth + ok
        path[rows, depth] = torch.where(ok, t, path[rows, depth])
    s["node"].copy_(node)
    s["len"].copy_(depth)
    s["path"].copy_(path)
    plain = w[rows, node]
    if case["drafts"]:
        rest = torch.clamp(plain - s["dq"][rows, node].double(), min=0)
        rest = torch.where((node < T - 1).view(R, 1), rest, plain)
    else:
        rest = plain.scatter(1, tok, torch.where(out, 0.0, plain.gather(1, tok)))
        # a token that several positions carry is gone if any of them was rejected
        gone = torch.zeros_like(plain).scatter_add_(1, tok, out.double()) > 0
        rest = torch.where(gone, 0.0, rest)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, plain)
    c = torch.cumsum(rest, -1)
    s["bonus"].copy_((c <= u[:, :1] * c[:, -1:]).sum(-1).clamp(max=V - 1))


def _plain_pages(s):
    case = s["case"]
    R, S, pre = case["R"], case["page"], case["prefix"]
    table, held, free, n_free = s["table"], s["held"], s["free"], s["n_free"]
    at = torch.arange(table.shape[1], device="cuda").view(1, -1)
    # back on top of the list, in the order of the requests
    keep = ((s["keep"] + S - 1) // S).clamp(min=pre)
    back = (at >= keep.view(R, 1)) & (at < held.view(R, 1))
    place = torch.cumsum(back.view(-1).long(), 0).view(R, -1) - 1 + n_free
    spill = torch.cat([free, free[:1]])                              # one more place for what is not given back
    spill.scatter_(0, torch.where(back, place, free.shape[0]).view(-1), table.view(-1))
    free.copy_(spill[:-1])
    n_free.add_(back.sum().int())
    table.copy_(torch.where(back, -1, table))
    held.copy_(torch.minimum(held, keep))
    # off the top, in the order of the requests, while they last
    have = held.clamp(min=pre)
    want = (s["seq_len"] + s["n_new"] + S - 1) // S
    need = (want - have).clamp(min=0)
    upto = torch.cumsum(need.long(), 0)
    given = torch.where((need == 0) | (upto <= n_free), need, 0)
    upto = torch.cumsum(given.long(), 0)
    base = n_free - upto[-1]
    got = (at >= have.view(R, 1)) & (at < (have + given).view(R, 1))
    source = (base + upto - given - have).view(R, 1) + at
    table.copy_(torch.where(got, free[source.clamp(0, free.shape[0] - 1)], table))
    if pre:
        table[:, :pre] = torch.where(held.view(R, 1) < pre, s["prefix_table"], table[:, :pre])
    held.copy_(have + given)
    n_free.copy_(base)
    t = torch.arange(case["new"], device="cuda")
    slot = s["seq_len"].view(R, 1).long() + t
    page = table.gather(1, (slot // S).clamp(max=table.shape[1] - 1)).long()
    on = (t < s["n_new"].view(R, 1)) & (slot // S < held.view(R, 1))
    s["slots"].copy_(torch.where(on, page * S + slot % S, -1))


_PLAIN = {"attn": _plain_attn, "sample": _plain_sample, "pages": _plain_pages}


# --- what a pass cannot do without --------------------------------------------

def work(case):
    R = case["R"]
    if case["op"] == "attn":
        T, Hq, Hkv, D, P, W = (case[x] for x in ("T", "Hq", "Hkv", "D", "prefix", "window"))
        lens = [P + x for x in _own_lengths(case)]
        first = [max(0, n - W) if W else 0 for n in lens]
        prefix = max(0, P - min(first))
        own_slots = sum(n - max(P, f) for n, f in zip(lens, first))
        seen = sum(n - f for n, f in zip(lens, first))
        span = R * T * (2 * Hq + 2 * Hkv) * D * SIZE[case["dtype"]]
        return {"bytes": 2 * (prefix + own_slots) * Hkv * D * SIZE[case["cache"]] + span,
                "flops": 4 * D * Hq * T * (seen + R * (T + 1) / 2)}
    if case["op"] == "sample":
        n = R * case["T"] * case["V"]
        row = R * case["V"] * 4 if case["drafts"] else 0             # one row of draft probabilities a request
        return {"bytes": n * SIZE[case["dtype"]] + row, "flops": 4 * n}
    if case["ctx"] == 1:
        entries = R * 0.75 * case["new"] / case["page"]
    else:
        entries = R * case["new"] / case["page"] + R / case["fresh"] * case["ctx"] / case["page"]
    return {"bytes": 16 * entries + 8 * R * case["new"] + 20 * R, "flops": 4 * R * case["new"]}


# --- the definition in 64 bits --------------------------------------------------

def exact(case, seed):
    if case["op"] == "attn":
        if case["R"] * case["T"] * case["Hq"] * (case["prefix"] + case["ctx"]) > 2.5e8:
            return None
        return _exact_attn(_inputs_attn(case, seed))
    if case["op"] == "sample":
        return _exact_sample(_inputs_sample(case, seed))
    return _exact_pages(_inputs_pages(case, seed))


def _exact_attn(s):
    case = s["case"]
    R, T, Hq, Hkv, D, S, W, P = (case[x] for x in ("R", "T", "Hq", "Hkv", "D", "page", "window", "prefix"))
    out = torch.zeros(R, T, Hq, D, dtype=torch.float64, device="cuda")
    G = Hq // Hkv
    for h in range(Hkv):
        caches = []
        for cache, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
            c = (cache[:, h].view(torch.uint8).contiguous().view(F8).float() if cache.dtype == F8 else cache[:, h]).double()
            caches.append(c if scale is None else c * scale[h].double())
        for r in range(R):
            n = int(s["seq_len"][r])
            at = torch.arange(n, device="cuda")
            pages = s["table"][r][at // S].long()
            pages[:P] = s["prefix_table"][at[:P] // S].long()
            k = torch.cat([caches[0][pages, at % S], s["k"][r, :, h].double()])
            v = torch.cat([caches[1][pages, at % S], s["v"][r, :, h].double()])
            dep = _depths(s["parent"][r])
            count = torch.zeros(T, n + T, dtype=torch.bool)
            for t in range(T):
                count[t, max(0, n + dep[t] - W + 1) if W else 0:n] = True
                a = t
                while a >= 0:
                    count[t, n + a] = W == 0 or dep[t] - dep[a] < W
                    a = s["parent"][r][a]
            q = s["q"][r, :, h * G:(h + 1) * G].double()               # [T, G, D]
            x = (q.reshape(T * G, D) @ k.t()).view(T, G, n + T) / math.sqrt(D)
            x = x.masked_fill(~count.cuda()[:, None], -math.inf)
            out[r, :, h * G:(h + 1) * G] = (torch.softmax(x, -1).reshape(T * G, -1) @ v).view(T, G, D)
    return out


def _exact_sample(s):
    case = s["case"]
    R, T, V = case["R"], case["T"], case["V"]
    prob = torch.ones(R, T, dtype=torch.float64)
    node, length, bonus = (torch.zeros(R, dtype=torch.int32) for _ in range(3))
    path = torch.full((R, T), -1, dtype=torch.int32)
    for r in range(R):
        k, top_p, min_p = int(s["top_k"][r]), float(s["top_p"][r]), float(s["min_p"][r])
        rows = []
        for t in range(T):
            full = torch.softmax(s["logits"][r, t].double() / s["tau"][r].double(), 0)
            by = torch.argsort(s["logits"][r, t].float(), descending=True, stable=True)
            if 0 < k < V:
                by = by[:k]
            mass = full[by]
            if top_p < 1:
                before = torch.cumsum(mass, 0) - mass
                by = by[:max(1, int((before < top_p * mass.sum()).sum()))]
            by = by[full[by] >= min_p * full.max()]
            row = torch.zeros_like(full)
            row[by] = full[by] / full[by].sum()
            rows.append(row)
        tok, u, par = s["tokens"][r].tolist(), s["u"][r].double().tolist(), s["parent"][r]
        for t in range(1, T):
            prob[r, t] = rows[par[t]][tok[t]]
        route, going = [0], True
        while going:
            going, at = False, route[-1]
            p = rows[at]
            rest = p.clone()
            for t in range(at + 1, T):
                if par[t] != at:
                    continue
                if case["drafts"]:
                    q = s["dq"][r, at].double()
                    going = u[t] * float(q[tok[t]]) < float(p[tok[t]])
                    if not going:
                        rest = torch.relu(p - q)
                else:
                    going = u[t] * float(rest.sum()) < float(rest[tok[t]])
                    if not going:
                        rest[tok[t]] = 0
                if going:
                    route.append(t)
                    break
        if float(rest.sum()) == 0:
            rest = p
        node[r], length[r] = route[-1], len(route) - 1
        path[r, :len(route)] = torch.tensor(route, dtype=torch.int32)
        c = torch.cumsum(rest, 0)
        bonus[r] = min(V - 1, int(torch.searchsorted(c, (u[0] * c[-1]).reshape(1), right=True)))
    return prob, node, length, path, bonus


def _exact_pages(s):
    case = s["case"]
    S, pre = case["page"], case["prefix"]
    table = s["table"].cpu().numpy().copy()
    held, keep, start, new = (s[x].tolist() for x in ("held", "keep", "seq_len", "n_new"))
    stack = s["free"].tolist()
    top = int(s["n_free"][0])
    shared = s["prefix_table"].cpu().numpy() if pre else None
    for r in range(case["R"]):
        kept = max(pre, -(-keep[r] // S))
        if kept < held[r]:
            stack[top:top + held[r] - kept] = table[r, kept:held[r]].tolist()
            top += held[r] - kept
            table[r, kept:held[r]] = -1
            held[r] = kept
    left, gets = top, []
    for r in range(case["R"]):
        need = max(0, -(-(start[r] + new[r]) // S) - max(pre, held[r]))
        left -= need
        gets.append(need if need == 0 or left >= 0 else 0)
    top -= sum(gets)
    at = top
    slots = torch.full((case["R"], case["new"]), -1, dtype=torch.int64)
    for r in range(case["R"]):
        if held[r] < pre:
            table[r, held[r]:pre] = shared[held[r]:pre]
            held[r] = pre
        table[r, held[r]:held[r] + gets[r]] = stack[at:at + gets[r]]
        at += gets[r]
        held[r] += gets[r]
        j = torch.arange(start[r], start[r] + new[r])
        page = torch.from_numpy(table[r])[(j // S).clamp(max=table.shape[1] - 1)].long()
        slots[r, :new[r]] = torch.where(j // S < held[r], page * S + j % S, -1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return torch.from_numpy(table), i32(held), i32(stack), i32([top]), slots

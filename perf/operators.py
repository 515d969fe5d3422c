"""Windowed attention with sinks, attention over a paged cache, and the cache's writes: cases, inputs, plain forms.

Four calls are covered, named by a case's "op":

* ``window``      forward of causal attention with a sliding window and a few first tokens that stay visible
                  (what a prompt costs): o, lse.
* ``window_grad`` the same forward and its backward (a training step's attention): o, lse, dq, dk, dv.
* ``attend``      attention of T new tokens per sequence -- one, or a tree of drafted ones -- over a paged cache,
                  split and joined along the context: o, lse.
* ``append``      the new tokens' keys and values written into the cache's pages: both pools.
* ``accept``      drafted tokens written into the pages, then the accepted ones moved up behind the context: both pools.

Notation: q has H heads, k and v have Hkv (H a multiple of Hkv; head h reads head h // (H // Hkv)).  Query i sees key
j if j <= i and (i - j < window or j < sinks).  Over a cache, slot j < ctx holds position j, drafted token u sits in
slot ctx + u and stands at position ctx + (number of tokens it sees among the drafted, itself included) - 1; a drafted
token whose word in ``tree`` is zero is absent and its row is empty (o = 0, lse = -inf).
"""

import math

import numpy as np
import torch

own = False

NO_WINDOW = 2**31 - 1


# ------------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # training attention of a small language model (12 heads, context 1024) with a window of a quarter of it
        dict(name="grad_small", op="window_grad", B=8, H=12, Hkv=12, N=1024, d=64, window=256, sinks=4, layout="bhnd"),
        # training on long rows, query heads in groups of four that share keys and values, [B, N, H, d] tensors
        dict(name="grad_long", op="window_grad", B=2, H=16, Hkv=4, N=8192, d=128, window=1024, sinks=16, layout="bnhd"),
        # a training batch of odd sizes: ragged last tile, odd window, sinks that end inside a tile
        dict(name="grad_odd", op="window_grad", B=3, H=6, Hkv=2, N=1999, d=64, window=501, sinks=130, layout="bnhd"),
        # one short prompt: the smallest call, launch latency
        dict(name="prompt_short", op="window", B=1, H=12, Hkv=12, N=97, d=64, window=32, sinks=4, layout="bhnd"),
        # a long prompt with shared heads
        dict(name="prompt_long", op="window", B=1, H=8, Hkv=2, N=16384, d=128, window=4096, sinks=64, layout="bnhd"),
        # generation of one token for one user: latency
        dict(name="one_token", op="attend", B=1, H=12, Hkv=12, T=1, ctx=1000, ragged=False, d=64, page=16,
             window=NO_WINDOW, sinks=0, tree=False),
        # a serving batch, one token each, contexts of very different lengths
        dict(name="batch_tokens", op="attend", B=64, H=16, Hkv=4, T=1, ctx=8192, ragged=True, d=128, page=64,
             window=NO_WINDOW, sinks=0, tree=False),
        # drafted trees of 13 tokens under a window with sinks
        dict(name="tree_window", op="attend", B=16, H=16, Hkv=16, T=13, ctx=8192, ragged=True, d=128, page=32,
             window=2048, sinks=4, tree=True),
        # wide trees over long contexts with eight query heads to a key head: the largest, near compute bound
        dict(name="tree_wide", op="attend", B=4, H=32, Hkv=4, T=64, ctx=32768, ragged=True, d=128, page=128,
             window=NO_WINDOW, sinks=0, tree=True),
        # prompts of different lengths written into the cache
        dict(name="fill_prompts", op="append", B=8, Hkv=8, T=4096, ctx=0, ragged=True, d=128, page=64),
        # one decoding step's new token of a batch
        dict(name="fill_tokens", op="append", B=64, Hkv=4, T=1, ctx=777, ragged=True, d=128, page=16),
        # the end of a step with drafted trees: the accepted path moves up
        dict(name="accept_trees", op="accept", B=32, Hkv=16, T=32, ctx=500, ragged=True, d=128, page=32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_grad", "window_grad", "window", "attend", "attend", "attend", "append", "accept"])
    d = rng.choice([64, 128])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    if op in ("window", "window_grad"):
        # (where every row sees one key alone, dq and dk are zero and there is nothing to compare: training rows have more)
        N = _log_int(rng, 1, 16384) if op == "window" else _log_int(rng, 8, 8192)
        H = Hkv * group
        window = rng.choice([_log_int(rng, 1 if op == "window" else 4, 8192), _log_int(rng, 64, 2048)])
        sinks = rng.choice([0, rng.randint(1, 16), _log_int(rng, 1, 300)])
        # no more score entries than the largest listed case of its kind (the plain form writes them all)
        room = (2 * 16 * 8192**2) // (N * N * H) if op == "window_grad" else (8 * 16384**2) // (N * N * H)
        while room < 1:
            group, Hkv = (max(1, group // 2), Hkv) if group > 1 else (1, max(1, Hkv // 2))
            H = Hkv * group
            room = (2 * 16 * 8192**2) // (N * N * H) if op == "window_grad" else (8 * 16384**2) // (N * N * H)
        B = _log_int(rng, 1, min(room, 16))
        return dict(op=op, B=B, H=H, Hkv=Hkv, N=N, d=d, window=window, sinks=sinks, layout=rng.choice(["bhnd", "bnhd"]))
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "attend":
        tree = rng.random() < 0.5
        T = _log_int(rng, 2, 64) if tree else rng.choice([1, 1, rng.randint(2, 8)])
        ctx = _log_int(rng, 1, 32768)
        rows = max(1, (64 * 8192 * 4 * 128) // (ctx * Hkv * d))           # cache size of the largest listed case
        rows = min(rows, max(1, (4 * 32 * 64 * 32768 * 128) // (Hkv * group * T * ctx * d)))  # and its products
        B = _log_int(rng, 1, min(rows, 64))
        while B * Hkv * group * T * ctx * d > 4 * 32 * 64 * 32768 * 128:
            group, T = (group // 2, T) if group > 1 else (1, max(1, T // 2))
        window = rng.choice([NO_WINDOW, _log_int(rng, 1, 16384)])
        return dict(op=op, B=B, H=Hkv * group, Hkv=Hkv, T=T, ctx=ctx, ragged=rng.random() < 0.7, d=d, page=page,
                    window=window, sinks=rng.choice([0, rng.randint(1, 200)]), tree=tree)
    T = _log_int(rng, 1, 4096) if op == "append" else _log_int(rng, 2, 64)
    ctx = _log_int(rng, 1, 1000)
    room = (8 * 8 * 4096 * 128) // (Hkv * (T + ctx) * d)
    return dict(op=op, B=_log_int(rng, 1, max(1, min(room, 64))), Hkv=Hkv, T=T, ctx=ctx, ragged=rng.random() < 0.7, d=d,
                page=page)


# ----------------------------------------------------------------------------------------------------------- inputs

def _host(case, seed):
    """What the sizes of a batch are made of, on the host: context lengths, tokens per sequence, pages, trees."""
    rng = np.random.RandomState((int(seed) * 1000003 + 17) % (2**31))
    B, T, ctx, page = case["B"], case["T"], case["ctx"], case["page"]
    h = {}
    h["ctx"] = rng.randint(ctx // 4, ctx + 1, B) if case["ragged"] else np.full(B, ctx)
    if case["op"] == "append":
        h["count"] = rng.randint((T + 1) // 2, T + 1, B) if case["ragged"] else np.full(B, T)
    width = -(-(ctx + T) // page)  # pages of the longest sequence
    used = -(-(h["ctx"] + T) // page)
    pages = B * width + 3  # a pool with room to spare
    order = rng.permutation(pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    h["table"], h["pages"] = table, pages
    if case["op"] == "accept" or case.get("tree"):
        # a random tree per sequence: token u's parent is an earlier token; token 0 is the root
        sees = np.zeros((B, T, T), bool)
        for u in range(T):
            if u:
                parent = rng.randint(max(0, u - 8), u, B)
                sees[:, u, :] = sees[np.arange(B), parent]
            sees[:, u, u] = True
        if T > 4 and case["ragged"]:  # some sequences drafted fewer tokens: the last ones are absent
            for b in range(0, B, 3):
                sees[b, T - 1 - (b % 3):] = False
        h["tree"] = (sees.astype(np.uint64) << np.arange(T, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)
        leaf = rng.randint(0, max(1, T - 4), B)
        path = sees[np.arange(B), leaf]  # the accepted tokens: one branch, in order
        h["taken"] = path.sum(-1)
        h["src"] = np.argsort(~path, axis=-1, kind="stable")
    return h


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=g, dtype=torch.float32).to(torch.bfloat16)

    s = {"case": dict(case)}
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] in ("window", "window_grad"):
        N, H = case["N"], case["H"]

        def heads(n):
            return normal(B, n, N, d) if case["layout"] == "bhnd" else normal(B, N, n, d).transpose(1, 2)

        s["q"], s["k"], s["v"] = heads(H), heads(Hkv), heads(Hkv)
        if case["op"] == "window_grad":
            s["do"] = heads(H)
        return s
    h = _host(case, seed)

    def whole(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)

    s["ctx_len"], s["table"] = whole(h["ctx"]), whole(h["table"])
    s["k_pages"] = normal(h["pages"], Hkv, case["page"], d)
    s["v_pages"] = normal(h["pages"], Hkv, case["page"], d)
    if case["op"] == "attend":
        s["q"] = normal(B, case["T"], case["H"], d).transpose(1, 2)
        s["tree"] = torch.from_numpy(h["tree"]).to(dev) if case["tree"] else None
        return s
    s["k_new"] = normal(B, case["T"], Hkv, d).transpose(1, 2)
    s["v_new"] = normal(B, case["T"], Hkv, d).transpose(1, 2)
    if case["op"] == "append":
        s["count"] = whole(h["count"])
    else:
        s["src"], s["taken"] = whole(h["src"]), whole(h["taken"])
    return s


# ------------------------------------------------------------------------------------------------------ plain forms

def _plain_window(s, grad):
    c = s["case"]
    B, H, Hkv, N, d = (c[x] for x in ("B", "H", "Hkv", "N", "d"))
    G = H // Hkv
    q = s["q"].float().reshape(B, Hkv, G, N, d)
    k, v = s["k"].float().unsqueeze(2), s["v"].float().unsqueeze(2)
    at = torch.arange(N, device=q.device)
    i, j = at[:, None], at[None, :]
    hidden = ~((j <= i) & ((i - j < c["window"]) | (j < c["sinks"])))
    scale = 1.0 / math.sqrt(d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    p = x.div_(total)
    o = torch.matmul(p, v)
    lse = (top + total.log()).reshape(B, H, N)
    out = [o.reshape(B, H, N, d).to(torch.bfloat16), lse]
    if grad:
        do = s["do"].float().reshape(B, Hkv, G, N, d)
        delta = (do * o).sum(-1, keepdim=True)
        dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
        ds = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(scale)
        dq = torch.matmul(ds, k).reshape(B, H, N, d)
        dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
        out += [t.to(torch.bfloat16) for t in (dq, dk, dv)]
    return out


def _plain_attend(s):
    c = s["case"]
    B, H, Hkv, T, d, page = (c[x] for x in ("B", "H", "Hkv", "T", "d", "page"))
    G = H // Hkv
    table, ctx = s["table"].long(), s["ctx_len"].long()
    slots = table.shape[1] * page
    slot = torch.arange(slots, device=table.device)
    pages = table.clamp_min(0)
    k = s["k_pages"][pages].float().transpose(1, 2).reshape(B, Hkv, slots, d)
    v = s["v_pages"][pages].float().transpose(1, 2).reshape(B, Hkv, slots, d)
    token = torch.arange(T, device=table.device)
    if s["tree"] is None:
        sees = (token[:, None] >= token[None, :]).expand(B, T, T)
    else:
        sees = ((s["tree"].unsqueeze(-1) >> token) & 1).bool()
    place = ctx[:, None] + sees.sum(-1) - 1                                     # [B, T] positions of the new tokens
    drafted = (slot[None, :] - ctx[:, None])                                    # [B, slots]
    new = (drafted >= 0) & (drafted < T)
    which = drafted.clamp(0, T - 1)
    where = torch.where(new, place.gather(1, which), slot[None, :])             # position of every slot's token
    seen = torch.where(new[:, None, :], sees.gather(2, which[:, None, :].expand(B, T, slots)), (drafted < 0)[:, None, :])
    near = (place[:, :, None] - where[:, None, :] < c["window"]) | (where < c["sinks"])[:, None, :]
    seen = seen & near & sees.any(-1)[:, :, None]                               # [B, T, slots]
    q = s["q"].float().reshape(B, Hkv, G, T, d)
    x = torch.matmul(q, k.unsqueeze(2).transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v.unsqueeze(2)) / torch.where(total == 0, 1.0, total)
    return [o.reshape(B, H, T, d).to(torch.bfloat16), (top + total.log()).reshape(B, H, T)]


def _plain_append(s):
    c = s["case"]
    B, T, page = c["B"], c["T"], c["page"]
    ctx, token = s["ctx_len"].long(), torch.arange(T, device=s["table"].device)
    slot = ctx[:, None] + token
    if "count" in s:
        b, t = torch.nonzero(token[None, :] < s["count"][:, None], as_tuple=True)
    else:
        b, t = torch.arange(B, device=ctx.device).repeat_interleave(T), token.repeat(B)
    at = slot[b, t]
    to = s["table"].long()[b, at // page]
    s["k_pages"][to, :, at % page] = s["k_new"][b, :, t]
    s["v_pages"][to, :, at % page] = s["v_new"][b, :, t]
    return [s["k_pages"], s["v_pages"]]


def _plain_compact(s):
    page, table = s["case"]["page"], s["table"].long()
    place = torch.arange(s["src"].shape[1], device=table.device)
    b, n = torch.nonzero(place[None, :] < s["taken"][:, None], as_tuple=True)
    ctx = s["ctx_len"].long()[b]
    old, new = ctx + s["src"].long()[b, n], ctx + n
    pools = (s["k_pages"], s["v_pages"])
    rows = [p[table[b, old // page], :, old % page] for p in pools]
    for p, r in zip(pools, rows):
        p[table[b, new // page], :, new % page] = r
    return list(pools)


def _own(s):
    import bf16_numerics_b200 as fa

    c = s["case"]
    if c["op"] == "window":
        o, lse, _ = fa.window_attention_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"], with_stats=False)
        return [o, lse]
    if c["op"] == "window_grad":
        if "workspace" not in s:
            size = fa.fa_window_bwd_workspace_bytes(c["B"], c["H"], c["Hkv"], c["N"], c["d"], c["window"], c["sinks"])
            s["workspace"] = torch.empty(size, device=s["q"].device, dtype=torch.uint8)
        o, lse, stats = fa.window_attention_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"])
        dq, dk, dv, _ = fa.window_attention_backward(s["q"], s["k"], s["v"], o, s["do"], lse, stats.m, c["window"],
                                                     c["sinks"], workspace=s["workspace"])
        return [o, lse, dq, dk, dv]
    if c["op"] == "attend":
        if "workspace" not in s:
            size = fa.fa_cached_workspace_bytes(c["B"], c["H"], c["Hkv"], c["T"], c["d"])
            s["workspace"] = torch.empty(size, device=s["q"].device, dtype=torch.uint8)
        return list(fa.cached_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["ctx_len"], s["tree"],
                                        window=c["window"], sinks=c["sinks"], workspace=s["workspace"]))
    fa.fa_cache_append(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["ctx_len"], s.get("count"))
    if c["op"] == "accept":
        fa.fa_cache_compact(s["k_pages"], s["v_pages"], s["table"], s["ctx_len"], s["src"], s["taken"])
    return [s["k_pages"], s["v_pages"]]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("window", "window_grad"):
        return _plain_window(state, op == "window_grad")
    if op == "attend":
        return _plain_attend(state)
    out = _plain_append(state)
    return _plain_compact(state) if op == "accept" else out


# ------------------------------------------------------------------------------------------------------- what it costs

def _window_pairs(N, window, sinks):
    """Visible (query, key) pairs of one head."""
    i = np.arange(N, dtype=np.int64)
    first = np.maximum(0, i - window + 1)
    return int((i + 1 - first + np.minimum(sinks, first)).sum())


def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    if case["op"] in ("window", "window_grad"):
        H, N = case["H"], case["N"]
        pairs = B * H * _window_pairs(N, case["window"], case["sinks"])
        row, kv = B * H * N, B * Hkv * N
        if case["op"] == "window":
            return {"bytes": 2 * d * (2 * row + 2 * kv) + 4 * row, "flops": 4 * d * pairs}
        return {"bytes": 2 * d * (4 * row + 4 * kv) + 4 * row, "flops": 14 * d * pairs}
    h = _host(case, 0)
    if case["op"] == "attend":
        T, H = case["T"], case["H"]
        keys = pairs = 0
        for n in (int(x) for x in h["ctx"]):
            first = max(0, n - case["window"] + 1)
            seen = n - first + min(case["sinks"], first) + T
            keys += seen
            pairs += seen * T
        return {"bytes": 4 * d * Hkv * keys + 4 * d * B * H * T + 4 * B * H * T, "flops": 4 * d * H * pairs}
    if case["op"] == "append":
        return {"bytes": 8 * d * Hkv * int(h["count"].sum()), "flops": 0}
    return {"bytes": 8 * d * Hkv * (B * case["T"] + int(h["taken"].sum())), "flops": 0}


# ------------------------------------------------------------------------------------------------------ in 64 bits

def _exact_window(s, grad):
    c = s["case"]
    B, H, Hkv, N, d = (c[x] for x in ("B", "H", "Hkv", "N", "d"))
    G = H // Hkv
    j = torch.arange(N, device=s["q"].device)
    dist = j[:, None] - j[None, :]
    keep = (dist >= 0) & ((dist < c["window"]) | (j[None, :] < c["sinks"]))
    like = dict(device=s["q"].device, dtype=torch.float64)
    o, lse = torch.empty(B, H, N, d, **like), torch.empty(B, H, N, **like)
    dq, dk, dv = torch.empty(B, H, N, d, **like), torch.zeros(B, Hkv, N, d, **like), torch.zeros(B, Hkv, N, d, **like)
    for b in range(B):
        for h in range(H):
            leaf = [s["q"][b, h], s["k"][b, h // G], s["v"][b, h // G]]
            q, k, v = (t.detach().double().requires_grad_(grad) for t in leaf)
            with torch.set_grad_enabled(grad):
                x = torch.where(keep, q @ k.t() / math.sqrt(d), -math.inf)
                lse[b, h] = torch.logsumexp(x.detach(), -1)
                y = torch.softmax(x, -1) @ v
            o[b, h] = y.detach()
            if grad:
                gq, gk, gv = torch.autograd.grad(y, (q, k, v), s["do"][b, h].double())
                dq[b, h] = gq
                dk[b, h // G] += gk
                dv[b, h // G] += gv
    return [o, lse] + ([dq, dk, dv] if grad else [])


def _exact_attend(s, h):
    c = s["case"]
    B, H, Hkv, T, d, page = (c[x] for x in ("B", "H", "Hkv", "T", "d", "page"))
    G = H // Hkv
    dev = s["q"].device
    o = torch.zeros(B, H, T, d, device=dev, dtype=torch.float64)
    lse = torch.full((B, H, T), -math.inf, device=dev, dtype=torch.float64)
    words = h["tree"].view(np.uint64) if c["tree"] else None
    for b in range(B):
        n = int(h["ctx"][b])
        seen = np.zeros((T, n + T), bool)
        bits = np.tril(np.ones((T, T), bool))
        if words is not None:
            bits = np.array([[(int(words[b, t]) >> u) & 1 for u in range(T)] for t in range(T)], bool)
        stands = np.concatenate([np.arange(n), n + bits.sum(1) - 1])
        for t in range(T):
            if bits[t].any():
                seen[t, :n] = True
                seen[t, n:] = bits[t]
                seen[t] &= (stands[n + t] - stands < c["window"]) | (stands < c["sinks"])
        slots = np.arange(n + T)
        of = torch.from_numpy(h["table"][b][slots // page]).to(dev), torch.from_numpy(slots % page).to(dev)
        live = torch.from_numpy(seen.any(1)).to(dev)
        hide = torch.from_numpy(~seen).to(dev)
        for kv in range(Hkv):
            k, v = (s[x][of[0], kv, of[1]].double() for x in ("k_pages", "v_pages"))
            x = (s["q"][b, kv * G:(kv + 1) * G].double() @ k.t() / math.sqrt(d)).masked_fill(hide, -math.inf)
            lse[b, kv * G:(kv + 1) * G] = torch.logsumexp(x, -1)
            y = torch.softmax(x, -1) @ v
            o[b, kv * G:(kv + 1) * G] = torch.where(live[None, :, None], y, 0.0)
    return [o, lse]


def _exact_pools(s, h):
    c = s["case"]
    page = c["page"]
    pools = []
    for pool, new in (("k_pages", "k_new"), ("v_pages", "v_new")):
        x, rows = s[pool].double(), s[new].double()
        for b in range(c["B"]):
            n = int(h["ctx"][b])
            put = np.arange(int(h["count"][b]) if c["op"] == "append" else c["T"])
            to = torch.from_numpy(h["table"][b][(n + put) // page]).to(x.device)
            x[to, :, torch.from_numpy((n + put) % page).to(x.device)] = rows[b, :, :len(put)].transpose(0, 1)
            if c["op"] == "accept":
                took = h["src"][b][:int(h["taken"][b])]
                for i, t in enumerate(took):
                    x[int(h["table"][b][(n + i) // page]), :, (n + i) % page] = rows[b, :, int(t)]
        pools.append(x)
    return pools


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("window", "window_grad"):
        return _exact_window(s, case["op"] == "window_grad")
    h = _host(case, seed)
    return _exact_attend(s, h) if case["op"] == "attend" else _exact_pools(s, h)

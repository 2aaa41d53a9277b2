"""The operators between the encoder's ids and the decoder's text, in plain form and as this package runs them:
placing requests in a paged key/value cache (`kv_plan`), norm + rotation + store of their rows (`KVCache.append`)
and attention of new or drafted tokens over the cache (`KVCache.attend`)."""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one decode step of an ordinary batch: one token a request, few new blocks (pure latency)
        dict(name="plan decode 64", op="plan", requests=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=8000,
             block=16, tree=False, shape=1),
        # one verification step: a drafted tree a request, positions by depth, ancestor masks
        dict(name="plan trees 256", op="plan", requests=256, new_lo=1, new_hi=64, ctx_lo=0, ctx_hi=8000,
             block=32, tree=True, shape=2),
        # admission of a serving batch: the prompts of 4,096 requests placed at once
        dict(name="plan prompts 4096", op="plan", requests=4096, new_lo=1, new_hi=8192, ctx_lo=0, ctx_hi=0,
             block=64, tree=False, shape=3),
        # one decode step's rows: latency
        dict(name="append 64 rows", op="append", rows=64, q_heads=32, kv_heads=8, dim=128, rot=128, pairs="halves",
             block=16, norm=True, type="bf16", skip=0),
        # odd sizes: partial rotation of neighbouring pairs, 5 query heads a key head, padding rows without a slot
        dict(name="append 3001 odd rows", op="append", rows=3001, q_heads=20, kv_heads=4, dim=96, rot=32,
             pairs="neighbours", block=32, norm=True, type="f16", skip=7),
        # a prefill step of a full batch
        dict(name="append 32768 rows", op="append", rows=32768, q_heads=32, kv_heads=8, dim=128, rot=128, pairs="halves",
             block=64, norm=True, type="bf16", skip=0),
        # a single chat turn: one token of one request over a short cache (latency)
        dict(name="attend 1 x 1 over 200", op="attend", requests=1, new_lo=1, new_hi=1, ctx_lo=199, ctx_hi=199, q_heads=32,
             kv_heads=8, dim=128, block=16, tree=False, type="bf16", shape=4),
        # one decode step of a large batch: the cache read once (bandwidth)
        dict(name="attend 128 x 1 over 6k", op="attend", requests=128, new_lo=1, new_hi=1, ctx_lo=2000, ctx_hi=10000, q_heads=32,
             kv_heads=8, dim=128, block=64, tree=False, type="bf16", shape=5),
        # drafted trees of up to 24 tokens for a batch of ragged requests, 4 query heads a key head
        dict(name="attend 32 trees over 8k", op="attend", requests=32, new_lo=3, new_hi=24, ctx_lo=0, ctx_hi=16000, q_heads=32,
             kv_heads=8, dim=128, block=16, tree=True, type="bf16", shape=6),
        # a wide tree of one long request: matrix products over 512 rows a key head
        dict(name="attend 64 tree over 131k", op="attend", requests=1, new_lo=64, new_hi=64, ctx_lo=130999, ctx_hi=130999, q_heads=64,
             kv_heads=8, dim=128, block=128, tree=True, type="bf16", shape=7),
        # no shared heads, small heads, fp16
        dict(name="attend 24 trees f16 d64", op="attend", requests=24, new_lo=1, new_hi=17, ctx_lo=5, ctx_hi=3000, q_heads=12,
             kv_heads=12, dim=64, block=32, tree=True, type="f16", shape=8),
        # a chunk of a long prompt after what is cached already
        dict(name="attend 3 x 700 over 9k", op="attend", requests=3, new_lo=500, new_hi=900, ctx_lo=4000, ctx_hi=14000, q_heads=32,
             kv_heads=8, dim=128, block=64, tree=False, type="bf16", shape=9),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend"])
    shape = rng.randrange(1 << 30)
    if op == "plan":
        tree = rng.random() < 0.5
        lo, hi = (1, _log(rng, 1, 64)) if tree else (rng.choice([0, 1]), _log(rng, 1, 8192))
        return dict(op=op, requests=_log(rng, 1, 4096), new_lo=lo, new_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 20000),
                    block=rng.choice([16, 32, 64, 128]), tree=tree, shape=shape)
    if op == "append":
        dim = rng.choice([64, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        most = 32768 * 48 * 128 // ((group + 2) * kv * dim)
        return dict(op=op, rows=_log(rng, 1, min(32768, most)), q_heads=kv * group, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), pairs=rng.choice(["halves", "neighbours"]),
                    block=rng.choice([16, 32, 64, 128]), norm=rng.random() < 0.8, type=rng.choice(list(TYPES)),
                    skip=rng.choice([0, 0, 5]))
    kind = rng.choice(["one", "tree", "tree", "chain"])
    kv = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    most = {"one": 1, "tree": _log(rng, 2, 64), "chain": _log(rng, 2, 900)}[kind]
    case = dict(op=op, requests=_log(rng, 1, 256), new_lo=1, new_hi=most, ctx_lo=0, ctx_hi=_log(rng, 16, 60000),
                q_heads=kv * group, kv_heads=kv, dim=rng.choice([64, 128]), block=rng.choice([16, 32, 64, 128]), tree=kind == "tree",
                type=rng.choice(list(TYPES)), shape=shape)
    while work(case)["bytes"] > 2.5e9 or work(case)["flops"] > 2.5e11:
        case["requests"] = (case["requests"] + 1) // 2
        case["ctx_hi"] = case["ctx_hi"] * 2 // 3
    return case


def _lengths(case):
    """(new tokens, cached tokens) of every request: ragged, and a matter of the case, not of the seed."""
    rng = random.Random(case["shape"])
    a, b, c, d = case["new_lo"], case["new_hi"], case["ctx_lo"], case["ctx_hi"]
    new, ctx = [], []
    for _ in range(case["requests"]):
        n = rng.randint(a, b)
        if b > 64:  # prompts: many short ones, a few long
            n = max(a, min(b, int(rng.lognormvariate(math.log(max(1, b / 12)), 1.2)))) if a <= 1 else n
        new.append(n)
        ctx.append(rng.randint(c, d))
    if not sum(new):
        new[0] = 1
    return new, ctx


def _parents(new, gen, device):
    """Drafted trees: every token hangs on one of the few tokens before it, the first ones on the context (-1)."""
    pos = torch.cat([torch.arange(n) for n in new]).to(device)
    back = (torch.rand(pos.numel(), generator=gen, device=device) ** 2 * 6).long()
    return torch.clamp(pos - 1 - back, min=-1).int()


def _ancestors(parents, off, req):
    """(mask, depth): bit j of a token's mask says that drafted token j of its request is the token or above it."""
    local = torch.arange(parents.numel(), device=parents.device) - off[req]
    mask = torch.ones_like(local) << local
    depth = (parents >= 0).long()
    up = torch.where(parents >= 0, off[req] + parents.long(), torch.full_like(local, -1))
    for _ in range(6):  # pointers double: 2^6 covers trees of 64
        has, at = up >= 0, up.clamp(min=0)
        mask = torch.where(has, mask | mask[at], mask)
        depth = torch.where(has, depth + depth[at], depth)
        up = torch.where(has, up[at], up)
    return mask, depth


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        import byte_level_bpe_gb300 as tk
        state["tk"] = tk
        if case["op"] != "plan":
            state["cache"] = tk.KVCache(state["k"], state["v"])
        if case["op"] == "attend":
            state["ws"] = tk.KVWorkspace()
    return state


def _inputs(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] == "append":
        return _rows(case, gen, dev)
    new, ctx = _lengths(case)
    off = torch.zeros(len(new) + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(torch.tensor(new), 0)
    state = {"case": case, "new": new, "ctx": ctx, "tokens": sum(new), "off": off.to(dev),
             "context": torch.tensor(ctx, dtype=torch.int32, device=dev)}
    state.update((_requests if case["op"] == "plan" else _cached)(case, state, gen, dev))
    return state


def _requests(case, s, gen, dev):
    bs = case["block"]
    wide = max(-(-(c + n) // bs) for c, n in zip(s["ctx"], s["new"])) + 3
    have = [-(-c // bs) for c in s["ctx"]]
    need = sum(-(-(c + n) // bs) - h for c, n, h in zip(s["ctx"], s["new"], have))
    ids = torch.randperm(need + 8 + sum(have), generator=gen, device=dev).int()
    table = torch.full((len(have), wide), -1, dtype=torch.int32, device=dev)
    held = torch.arange(wide, device=dev)[None] < torch.tensor(have, device=dev)[:, None]
    table[held] = ids[need + 8:]
    parents = _parents(s["new"], gen, dev) if case["tree"] else None
    return {"table": table, "free": ids[:need + 8].contiguous(), "parents": parents}


def _rows(case, gen, dev):
    t, d, bs = case["rows"], case["dim"], case["block"]
    heads = case["q_heads"] + 2 * case["kv_heads"]
    blocks = -(-t // bs) + 2
    dt = TYPES[case["type"]]
    # projections: channels of different sizes, a few large ones
    size = torch.exp(torch.randn(heads * d, generator=gen, device=dev) * 0.7)
    qkv = (torch.randn(t, heads * d, generator=gen, device=dev) * size).to(dt)
    pool = (torch.randn(2, blocks, case["kv_heads"], bs, d, generator=gen, device=dev)).to(dt)
    most = 40000
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
    angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * freq
    # requests' rows are runs of neighbouring slots: blocks in random order, tokens in order within one
    order = torch.randperm(blocks, generator=gen, device=dev)
    slots = (order[:, None] * bs + torch.arange(bs, device=dev)).reshape(-1)[:t].contiguous()
    if case["skip"]:
        slots[::case["skip"]] = -1
    gains = 1 + 0.2 * torch.randn(2, d, generator=gen, device=dev)
    return {"case": case, "qkv": qkv, "k": pool[0], "v": pool[1], "slots": slots,
            "positions": torch.randint(0, most, (t,), generator=gen, device=dev).int(),
            "rope": torch.stack([angle.cos(), angle.sin()], -1).float().contiguous(),
            "q_gain": gains[0].contiguous() if case["norm"] else None, "k_gain": gains[1].contiguous() if case["norm"] else None}


def _cached(case, s, gen, dev):
    bs, d, dt = case["block"], case["dim"], TYPES[case["type"]]
    total = [c + n for c, n in zip(s["ctx"], s["new"])]
    used = [-(-n // bs) for n in total]
    blocks = sum(used) + 2
    pool = torch.empty(2, blocks, case["kv_heads"], bs, d, dtype=dt, device=dev)
    pool.normal_(generator=gen)
    table = torch.zeros(len(used), max(used) + 1, dtype=torch.int32, device=dev)
    held = torch.arange(table.shape[1], device=dev)[None] < torch.tensor(used, device=dev)[:, None]
    table[held] = torch.randperm(blocks, generator=gen, device=dev)[:sum(used)].int()
    # queries a little longer than keys: some rows attend to few places, some to many
    q = torch.randn(s["tokens"], case["q_heads"], d, generator=gen, device=dev)
    q = (q * torch.exp(0.5 * torch.randn(s["tokens"], case["q_heads"], 1, generator=gen, device=dev))).to(dt)
    masks = None
    if case["tree"]:
        req = torch.repeat_interleave(torch.arange(len(used), device=dev), torch.tensor(s["new"], device=dev))
        masks = _ancestors(_parents(s["new"], gen, dev), s["off"], req)[0]
    return {"k": pool[0], "v": pool[1], "table": table, "q": q, "masks": masks, "total": total,
            "lengths": torch.tensor(total, dtype=torch.int32, device=dev)}


def run(state):
    return {"plan": _run_plan, "append": _run_append, "attend": _run_attend}[state["case"]["op"]](state)


def _run_plan(s):
    if own:
        p = s["tk"].kv_plan(s["off"], s["context"], s["table"], s["free"], s["case"]["block"], s["tokens"], parents=s["parents"])
        return {"table": s["table"], "positions": p.positions, "slots": p.slots, "requests": p.requests,
                "lengths": p.lengths, "info": p.info, "masks": p.masks}
    bs, off, table, free = s["case"]["block"], s["off"], s["table"], s["free"]
    ctx = s["context"].long()
    n = off[1:] - off[:-1]
    have, want = (ctx + bs - 1) // bs, (ctx + n + bs - 1) // bs
    good = (n >= 0) & (ctx >= 0) & (want <= table.shape[1])
    if s["parents"] is not None:
        good = good & (n <= 64)
    need = torch.where(good, want - have, torch.zeros_like(want))
    end = torch.cumsum(need, 0)
    fits = good & ((need == 0) | (end <= free.numel()))
    j = torch.arange(table.shape[1], device=table.device)[None]
    fresh = fits[:, None] & (j >= have[:, None]) & (j < want[:, None])
    at = (end - need)[:, None] + j - have[:, None]
    table.copy_(torch.where(fresh, free[at.clamp(0, free.numel() - 1)], table))
    t = torch.arange(s["tokens"], device=table.device)
    req = torch.searchsorted(off[1:].contiguous(), t, right=True)
    i = t - off[req]
    spot = ctx[req] + i
    slots = torch.where(fits[req], table[req, (spot // bs).clamp(max=table.shape[1] - 1)].long() * bs + spot % bs, torch.full_like(t, -1))
    masks, positions = None, spot
    if s["parents"] is not None:
        masks, depth = _ancestors(s["parents"], off, req)
        positions = ctx[req] + depth
    bad = ~good
    short = good & ~fits
    code = torch.where(bad, -9, torch.where(short, -4, 0))
    first = torch.argmax((code != 0).int())
    which = torch.where(code[first] != 0, first, torch.full_like(first, -1))
    info = torch.stack([torch.where(fits, need, torch.zeros_like(need)).sum(), need.sum(), code[first], which])
    return {"table": table, "positions": positions.int(), "slots": slots, "requests": req.int(),
            "lengths": torch.where(fits, ctx + n, ctx).int(), "info": info, "masks": masks}


def _run_append(s):
    c = s["case"]
    if own:
        q = s["cache"].append(s["qkv"], s["positions"], s["slots"], c["q_heads"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                              rope=s["rope"], eps=1e-6, neighbours=c["pairs"] == "neighbours")
        return {"q": q, "k": s["k"], "v": s["v"]}
    t, d, hq, hk = c["rows"], c["dim"], c["q_heads"], c["kv_heads"]
    x = s["qkv"].float().view(t, hq + 2 * hk, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    cos, sin = s["rope"][s["positions"].long()].unbind(-1)
    out = []
    for y, gain in ((q, s["q_gain"]), (k, s["k_gain"])):
        if gain is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * gain
        turn, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        if c["pairs"] == "halves":
            a, b = turn[..., :c["rot"] // 2], turn[..., c["rot"] // 2:]
        else:
            a, b = turn[..., 0::2], turn[..., 1::2]
        a, b = a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]
        turn = torch.cat([a, b], -1) if c["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
        out.append(torch.cat([turn, rest], -1).to(s["qkv"].dtype))
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    block, spot = at // c["block"], at % c["block"]
    s["k"][block, :, spot] = out[1][kept]
    s["v"][block, :, spot] = s["qkv"].view(t, hq + 2 * hk, d)[:, hq + hk:][kept]
    return {"q": out[0], "k": s["k"], "v": s["v"]}


def _run_attend(s):
    c = s["case"]
    scale = c["dim"] ** -0.5
    if own:
        return s["cache"].attend(s["q"], s["off"], s["lengths"], s["table"], s["ws"], masks=s["masks"], scale=scale,
                                 max_new=c["new_hi"])
    hk, d = c["kv_heads"], c["dim"]
    group = c["q_heads"] // hk
    out = torch.empty_like(s["q"])
    at = 0
    for r, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        if not n:
            continue
        rows = s["table"][r, :-(-(ctx + n) // c["block"])].long()
        k, v = (x[rows].transpose(0, 1).reshape(hk, -1, d)[:, :ctx + n].float() for x in (s["k"], s["v"]))
        q = s["q"][at:at + n].float().view(n, hk, group, d).permute(1, 2, 0, 3).reshape(hk, group * n, d)
        w = (q @ k.transpose(1, 2)).mul_(scale).view(hk, group, n, ctx + n)
        j = torch.arange(n, device=q.device)
        if s["masks"] is None:
            seen = j[None] <= j[:, None]
        else:
            seen = (s["masks"][at:at + n, None] >> j[None]) & 1 != 0
        w[..., ctx:].masked_fill_(~seen, -math.inf)
        top = w.amax(-1, keepdim=True).clamp(min=-1e30)
        w = w.sub_(top).exp_()
        total = w.sum(-1, keepdim=True)
        o = (w.view(hk, group * n, -1) @ v).view(hk, group, n, d) / torch.where(total > 0, total, torch.ones_like(total))
        out[at:at + n] = o.permute(2, 0, 1, 3).reshape(n, -1, d).to(out.dtype)
        at += n
    return out


def work(case):
    if case["op"] == "append":
        t, d = case["rows"], case["dim"]
        heads = case["q_heads"] + 2 * case["kv_heads"]
        return {"bytes": t * (heads * d * 4 + 12 + case["rot"] * 4), "flops": t * (case["q_heads"] + case["kv_heads"]) * (4 * d + 3 * case["rot"])}
    new, ctx = _lengths(case)
    t, r = sum(new), len(new)
    if case["op"] == "plan":
        bs = case["block"]
        need = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, new))
        return {"bytes": 8 * (r + 1) + 8 * r + 16 * t + 8 * need + (12 * t if case["tree"] else 0), "flops": 10 * t}
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    pairs = sum(n * c + (n if case["tree"] else n * (n + 1) // 2) for n, c in zip(new, ctx))
    keys = sum(n + c for n, c in zip(new, ctx))
    return {"bytes": keys * hk * d * 4 + t * hq * d * 4 + 4 * keys // case["block"], "flops": 4 * d * hq * pairs}


# The definitions once more in 64 bits, written on their own: token by token and head by head.

def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers: the plain form is the definition
    s = _inputs(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attend)(case, s)


def _exact_append(c, s):
    hq, hk, d, rot = c["q_heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qkv"].double().reshape(-1, hq + 2 * hk, d)
    z = torch.view_as_complex(s["rope"].double())[s["positions"].long()]  # cos + i sin
    k, v = s["k"].double(), s["v"].double()
    q_out = torch.empty(x.shape[0], hq, d, dtype=torch.float64, device=x.device)
    kept = (s["slots"] >= 0).nonzero().flatten()
    blocks, spots = s["slots"][kept] // c["block"], s["slots"][kept] % c["block"]
    half = rot // 2
    first = torch.arange(half, device=x.device) * (1 if c["pairs"] == "halves" else 2)
    second = first + (half if c["pairs"] == "halves" else 1)
    for h in range(hq + hk):
        y = x[:, h].clone()
        gain = s["q_gain"] if h < hq else s["k_gain"]
        if gain is not None:
            y *= (y.pow(2).sum(1, keepdim=True) / d + 1e-6).rsqrt() * gain.double()
        turned = torch.complex(y[:, first], y[:, second]) * z
        y[:, first], y[:, second] = turned.real, turned.imag
        if h < hq:
            q_out[:, h] = y
        else:
            k[blocks, h - hq, spots] = y[kept]
    for h in range(hk):
        v[blocks, h, spots] = x[kept, hq + hk + h]
    return {"q": q_out, "k": k, "v": v}


def _exact_attend(c, s):
    hq, hk, d, bs = c["q_heads"], c["kv_heads"], c["dim"], c["block"]
    out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device=s["q"].device)
    start = 0
    for r, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        place = torch.arange(ctx + n, device=out.device)
        rows, spots = s["table"][r].long()[place // bs], place % bs
        i, j = torch.arange(n, device=out.device)[:, None], place[None] - ctx
        if s["masks"] is None:
            hidden = j > i
        else:
            hidden = (j >= 0) & ((s["masks"][start:start + n, None] >> j.clamp(min=0)) & 1 == 0)
        for g in range(hk):
            k, v = s["k"][rows, g, spots].double(), s["v"][rows, g, spots].double()
            for h in range(g * hq // hk, (g + 1) * hq // hk):
                logit = torch.einsum("nd,jd->nj", s["q"][start:start + n, h].double(), k) / math.sqrt(d)
                logit = logit.masked_fill(hidden, -math.inf)
                weight = torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True))
                out[start:start + n, h] = weight @ v
        start += n
    return out

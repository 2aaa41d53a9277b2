"""The paged key/value cache in 8 bits and its windowed attention, in plain form and as this package runs them:
storing new rows with a scale for each block and head (`KVCache.append` of a cache of 8-bit blocks), attention over
such a cache (`KVCache.attend`), and attention with a sliding window and first tokens that stay visible
(`KVCache.attend` with `window` and `sinks`), over 16-bit and 8-bit blocks."""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
LARGEST = 448.0       # of e4m3
LEAST_SCALE = 2.0 ** -100  # of a block of zeros


def listed():
    return [
        # one decode step's rows into a large pool: each in a block of its own that holds older rows (latency)
        dict(name="store 64 rows", op="store", requests=64, new_lo=1, new_hi=1, q_heads=32, kv_heads=8, dim=128, rot=128,
             pairs="halves", block=16, pool=2048, norm=True, type="bf16", skip=0, shape=1),
        # odd sizes: partial rotation of neighbouring pairs, 5 query heads a key head, requests that found no place
        dict(name="store 41 odd chunks", op="store", requests=41, new_lo=1, new_hi=151, q_heads=20, kv_heads=4, dim=96, rot=32,
             pairs="neighbours", block=32, pool=300, norm=True, type="f16", skip=7, shape=2),
        # a prefill step of a full batch
        dict(name="store 16 x 2k rows", op="store", requests=16, new_lo=1100, new_hi=2900, q_heads=32, kv_heads=8, dim=128, rot=128,
             pairs="halves", block=64, pool=600, norm=True, type="bf16", skip=0, shape=3),
        # a single chat turn: one token of one request over a short cache (latency)
        dict(name="read 1 x 1 over 200", op="read", bits=8, requests=1, new_lo=1, new_hi=1, ctx_lo=199, ctx_hi=199, q_heads=32,
             kv_heads=8, dim=128, block=16, tree=False, type="bf16", window=0, sinks=0, shape=4),
        # one decode step of a large batch: the cache read once (bandwidth)
        dict(name="read 128 x 1 over 6k", op="read", bits=8, requests=128, new_lo=1, new_hi=1, ctx_lo=2000, ctx_hi=10000, q_heads=32,
             kv_heads=8, dim=128, block=64, tree=False, type="bf16", window=0, sinks=0, shape=5),
        # drafted trees of up to 24 tokens for a batch of ragged requests, no shared heads, small ones, fp16
        dict(name="read 24 trees f16 d64", op="read", bits=8, requests=24, new_lo=1, new_hi=17, ctx_lo=5, ctx_hi=3000, q_heads=12,
             kv_heads=12, dim=64, block=32, tree=True, type="f16", window=0, sinks=0, shape=6),
        # a wide tree of one long request: matrix products over 512 rows a key head
        dict(name="read 64 tree over 131k", op="read", bits=8, requests=1, new_lo=64, new_hi=64, ctx_lo=130999, ctx_hi=130999, q_heads=64,
             kv_heads=8, dim=128, block=128, tree=True, type="bf16", window=0, sinks=0, shape=7),
        # chunks of long prompts after what is cached already
        dict(name="read 3 x 700 over 9k", op="read", bits=8, requests=3, new_lo=500, new_hi=900, ctx_lo=4000, ctx_hi=14000, q_heads=32,
             kv_heads=8, dim=128, block=64, tree=False, type="bf16", window=0, sinks=0, shape=8),
        # one decode step of a layer with a window, 16-bit cache (bandwidth)
        dict(name="window 64 x 1 over 14k", op="read", bits=16, requests=64, new_lo=1, new_hi=1, ctx_lo=5000, ctx_hi=23000, q_heads=32,
             kv_heads=8, dim=128, block=64, tree=False, type="bf16", window=4096, sinks=4, shape=9),
        # one decode step of a few requests with a short window: latency
        dict(name="window 5 x 1 f16 d64", op="read", bits=16, requests=5, new_lo=1, new_hi=1, ctx_lo=3, ctx_hi=2000, q_heads=14,
             kv_heads=2, dim=64, block=16, tree=False, type="f16", window=128, sinks=4, shape=10),
        # chunks of long prompts in a layer with a window, 16-bit cache (matrix products)
        dict(name="window 4 x 2k over 6k", op="read", bits=16, requests=4, new_lo=1500, new_hi=2500, ctx_lo=3000, ctx_hi=9000, q_heads=32,
             kv_heads=8, dim=128, block=64, tree=False, type="bf16", window=1024, sinks=16, shape=11),
        # drafted trees over a windowed cache in 8 bits
        dict(name="window 32 trees over 8k", op="read", bits=8, requests=32, new_lo=3, new_hi=24, ctx_lo=0, ctx_hi=16000, q_heads=32,
             kv_heads=8, dim=128, block=16, tree=True, type="bf16", window=2048, sinks=4, shape=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    shape = rng.randrange(1 << 30)
    if rng.random() < 0.25:
        dim = rng.choice([64, 96, 128, 256])
        kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
        block = rng.choice([16, 32, 64, 128])
        most = min(32768, 32768 * 48 * 128 // ((group + 2) * kv * dim))
        requests = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, most // requests))
        return dict(op="store", requests=requests, new_lo=1, new_hi=new, q_heads=kv * group, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), pairs=rng.choice(["halves", "neighbours"]), block=block,
                    pool=requests * (new // block + 2), norm=rng.random() < 0.8, type=rng.choice(list(TYPES)),
                    skip=rng.choice([0, 0, 5]), shape=shape)
    kind = rng.choice(["one", "tree", "tree", "chain"])
    kv, group = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 4, 5, 7, 8])
    most = {"one": 1, "tree": _log(rng, 2, 64), "chain": _log(rng, 2, 900)}[kind]
    windowed = rng.random() < 0.5
    case = dict(op="read", bits=16 if windowed and rng.random() < 0.6 else 8, requests=_log(rng, 1, 256), new_lo=1, new_hi=most,
                ctx_lo=0, ctx_hi=_log(rng, 16, 60000), q_heads=kv * group, kv_heads=kv, dim=rng.choice([64, 128]),
                block=rng.choice([16, 32, 64, 128]), tree=kind == "tree", type=rng.choice(list(TYPES)),
                window=_log(rng, 64, 8192) if windowed else 0, sinks=rng.choice([0, 1, 4, 64]) if windowed else 0, shape=shape)
    while work({**case, "window": 0})["bytes"] > 2.5e9 or work({**case, "window": 0})["flops"] > 2.5e11:
        case["requests"] = (case["requests"] + 1) // 2
        case["ctx_hi"] = case["ctx_hi"] * 2 // 3
    return case


def _lengths(case):
    """(new tokens, cached tokens) of every request: ragged, and a matter of the case, not of the seed."""
    rng = random.Random(case["shape"])
    pairs = [(rng.randint(case["new_lo"], case["new_hi"]), rng.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 4 * case["block"])))
             for _ in range(case["requests"])]
    return [n for n, _ in pairs], [c for _, c in pairs]


def _in_8_bits(x):
    """[..., tokens, dim] -> e4m3 values and the scale of each block: the least power of two that the largest fits."""
    mantissa, exponent = torch.frexp(x.abs().amax((-2, -1)).float() / LARGEST)
    scale = torch.ldexp(torch.ones_like(mantissa), exponent - (mantissa == 0.5).int()).clamp(min=LEAST_SCALE)
    return (x / scale[..., None, None]).to(E4M3), scale


def _pool(blocks, case, gen, dev):
    """Keys or values of a pool of blocks; their sizes differ from block to block and from head to head."""
    shape = (blocks, case["kv_heads"], case["block"], case["dim"])
    if case.get("bits", 8) == 16:
        return torch.empty(shape, dtype=TYPES[case["type"]], device=dev).normal_(generator=gen), None
    x, scale = torch.empty(shape, dtype=E4M3, device=dev), torch.empty(shape[:2], device=dev)
    for part in range(0, blocks, 4096):
        here = slice(part, min(blocks, part + 4096))
        size = torch.exp(0.4 * torch.randn(scale[here].shape, generator=gen, device=dev))
        x[here], scale[here] = _in_8_bits(torch.randn(x[here].shape, generator=gen, device=dev) * size[..., None, None])
    return x, scale


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        import byte_level_bpe_gb300 as tk
        scales = (state["k_scale"], state["v_scale"], TYPES[case["type"]]) if state["k_scale"] is not None else ()
        state["cache"] = tk.KVCache(state["k"], state["v"], *scales)
        if case["op"] == "read":
            state["ws"] = tk.KVWorkspace()
    return state


def _inputs(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    return (_rows if case["op"] == "store" else _cached)(case, gen, dev)


def _rows(case, gen, dev):
    """The projections of new tokens and their slots: each request goes on behind its older rows."""
    d, bs, dt = case["dim"], case["block"], TYPES[case["type"]]
    heads = case["q_heads"] + 2 * case["kv_heads"]
    new, ctx = _lengths(case)
    new_t, begin = torch.tensor(new, device=dev), torch.tensor([c % bs for c in ctx], device=dev)
    t = sum(new)
    req = torch.repeat_interleave(torch.arange(len(new), device=dev), new_t, output_size=t)
    first = torch.cumsum(new_t, 0) - new_t
    place = begin[req] + torch.arange(t, device=dev) - first[req]
    used = (begin + new_t + bs - 1) // bs
    blocks = max(case["pool"], int(used.sum()))
    order = torch.randperm(blocks, generator=gen, device=dev)
    slots = order[(torch.cumsum(used, 0) - used)[req] + place // bs] * bs + place % bs
    if case["skip"]:  # requests that found no place
        slots = torch.where(req % case["skip"] == case["skip"] - 1, torch.full_like(slots, -1), slots)
    # channels of different sizes, a few large ones; tokens too
    size = torch.exp(0.7 * torch.randn(heads * d, generator=gen, device=dev))
    loud = torch.exp(0.5 * torch.randn(t, 1, generator=gen, device=dev))
    qkv = (torch.randn(t, heads * d, generator=gen, device=dev) * size * loud).to(dt)
    (k, k_scale), (v, v_scale) = _pool(blocks, case, gen, dev), _pool(blocks, case, gen, dev)
    most = 40000
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
    angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * freq
    gains = 1 + 0.2 * torch.randn(2, d, generator=gen, device=dev)
    return {"case": case, "qkv": qkv, "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "slots": slots.contiguous(),
            "positions": torch.randint(0, most, (t,), generator=gen, device=dev).int(),
            "rope": torch.stack([angle.cos(), angle.sin()], -1).float().contiguous(),
            "q_gain": gains[0].contiguous() if case["norm"] else None, "k_gain": gains[1].contiguous() if case["norm"] else None}


def _trees(new, gen, dev):
    """Ancestor masks of drafted trees: every token hangs on one of the few before it or on the context."""
    rows = torch.zeros(len(new), max(new), dtype=torch.int64, device=dev)
    back = (torch.rand(rows.shape, generator=gen, device=dev) ** 2 * 6).long()
    for i in range(rows.shape[1]):
        up = i - 1 - back[:, i]
        rows[:, i] = torch.where(up >= 0, rows.gather(1, up.clamp(min=0)[:, None])[:, 0], 0) | 1 << i
    return rows


def _cached(case, gen, dev):
    bs, d, dt = case["block"], case["dim"], TYPES[case["type"]]
    new, ctx = _lengths(case)
    total, t = [c + n for c, n in zip(ctx, new)], sum(new)
    used = [-(-n // bs) for n in total]
    blocks = sum(used) + 2
    (k, k_scale), (v, v_scale) = _pool(blocks, case, gen, dev), _pool(blocks, case, gen, dev)
    table = torch.zeros(len(used), max(used) + 1, dtype=torch.int32, device=dev)
    held = torch.arange(table.shape[1], device=dev)[None] < torch.tensor(used, device=dev)[:, None]
    table[held] = torch.randperm(blocks, generator=gen, device=dev)[:sum(used)].int()
    # queries a little longer than keys: some rows attend to few places, some to many
    q = torch.randn(t, case["q_heads"], d, generator=gen, device=dev)
    q = (q * torch.exp(0.5 * torch.randn(t, case["q_heads"], 1, generator=gen, device=dev))).to(dt)
    off = torch.zeros(len(new) + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(torch.tensor(new), 0)
    off, new_t = off.to(dev), torch.tensor(new, device=dev)
    masks = None
    if case["tree"]:
        drafted = torch.arange(max(new), device=dev)[None] < new_t[:, None]
        masks = _trees(new, gen, dev)[drafted].contiguous()
    return {"case": case, "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "table": table, "q": q, "masks": masks, "off": off,
            "most_new": max(new), "most": max(total), "tokens": t, "lengths": torch.tensor(total, dtype=torch.int32, device=dev)}


def run(state):
    return (_run_store if state["case"]["op"] == "store" else _run_read)(state)


def _turned(x, gain, s):
    """Norm and rotation, in x's type."""
    c = s["case"]
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain
    cos, sin = s["rope"][s["positions"].long()].to(x.dtype).unbind(-1)
    turn, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["pairs"] == "halves":
        a, b = turn[..., :c["rot"] // 2], turn[..., c["rot"] // 2:]
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
    a, b = a * cos[:, None] - b * sin[:, None], b * cos[:, None] + a * sin[:, None]
    turn = torch.cat([a, b], -1) if c["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turn, rest], -1)


def _run_store(s):
    c = s["case"]
    if own:
        q = s["cache"].append(s["qkv"], s["positions"], s["slots"], c["q_heads"], q_gain=s["q_gain"], k_gain=s["k_gain"],
                              rope=s["rope"], eps=1e-6, neighbours=c["pairs"] == "neighbours")
        return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    hq, hk, bs = c["q_heads"], c["kv_heads"], c["block"]
    x = s["qkv"].view(-1, hq + 2 * hk, c["dim"])
    q = _turned(x[:, :hq].float(), s["q_gain"], s).to(x.dtype)
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    block, spot = at // bs, at % bs
    blocks = block[torch.cat([block[:1] >= 0, block[1:] != block[:-1]])]  # a block's rows follow one another
    begun = torch.zeros(s["k"].shape[0], dtype=torch.bool, device=x.device).index_fill_(0, block[spot == 0], True)[blocks]
    # keys in 64 bits: what lies next to a border between two e4m3 values shall not go by the order of a sum
    for name, y in (("k", _turned(x[:, hq:hq + hk].double(), s["k_gain"], s)), ("v", x[:, hq + hk:].double())):
        y, pool, scales = y[kept], s[name], s[name + "_scale"]
        top = torch.zeros(scales.shape, dtype=y.dtype, device=y.device).index_reduce_(0, block, y.abs().amax(-1), "amax")[blocks]
        mantissa, exponent = torch.frexp(top / LARGEST)
        need = torch.ldexp(torch.ones_like(mantissa), exponent - (mantissa == 0.5).int()).clamp(min=LEAST_SCALE).float()
        old = scales[blocks]
        scale = torch.where(begun[:, None], need, torch.maximum(need, old))
        scales[blocks] = scale
        # older rows of a block that gets a larger scale are rounded once more
        bytes_ = pool.view(torch.uint8)
        ratio = torch.where(begun[:, None], torch.ones_like(old), old / scale)
        bytes_[blocks] = (bytes_[blocks].view(E4M3).float() * ratio[..., None, None]).to(E4M3).view(torch.uint8)
        bytes_[block, :, spot] = (y / scales[block][..., None].double()).float().to(E4M3).view(torch.uint8)
    return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _run_read(s):
    c = s["case"]
    scale = c["dim"] ** -0.5
    if own:
        kind = dict(window=c["window"], sinks=c["sinks"]) if c["window"] else {}
        return s["cache"].attend(s["q"], s["off"], s["lengths"], s["table"], s["ws"], masks=s["masks"], scale=scale,
                                 max_new=c["new_hi"], **kind)
    # all requests at once, filled up to the longest
    hk, d, bs, n = c["kv_heads"], c["dim"], c["block"], s["most_new"]
    group = c["q_heads"] // hk
    off, total = s["off"], s["lengths"].long()
    new = off[1:] - off[:-1]
    ctx = total - new
    i = torch.arange(n, device=off.device)
    real = i[None] < new[:, None]
    row = (off[:-1, None] + i).clamp(max=s["tokens"] - 1)
    masks = s["masks"][row] if c["tree"] else None
    position = ctx[:, None] + i
    if c["tree"]:
        position = ctx[:, None] + sum((masks >> j) & 1 for j in range(n)) - 1  # a token's depth: those above it
    # the places that are read: the first ones, and from where the first token's window begins
    sinks = c["sinks"]
    wide = min(s["most"], c["window"] + n - 1) if c["window"] else s["most"]
    start = (ctx + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(ctx)
    place = torch.cat([torch.arange(sinks, device=off.device).expand(len(start), sinks), start[:, None] + torch.arange(wide, device=off.device)], 1)
    once = torch.cat([torch.ones_like(place[:, :sinks]), place[:, sinks:] >= sinks], 1).bool()
    once &= place < total[:, None]
    place = place.clamp(max=s["most"] - 1)
    at = s["table"].gather(1, place // bs).long()
    k, v = (s[x][at, :, place % bs].float() if s[x + "_scale"] is None
            else s[x].view(torch.uint8)[at, :, place % bs].view(E4M3).float() * s[x + "_scale"][at][..., None] for x in "kv")
    k, v = k.permute(0, 2, 3, 1), v.transpose(1, 2)                       # [R, hk, d, places], [R, hk, places, d]
    q = s["q"][row].float().view(-1, n, hk, group, d).permute(0, 2, 3, 1, 4).reshape(-1, hk, group * n, d)
    w = (q @ k).mul_(scale).view(-1, hk, group, n, place.shape[1])
    j = place[:, None]                                                     # [R, 1, places]
    seen = (j < ctx[:, None, None]) if c["tree"] else j <= position[..., None]
    if c["window"]:
        seen = seen & ((j < sinks) | (j > position[..., None] - c["window"]))
    if c["tree"]:
        drafted = j - ctx[:, None, None]
        seen = seen | ((drafted >= 0) & ((masks[..., None] >> drafted.clamp(0, 63)) & 1 != 0))
    w.masked_fill_(~(seen & once[:, None])[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = w.sub_(top).exp_()
    sums = w.sum(-1, keepdim=True)
    o = (w.view(-1, hk, group * n, w.shape[-1]) @ v).view(-1, hk, group, n, d) / torch.where(sums > 0, sums, torch.ones_like(sums))
    return o.permute(0, 3, 1, 2, 4)[real].reshape(-1, c["q_heads"], d).to(s["q"].dtype)


def work(case):
    new, ctx = _lengths(case)
    t, d, hq, hk, bs = sum(new), case["dim"], case["q_heads"], case["kv_heads"], case["block"]
    if case["op"] == "store":
        blocks = sum(-(-(c % bs + n) // bs) for n, c in zip(new, ctx))
        # rows in, queries out in 16 bits, keys and values in 8; slots, positions and angles; scales in and out
        return {"bytes": t * ((2 * hq + 2 * hk) * d * 2 + 2 * hk * d + 12 + case["rot"] * 4) + blocks * hk * 16,
                "flops": t * (hq + hk) * (4 * d + 3 * case["rot"]) + 2 * t * hk * d}
    size, window, sinks = case["bits"] // 8, case["window"], case["sinks"]
    keys = pairs = 0
    for n, c in zip(new, ctx):
        keys += min(c + n, sinks + window + n - 1) if window else c + n
        for i in range(n):
            p = c if case["tree"] else c + i
            pairs += p + 1 if not window or p < window else window + min(sinks, p + 1 - window)
    scales = 8 * hk * (keys // bs + len(new)) if size == 1 else 0
    return {"bytes": 2 * keys * hk * d * size + scales + t * hq * d * 4 + 4 * keys // bs, "flops": 4 * d * hq * pairs}


# The definitions once more in 64 bits, written on their own: head by head, request by request.

def exact(case, seed):
    s = _inputs(case, seed)
    return (_exact_store if case["op"] == "store" else _exact_read)(case, s)


def _exact_store(c, s):
    """Keys and values as multiples of their scale, before the rounding to 8 bits."""
    hq, hk, d, rot, bs = c["q_heads"], c["kv_heads"], c["dim"], c["rot"], c["block"]
    x = s["qkv"].double().reshape(-1, hq + 2 * hk, d)
    z = torch.view_as_complex(s["rope"].double())[s["positions"].long()]  # cos + i sin
    half = rot // 2
    first = torch.arange(half, device=x.device) * (1 if c["pairs"] == "halves" else 2)
    second = first + (half if c["pairs"] == "halves" else 1)
    out = {name: s[name].double() for name in ("k", "v", "k_scale", "v_scale")}
    out["q"] = torch.empty(x.shape[0], hq, d, dtype=torch.float64, device=x.device)
    kept = (s["slots"] >= 0).nonzero().flatten()
    blocks, spots = s["slots"][kept] // bs, s["slots"][kept] % bs
    touched = torch.zeros(s["k"].shape[0], dtype=torch.bool, device=x.device)
    touched[blocks] = True
    begun = torch.zeros_like(touched)
    begun[blocks[spots == 0]] = True
    for h in range(hq + 2 * hk):
        y = x[:, h].clone()
        gain = None if h >= hq + hk else s["q_gain"] if h < hq else s["k_gain"]
        if gain is not None:
            y *= (y.pow(2).sum(1, keepdim=True) / d + 1e-6).rsqrt() * gain.double()
        if h < hq + hk:
            turned = torch.complex(y[:, first], y[:, second]) * z
            y[:, first], y[:, second] = turned.real, turned.imag
        if h < hq:
            out["q"][:, h] = y
            continue
        name, g = ("k", h - hq) if h < hq + hk else ("v", h - hq - hk)
        y = y[kept]
        largest = torch.zeros(touched.shape[0], dtype=torch.float64, device=x.device)
        largest.scatter_reduce_(0, blocks, y.abs().amax(1), "amax")
        least = torch.exp2(torch.round(torch.log2(largest / LARGEST)) - 1).clamp(min=LEAST_SCALE)
        for _ in range(2):  # a logarithm may be off next to a whole number
            least = torch.where(largest > LARGEST * least, 2 * least, least)
        before = out[name + "_scale"][:, g].clone()
        after = torch.where(begun, least, torch.maximum(least, before))
        out[name + "_scale"][:, g] = torch.where(touched, after, before)
        out[name][:, g] *= torch.where(touched & ~begun, before / after, 1.0)[:, None, None]
        out[name][blocks, g, spots] = y / after[blocks][:, None]
    return out


def _exact_read(c, s):
    hq, hk, d, bs = c["q_heads"], c["kv_heads"], c["dim"], c["block"]
    dev = s["q"].device
    out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device=dev)
    new, ctx = _lengths(c)
    start = 0
    for r, (n, before) in enumerate(zip(new, ctx)):
        place = torch.arange(before + n, device=dev)
        i = torch.arange(n, device=dev)[:, None]
        if c["tree"]:
            bits = (s["masks"][start:start + n, None] >> torch.arange(n, device=dev)) & 1
            at = before + bits.sum(1, keepdim=True) - 1
        else:
            at = before + i
        if c["window"]:  # only the places that some token sees
            low = before + 1 - c["window"]
            place = place[(place < c["sinks"]) | (place >= low)]
        rows, spots = s["table"][r].long()[place // bs], place % bs
        if c["tree"]:
            later = torch.where(place >= before, bits[:, (place - before).clamp(min=0)] == 0, False)
        else:
            later = place[None] > at
        if c["window"]:
            far = (place[None] >= c["sinks"]) & (place[None] <= at - c["window"])
            later = later | (far & (place[None] < before) if c["tree"] else far)
        for g in range(hk):
            if s["k_scale"] is None:
                k, v = s["k"][rows, g, spots].double(), s["v"][rows, g, spots].double()
            else:
                k, v = (s[x].view(torch.uint8)[rows, g, spots].view(E4M3).double() * s[x + "_scale"][rows, g].double()[:, None] for x in "kv")
            for h in range(g * hq // hk, (g + 1) * hq // hk):
                logit = torch.einsum("nd,jd->nj", s["q"][start:start + n, h].double(), k) / math.sqrt(d)
                logit = logit.masked_fill(later, -math.inf)
                out[start:start + n, h] = torch.exp(logit - torch.logsumexp(logit, 1, keepdim=True)) @ v
        start += n
    return out

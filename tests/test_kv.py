"""The paged cache calls (tk_kv_*) against plain 64-bit implementations, and their refusals.

Tolerances. A rounding to the storage type changes a value by at most u =
finfo.eps / 2 of it: 2^-8 (bf16, 8 significant bits) or 2^-11 (fp16).
  append: y is computed in fp32 (a mean of at most 256 squares, a square root,
  a division, three products and one sum: under 2^-17 relative to the terms)
  and rounded once: |err| <= 1.02 u |y| + 2^-17 (|a| + |b|), with a, b the pair
  before the rotation, plus half the smallest fp16 subnormal, 2^-25.
  attend: the weights are rounded to the type (u each, and 2^-25 absolute in
  fp16 where they are subnormal), the result once more; a score's fp32 sum of
  128 products is within 2^-17 of sum |q||k| scale = S, which moves weights by
  2 * 2^-17 S relative. With A = sum_j w_j |v_j|:
  |err| <= 1.02 u (|o| + A) + 2^-15 (1 + S) A + n 2^-24 max|v| (fp16).
  lse: the maximum's fp32 score and the sum's logarithm: 2^-16 (1 + S).
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def tk():
    import byte_level_bpe_gb300 as tk
    return tk


# ------------------------------------------------------------------- refusals

def _create(**kw):
    from byte_level_bpe_gb300 import native
    a = dict(k=4096, v=4096, type=native.TK_BF16, n=4, h=2, bs=16, d=64, stride=None)
    a.update(kw)
    h = ctypes.c_void_p()
    st = (ctypes.c_int64 * 3)(*a["stride"]) if a["stride"] else None
    return native.load().tk_kv_cache_create(a["k"], a["v"], a["type"], a["n"], a["h"], a["bs"], a["d"], st,
                                            ctypes.byref(h))


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(type=3), dict(n=0), dict(h=0), dict(h=1025),
                                dict(bs=8), dict(bs=24), dict(bs=256), dict(d=24), dict(d=272), dict(k=4104),
                                dict(stride=(2048, 1024, 60)), dict(stride=(2048, 1024, 56)),
                                dict(stride=(1 << 40, 1024, 64))])
def test_cache_refusals_are_host_side(kw):
    from byte_level_bpe_gb300 import native
    assert _create(**kw) == native.TK_E_ARG
    assert native.load().tk_last_error()


def test_plan_refusals_are_host_side():
    from byte_level_bpe_gb300 import native
    ok = dict(off=4096, ctx=4096, R=2, T=3, bs=16, table=4096, ts=4, tw=4, free=4096, nf=4, cur=None, par=None, pos=4096,
              slot=4096, req=4096, len=4096, mask=None, info=4096)
    for bad in (dict(bs=12), dict(R=-1), dict(T=-1), dict(T=1 << 31), dict(ts=3), dict(nf=-1), dict(off=None),
                dict(ctx=None), dict(info=None), dict(pos=None), dict(par=4096), dict(free=None), dict(slot=4104),
                dict(table=None), dict(len=None)):
        a = {**ok, **bad}
        assert native.load().tk_kv_plan(*a.values(), None) == native.TK_E_ARG, bad


def test_null_handles():
    from byte_level_bpe_gb300 import native
    lib = native.load()
    assert lib.tk_kv_append(None, 4096, 256, 1, 2, None, None, 0.0, None, 0, 0, 0, None, 4096, 4096, None) == native.TK_E_ARG
    assert lib.tk_kv_attend(None, None, 4096, 256, 2, 4096, 1, 1, 1, 4096, 4096, 1, 1, None, 1.0, 4096, None,
                            None) == native.TK_E_ARG
    assert lib.tk_kv_status(None, None, None) == native.TK_E_ARG
    assert lib.tk_kv_workspace_create(None) == native.TK_E_ARG


def test_no_cpu_fallback():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    import byte_level_bpe_gb300 as tk
    with pytest.raises(RuntimeError):
        tk.KVCache(torch.zeros(1, 1, 16, 64), torch.zeros(1, 1, 16, 64))


@pytest.mark.gpu
def test_call_refusals(tk):
    from byte_level_bpe_gb300.native import TK_E_ARG
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    k = z(4, 2, 16, 64)
    cache, ws = tk.KVCache(k, k.clone()), tk.KVWorkspace()
    pos, slots = z(3, t=torch.int32), z(3, t=torch.int64)
    off, ln, tab = torch.tensor([0, 3], device="cuda"), z(1, t=torch.int32) + 3, z(1, 2, t=torch.int32)
    rope = tk.rope_table(8, 64)
    for bad in (lambda: tk.KVCache(k.cpu(), k.cpu()), lambda: tk.KVCache(k, k.half()), lambda: tk.KVCache(k.float(), k.float()),
                lambda: tk.KVCache(k.transpose(2, 3), k.transpose(2, 3)), lambda: tk.KVCache(k, k[:2]),
                lambda: cache.append(z(3, 6 * 64), pos, slots, 4), lambda: cache.append(z(3, 8 * 64, t=torch.float16), pos, slots, 4),
                lambda: cache.append(z(3, 8 * 64), pos.long(), slots, 4, rope=rope),
                lambda: cache.append(z(3, 8 * 64), pos, slots[:2], 4), lambda: cache.append(z(3, 8 * 64), pos, slots, 4, rope=rope.half()),
                lambda: cache.append(z(3, 8 * 64), pos, slots, 4, q_gain=z(64)),
                lambda: cache.attend(z(3, 4, 32), off, ln, tab, ws), lambda: cache.attend(z(3, 4, 64), off.int(), ln, tab, ws),
                lambda: cache.attend(z(3, 4, 64), off, ln, tab.long(), ws), lambda: cache.attend(z(3, 4, 64).float(), off, ln, tab, ws),
                lambda: cache.attend(z(3, 4, 64), off, ln, tab, ws, masks=slots[:2]),
                lambda: tk.kv_plan(off, ln.long(), tab, pos, 16, 3), lambda: tk.kv_plan(off, ln, tab.cpu(), pos, 16, 3)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cache.attend(z(3, 3, 64), off, ln, tab, ws), lambda: cache.attend(z(3, 4, 64), off, ln, tab, ws, scale=0.0),
                lambda: cache.attend(z(3, 4, 64), off, ln, tab, ws, scale=float("nan")),
                lambda: cache.attend(z(3, 4, 64), off, ln, tab, ws, scale=-1.0),
                lambda: cache.append(z(3, 8 * 64 + 4)[:, :8 * 64], pos, slots, 4),
                lambda: cache.append(z(3, 8 * 64), pos, slots, 4, eps=-1.0),
                lambda: cache.append(z(3, 8 * 64), pos, slots, 4, rope=tk.rope_table(8, 24)),
                lambda: cache.append(z(3, 8 * 64), pos, slots, 4, rope=tk.rope_table(8, 80)),
                lambda: tk.kv_plan(off, ln, tab, pos, 24, 3)):
        with pytest.raises(tk.TkError) as e:
            bad()
        assert e.value.code == TK_E_ARG
    wide = tk.KVCache(z(4, 2, 16, 96), z(4, 2, 16, 96))  # stores, but attention takes 64 and 128 only
    with pytest.raises(tk.TkError):
        wide.attend(z(3, 4, 96), off, ln, tab, ws)


# ----------------------------------------------------------------------- plan

def plan_oracle(off, ctx, table, free, bs, T, parents=None, cursor=0):
    R, W = table.shape
    table = table.copy()
    pos, slot, req = np.zeros(T, np.int32), np.full(T, -1, np.int64), np.full(T, -1, np.int32)
    length, mask = ctx.copy(), np.zeros(T, np.int64)
    at, asked, code, who = cursor, 0, 0, -1
    end = cursor
    for r in range(R):
        n, c = int(off[r + 1] - off[r]), int(ctx[r])
        want, have = -(-(c + n) // bs), -(-c // bs)
        need = -1 if c < 0 or want > W or (parents is not None and n > 64) else want - have
        ok = need == 0
        if need > 0:
            asked += need
            end += need
            if end <= len(free):
                ok = True
                table[r, have:want] = free[end - need:end]
                at = end
        if ok:
            length[r] = c + n
        elif code == 0:
            code, who = (-9 if need < 0 else -4), r
        for i in range(n):
            t = int(off[r]) + i
            req[t] = r
            pos[t] = c + i
            if ok:
                slot[t] = table[r, (c + i) // bs] * bs + (c + i) % bs
            if parents is not None:
                if i >= 64:
                    pos[t] = c
                    continue
                m, d, k = 1 << i, 0, i
                while 0 <= parents[int(off[r]) + k] < k:
                    k = int(parents[int(off[r]) + k])
                    m |= 1 << k
                    d += 1
                pos[t] = c + d
                mask[t] = np.uint64(m).astype(np.int64)
    return table, pos, slot, req, length, mask, np.array([at, asked, code, who], np.int64)


def _plan_case(rng, R, hi, ctx_hi, bs, tree, zero=0.2):
    n = rng.integers(1, hi + 1, R)
    n[rng.random(R) < zero] = 0
    ctx = rng.integers(0, ctx_hi + 1, R).astype(np.int32)
    off = np.zeros(R + 1, np.int64)
    np.cumsum(n, out=off[1:])
    have = -(-ctx // bs)
    W = int((-(-(ctx + n) // bs)).max(initial=0)) + 2
    need = int((-(-(ctx + n) // bs) - have).sum())
    ids = rng.permutation(need + int(have.sum()) + 5).astype(np.int32)
    table = np.full((R, W), -7, np.int32)
    k = need + 5
    for r in range(R):
        table[r, :have[r]] = ids[k:k + have[r]]
        k += have[r]
    par = None
    if tree:
        par = np.concatenate([rng.integers(-1, np.maximum(np.arange(m), 1)) for m in n] or [np.zeros(0)]).astype(np.int32)
    return off, ctx, table, ids[:need + 5].copy(), par


def _check_plan(tk, off, ctx, table, free, bs, par=None, T=None, cursor=None, wide=False):
    T = int(off[-1]) if T is None else T
    d = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    dt = d(table)
    if wide:  # rows further apart than they are wide
        big = torch.full((table.shape[0], table.shape[1] + 3), 99, dtype=torch.int32, device="cuda")
        big[:, :table.shape[1]] = dt
        dt = big[:, :table.shape[1]]
    full = par
    if par is not None and T > len(par):
        full = np.concatenate([par, np.zeros(T - len(par), np.int32)])
    cur = None if cursor is None else torch.tensor([cursor], device="cuda")
    p = tk.kv_plan(d(off), d(ctx), dt, d(free), bs, T, parents=d(full), cursor=cur)
    want = plan_oracle(off, ctx, table, free, bs, T, full, cursor or 0)
    got = [dt, p.positions, p.slots, p.requests, p.lengths, p.masks, p.info]
    for name, g, w in zip(("table", "positions", "slots", "requests", "lengths", "masks", "info"), got, want):
        if g is None:
            assert par is None and name == "masks"
            continue
        assert np.array_equal(g.cpu().numpy(), w), name
    if wide:
        assert bool((big[:, table.shape[1]:] == 99).all())
    return p


@pytest.mark.gpu
@pytest.mark.parametrize("R,hi,ctx_hi,bs,tree", [(1, 1, 0, 16, False), (1, 1, 40, 16, True), (3, 5, 33, 16, False),
                                                 (7, 64, 300, 32, True), (64, 1, 1000, 16, False), (511, 3, 90, 16, False),
                                                 (513, 64, 50, 64, True), (1300, 2, 500, 128, False), (5, 40000, 7, 16, False),
                                                 (4096, 300, 0, 64, False), (2100, 64, 9, 16, True), (2, 1000003, 5, 32, False)])
@pytest.mark.parametrize("seed", [0, 1])
def test_plan(tk, R, hi, ctx_hi, bs, tree, seed):
    rng = np.random.default_rng(1000 * R + seed)
    off, ctx, table, free, par = _plan_case(rng, R, hi, ctx_hi, bs, tree)
    _check_plan(tk, off, ctx, table, free, bs, par, wide=seed == 1)


@pytest.mark.gpu
def test_plan_edges(tk):
    rng = np.random.default_rng(5)
    off, ctx, table, free, par = _plan_case(rng, 40, 60, 100, 16, True)
    _check_plan(tk, off, ctx, table, free, 16, par, T=int(off[-1]) + 1000)          # padding
    p = _check_plan(tk, off, ctx, table, free, 16, par, cursor=3)
    assert int(p.info[0]) == len(free) - 2
    for left in (0, 1, len(free) // 2):                                             # the free list runs out
        p = _check_plan(tk, off, ctx, table, free[:left], 16, par)
        assert int(p.info[2]) == tk.native.TK_E_CAPACITY
    bad = ctx.copy()
    bad[[3, 11]] = -1
    p = _check_plan(tk, off, bad, table, free, 16, par)
    assert p.info[2:].tolist() == [tk.native.TK_E_LIMIT, 3]
    p = _check_plan(tk, off, ctx, table[:, :6], free, 16, par)                      # a table that is too narrow
    assert int(p.info[2]) == tk.native.TK_E_LIMIT
    odd = par.copy()
    odd[::3] = rng.integers(-2 ** 31, 2 ** 31, len(odd[::3]))                       # parents that are none
    _check_plan(tk, off, ctx, table, free, 16, odd)
    off, ctx, table, free, par = _plan_case(rng, 30, 90, 50, 16, True)              # trees over 64 tokens
    p = _check_plan(tk, off, ctx, table, free, 16, par)
    assert int(p.info[2]) == tk.native.TK_E_LIMIT
    z = np.zeros(0, np.int32)
    p = _check_plan(tk, np.zeros(1, np.int64), z, np.zeros((0, 0), np.int32), z, 16, T=9)  # no request
    assert p.info.tolist() == [0, 0, 0, -1]
    _check_plan(tk, np.zeros(6, np.int64), np.zeros(5, np.int32), np.zeros((5, 1), np.int32), z, 16)  # no token


@pytest.mark.gpu
def test_plan_chain_of_calls(tk):
    """Steps of a server: one call's cursor is the next one's, without the host."""
    rng = np.random.default_rng(9)
    R, bs, W = 17, 16, 40
    free = rng.permutation(2000).astype(np.int32)
    table, ctx, cursor = np.zeros((R, W), np.int32), np.zeros(R, np.int32), 0
    d_table, d_ctx, d_free = (torch.from_numpy(x.copy()).cuda() for x in (table, ctx, free))
    d_cur = None
    for step in range(6):
        n = rng.integers(0, 90, R)
        off = np.zeros(R + 1, np.int64)
        np.cumsum(n, out=off[1:])
        p = tk.kv_plan(torch.from_numpy(off).cuda(), d_ctx, d_table, d_free, bs, int(off[-1]), cursor=d_cur)
        table, pos, slot, req, ctx, _, info = plan_oracle(off, ctx, table, free, bs, int(off[-1]), None, cursor)
        cursor = int(info[0])
        d_cur, d_ctx = p.info[:1], p.lengths
        assert np.array_equal(p.slots.cpu().numpy(), slot) and np.array_equal(d_table.cpu().numpy(), table)
        assert p.info.tolist() == info.tolist()


# --------------------------------------------------------------------- append

def _append_oracle(x, hq, hk, d, q_gain, k_gain, eps, rope, pos, neighbours):
    """(normed and rotated heads, the rotation's operands |a| + |b|), 64 bits."""
    T = x.shape[0]
    y = x.double().view(T, hq + 2 * hk, d).clone()
    size = torch.zeros_like(y)
    for h in range(hq + hk):
        g = q_gain if h < hq else k_gain
        if g is not None:
            y[:, h] = y[:, h] / torch.sqrt((y[:, h] ** 2).mean(1, keepdim=True) + eps) * g.double()
        size[:, h] = y[:, h].abs()
        if rope is None:
            continue
        half = rope.shape[1]
        a = torch.arange(half) * 2 if neighbours else torch.arange(half)
        b = a + 1 if neighbours else a + half
        c, s = rope.double()[pos.clamp(0, rope.shape[0] - 1).long()].unbind(-1)
        out = (pos < 0) | (pos >= rope.shape[0])
        c[out] = s[out] = float("nan")
        ya, yb = y[:, h, a].clone(), y[:, h, b].clone()
        y[:, h, a], y[:, h, b] = ya * c - yb * s, yb * c + ya * s
        size[:, h, a] = size[:, h, b] = ya.abs() + yb.abs()
    return y, size


def _close(got, want, tol, what=""):
    got, want = got.double().cpu(), want.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    err = torch.where(torch.isnan(want) | (got == want), torch.zeros_like(want), (got - want).abs())
    assert bool((err <= tol).all()), (what, float((err / tol).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,hq,hk,d,rot,neighbours,bs,norm", [
    (1, 1, 1, 16, 16, False, 16, True), (5, 4, 2, 64, 64, False, 16, True), (33, 7, 7, 64, 32, True, 32, True),
    (9, 20, 4, 96, 96, False, 16, False), (130, 8, 1, 128, 128, True, 64, True), (77, 12, 3, 128, 64, False, 128, True),
    (64, 32, 8, 128, 128, False, 16, True), (3, 2, 2, 256, 256, False, 16, True), (19, 6, 2, 240, 112, True, 32, True),
    (11, 5, 1, 80, 0, False, 16, True), (2, 1, 1, 48, 48, True, 16, False), (700, 3, 1, 112, 112, False, 16, True)])
def test_append(tk, dtype, T, hq, hk, d, rot, neighbours, bs, norm):
    gen = torch.Generator().manual_seed(T * d + rot)
    blocks = -(-T // bs) + 2
    wide = (hq + 2 * hk) * d
    pad = 8 * (T % 3)
    store = (torch.randn(T, wide + pad, generator=gen) * torch.exp(torch.randn(T, 1, generator=gen))).to(dtype)
    x = store[:, :wide]
    pool = torch.randn(2, blocks, bs, hk, d, generator=gen).to(dtype).cuda()
    order_tokens_first = d % 32 == 0  # the cache laid out [block][token][head] instead
    kv = [pool[i].transpose(1, 2) if order_tokens_first else pool[i].reshape(blocks, hk, bs, d) for i in (0, 1)]
    before = [c.clone() for c in kv]
    slots = torch.randperm(blocks * bs, generator=gen)[:T]
    slots[1::5] = -1
    if T > 4:
        slots[4], slots[3] = blocks * bs, 1 << 40
    pos = torch.randint(0, 500, (T,), generator=gen).int()
    rope = tk.rope_table(500, rot) if rot else None
    if T > 6:
        pos[5], pos[6] = -1, 500
    g = [1 + 0.3 * torch.randn(d, generator=gen) for _ in range(2)] if norm else [None, None]
    cache = tk.KVCache(kv[0], kv[1])
    q = cache.append(store.cuda()[:, :wide], pos.cuda(), slots.cuda(), hq, q_gain=g[0].cuda() if norm else None,
                     k_gain=g[1].cuda() if norm else None, rope=rope, eps=1e-5, neighbours=neighbours)
    y, size = _append_oracle(x, hq, hk, d, g[0], g[1], 1e-5, rope.cpu() if rot else None, pos, neighbours)
    tol = 1.02 * U[dtype] * y.abs().nan_to_num() + 2.0 ** -17 * size + 2.0 ** -25
    _close(q, y[:, :hq], tol[:, :hq], "q")
    want_k, want_v = before[0].double().cpu(), before[1].double().cpu()
    tol_k = torch.zeros_like(want_k)
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < blocks * bs:
            want_k[s // bs, :, s % bs] = y[t, hq:hq + hk]
            tol_k[s // bs, :, s % bs] = tol[t, hq:hq + hk]
            want_v[s // bs, :, s % bs] = y[t, hq + hk:]
    _close(kv[0], want_k, tol_k, "k")
    _close(kv[1], want_v, torch.zeros_like(want_v), "v")


@pytest.mark.gpu
def test_append_of_nothing_and_of_extremes(tk):
    d, hq, hk = 64, 2, 1
    k, v = (torch.zeros(2, hk, 16, d, dtype=torch.float16, device="cuda") for _ in "kv")
    cache = tk.KVCache(k, v)
    i32, i64 = torch.int32, torch.int64
    empty = cache.append(torch.zeros(0, 4 * d, dtype=torch.float16, device="cuda"), torch.zeros(0, dtype=i32, device="cuda"),
                         torch.zeros(0, dtype=i64, device="cuda"), hq)
    assert empty.shape == (0, hq, d)
    x = torch.zeros(3, 4 * d, dtype=torch.float16, device="cuda")
    x[1] = 65504.0          # squares far above fp16
    x[2, 5] = float("inf")
    one = torch.ones(d, device="cuda")
    q = cache.append(x, torch.zeros(3, dtype=i32, device="cuda"), torch.arange(3, device="cuda"), hq, q_gain=one, k_gain=one)
    assert bool((q[0] == 0).all()) and bool((q[1] == 1).all()) and bool(torch.isnan(q[2, 0, 5])) and bool((q[2, 1] == 0).all())


# --------------------------------------------------------------------- attend

def attend_oracle(q, k, v, off, lens, table, scale, masks=None):
    """(o, lse, A, S) in 64 bits; q [T, hq, d], k, v [blocks, hk, bs, d]."""
    T, hq, d = q.shape
    hk, bs = k.shape[1], k.shape[2]
    o, a = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64)
    lse = torch.full((T, hq), -np.inf, dtype=torch.float64)
    big = torch.zeros(T, hq, dtype=torch.float64)
    for r in range(len(lens)):
        n, L = int(off[r + 1] - off[r]), int(lens[r])
        ctx = L - n
        place = torch.arange(L)
        rows = table[r].long()[place // bs]
        kk, vv = k[rows, :, place % bs].double(), v[rows, :, place % bs].double()  # [L, hk, d]
        for i in range(n):
            t = int(off[r]) + i
            if masks is None:
                seen = place <= ctx + i
            else:
                m = int(masks[t]) & (2 ** 64 - 1)
                seen = torch.tensor([j < ctx or (m >> (j - ctx)) & 1 == 1 for j in range(L)], dtype=torch.bool)
            if not bool(seen.any()):
                continue
            for h in range(hq):
                g = h // (hq // hk)
                ks, vs = kk[seen, g], vv[seen, g]
                s = ks @ q[t, h].double() * scale
                lse[t, h] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[t, h])
                o[t, h], a[t, h] = w @ vs, w @ vs.abs()
                big[t, h] = (ks.abs() @ q[t, h].double().abs()).max() * scale
    return o, lse, a, big


def _attend_case(gen, new, ctx, hq, hk, d, bs, dtype, extra=2, poison=True, scale=1.5):
    """Tensors on the CPU. Places past a request's end hold NaN."""
    R = len(new)
    used = [-(-(c + n) // bs) for c, n in zip(ctx, new)]
    blocks = sum(used) + extra
    k, v = (torch.randn(blocks, hk, bs, d, generator=gen).to(dtype) for _ in "kv")
    ids = torch.randperm(blocks, generator=gen)
    table = torch.full((R, max(used, default=0) + 1), -1, dtype=torch.int32)
    at = 0
    for r in range(R):
        table[r, :used[r]] = ids[at:at + used[r]].int()
        at += used[r]
        end = ctx[r] + new[r]
        if poison and end % bs:
            k[table[r, used[r] - 1].long(), :, end % bs:] = float("nan")
            v[table[r, used[r] - 1].long(), :, end % bs:] = float("nan")
    if poison:
        for b in ids[at:]:
            k[b] = v[b] = float("nan")
    off = torch.zeros(R + 1, dtype=torch.int64)
    off[1:] = torch.cumsum(torch.tensor(new), 0)
    q = (torch.randn(int(off[-1]), hq, d, generator=gen) * scale).to(dtype)
    lens = torch.tensor([c + n for c, n in zip(ctx, new)], dtype=torch.int32)
    return q, k, v, off, lens, table


def _tree_masks(gen, new):
    out = []
    for n in new:
        m = []
        for i in range(n):
            p = int(torch.randint(-1, max(i, 1), (1,), generator=gen)) if i else -1
            m.append((1 << i) | (m[p] if p >= 0 else 0))
        out += [x - (1 << 64) if x >= 1 << 63 else x for x in m]
    return torch.tensor(out, dtype=torch.int64)


def _check_attend(tk, q, k, v, off, lens, table, masks=None, scale=None, max_new=None, ws=None, want=None):
    dtype, d = q.dtype, q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, lse, a, big = want or attend_oracle(q, k, v, off, lens, table, scale, masks)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    cache = tk.KVCache(c(k), c(v))
    ws = ws or tk.KVWorkspace()
    got, got_lse = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), scale=scale, max_new=max_new, lse=True)
    ws.status()
    n = float(lens.max()) if len(lens) else 0.0
    tol = 1.02 * U[dtype] * (o.abs() + a) + 2.0 ** -15 * (1 + big[..., None]) * a + 2.0 ** -24
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -24 * v[~torch.isnan(v)].abs().max().double()
    _close(got, o, tol, "out")
    fin = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got_lse.cpu()), ~fin)
    assert bool(((got_lse.cpu().double() - lse).abs()[fin] <= (2.0 ** -16 * (1 + big))[fin]).all())
    again = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), scale=scale, max_new=max_new)
    assert torch.equal(again, got)  # the same bits
    _close(cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), scale=scale), o, tol, "no max_new")
    return got


SHAPES = [([1], [0], 1, 1, 16), ([1], [199], 4, 1, 16), ([1, 1, 1], [0, 15, 16], 8, 8, 16), ([1] * 5, [127, 128, 129, 255, 700], 6, 2, 32),
          ([3, 0, 17], [5, 9, 0], 4, 2, 64), ([64, 1, 33], [130, 1000, 2], 8, 1, 16), ([63, 64], [64, 383], 16, 2, 128),
          ([2] * 40, list(range(0, 800, 20)), 2, 2, 16), ([7], [3000], 5, 5, 32), ([5, 64], [2500, 1], 20, 4, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attend(tk, dtype, d, tree, shape):
    new, ctx, hq, hk, bs = SHAPES[shape]
    gen = torch.Generator().manual_seed(100 * shape + d)
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, d, bs, dtype)
    masks = _tree_masks(gen, new) if tree else None
    _check_attend(tk, q, k, v, off, lens, table, masks, max_new=max(new))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,ctx,hq,hk,d,bs", [([300], [0], 2, 1, 64, 16), ([129, 257, 1], [77, 0, 400], 4, 2, 128, 64),
                                                ([70], [1000], 8, 1, 128, 32)])
def test_attend_chunks_of_prompts(tk, dtype, new, ctx, hq, hk, d, bs):
    gen = torch.Generator().manual_seed(sum(new) + d)
    _check_attend(tk, *_attend_case(gen, new, ctx, hq, hk, d, bs, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_attend_masks_that_are_no_trees(tk, d):
    """Empty rows, bits past the request's tokens, rows that do not see themselves."""
    gen = torch.Generator().manual_seed(d)
    new, ctx = [5, 64, 3], [0, 40, 0]
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, 4, 2, d, 16, torch.bfloat16)
    masks = torch.randint(-2 ** 63, 2 ** 63 - 1, (72,), generator=gen)
    masks[:3] = 0
    masks[3] = -1
    masks[69:] = 0
    _check_attend(tk, q, k, v, off, lens, table, masks)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx", [0, 100, 120, 256])
def test_attend_hidden_nonfinite(tk, dtype, d, ctx):
    """A drafted token with infinite or NaN keys and values reaches the rows
    that see it and no others."""
    gen = torch.Generator().manual_seed(d + ctx)
    n, bs, hq, hk = 40, 16, 4, 2
    q, k, v, off, lens, table = _attend_case(gen, [n], [ctx], hq, hk, d, bs, dtype)
    clean = [k.clone(), v.clone()]
    bad = {7: float("nan"), 21: float("inf"), 39: float("-inf")}
    masks = torch.tensor([(1 << i) | ((1 << (i // 2)) if i % 3 == 0 else 0) for i in range(n)])
    for j, x in bad.items():
        b, s = int(table[0, (ctx + j) // bs]), (ctx + j) % bs
        v[b, :, s, 3::5] = x
        if j == 7:
            k[b, :, s] = x
    sees = torch.tensor([any((int(m) >> j) & 1 for j in bad) for m in masks])
    want = attend_oracle(q, clean[0], clean[1], off, lens, table, d ** -0.5, masks)
    c = lambda x: x.cuda()  # noqa: E731
    cache, ws = tk.KVCache(c(k), c(v)), tk.KVWorkspace()
    got = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks)).cpu()
    tol = 1.02 * U[dtype] * (want[0].abs() + want[2]) + 2.0 ** -15 * (1 + want[3][..., None]) * want[2] + 2.0 ** -24
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -24 * 8
    _close(got[~sees], want[0][~sees], tol[~sees], "rows that see none of them")
    for t in torch.nonzero(sees).flatten().tolist():
        m = int(masks[t])
        if (m >> 7) & 1:
            assert bool(torch.isnan(got[t]).all())
        elif (m >> 21) & 1:
            assert bool((got[t, :, 3::5] == float("inf")).all()) and bool(torch.isfinite(got[t, :, :3]).all())
        else:
            assert bool((got[t, :, 3::5] == float("-inf")).all()) and bool(torch.isfinite(got[t, :, :3]).all())


@pytest.mark.gpu
def test_attend_layouts_and_streams(tk):
    """A cache laid out [block][token][head], queries inside a wider row, rows
    of the table further apart, another stream, other block ids."""
    gen = torch.Generator().manual_seed(3)
    q, k, v, off, lens, table = _attend_case(gen, [3, 20, 1], [50, 301, 0], 8, 2, 128, 32, torch.bfloat16)
    masks = _tree_masks(gen, [3, 20, 1])
    base = _check_attend(tk, q, k, v, off, lens, table, masks)
    kt, vt = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (k, v))
    wide = torch.full((24, 8 * 128 + 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 256:256 + 1024] = q.reshape(24, -1).cuda()
    tab = torch.full((3, table.shape[1] + 5), 1 << 30, dtype=torch.int32, device="cuda")
    tab[:, :table.shape[1]] = table.cuda()
    ins = [off.cuda(), lens.cuda(), tab[:, :table.shape[1]], masks.cuda()]
    cache, ws = tk.KVCache(kt, vt), tk.KVWorkspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = cache.attend(wide[:, 256:1280].view(24, 8, 128), ins[0], ins[1], ins[2], ws, masks=ins[3])
        ws.status()
    s.synchronize()
    assert torch.equal(got, base)


@pytest.mark.gpu
def test_attend_requests_out_of_limits(tk):
    """They give zeros and a status; the others are not touched by it."""
    gen = torch.Generator().manual_seed(4)
    new, ctx = [2, 70, 3, 4], [20, 50, 10, 90]
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, 4, 2, 64, 16, torch.bfloat16)
    lens[2] = 1                      # fewer than its new tokens
    lens[3] = 16 * table.shape[1] + 1  # past the table
    masks = _tree_masks(gen, [2, 64, 3, 4])
    masks = torch.cat([masks[:66], torch.zeros(6, dtype=torch.int64), masks[66:]])
    c = lambda x: x.cuda()  # noqa: E731
    cache, ws = tk.KVCache(c(k), c(v)), tk.KVWorkspace()
    got, lse = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), lse=True)
    with pytest.raises(tk.TkError) as e:
        ws.status()
    assert e.value.code == tk.native.TK_E_LIMIT
    ws.status()  # reported once
    assert bool((got[2:] == 0).all()) and bool(torch.isneginf(lse[2:]).all())
    o, _, a, big = attend_oracle(q[:2], k, v, off[:2], lens[:1], table, 64 ** -0.5, masks[:2])
    _close(got[:2], o, 1.02 * U[q.dtype] * (o.abs() + a) + 2.0 ** -15 * (1 + big[..., None]) * a)
    cache.attend(c(q[:2]), c(off[:2]), c(lens[:1]), c(table[:1]), ws, max_new=1)  # 2 new tokens over the bound
    with pytest.raises(tk.TkError):
        ws.status()
    # ids outside the cache read as zeros: uniform weights over the keys, values 0
    wild = torch.tensor([[-5, 1 << 30]], dtype=torch.int32, device="cuda")
    got, lse = cache.attend(c(q[:1]), c(torch.tensor([0, 1])), c(torch.tensor([20], dtype=torch.int32)), wild, ws, lse=True)
    assert bool((got == 0).all()) and bool(((lse - np.log(20)).abs() < 1e-5).all())


@pytest.mark.gpu
def test_attend_many_requests(tk):
    """More requests than a block has threads; empty ones among them."""
    gen = torch.Generator().manual_seed(6)
    R = 1500
    new = torch.randint(0, 3, (R,), generator=gen).tolist()
    ctx = torch.randint(0, 60, (R,), generator=gen).tolist()
    _check_attend(tk, *_attend_case(gen, new, ctx, 2, 1, 64, 16, torch.float16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,ctx,hq,hk,d,bs,tree", [
    ([64], [9000], 16, 2, 128, 128, True),          # 512 rows a head, many pieces each
    ([64, 3], [3001, 70], 40, 8, 64, 32, True),     # 320 rows: a second stream with part of them
    ([16, 5, 16], [20000, 300, 0], 8, 1, 128, 16, True),  # one full row tile
    ([1], [33333], 6, 1, 64, 64, False), ([1] * 3, [9000, 8000, 40], 4, 4, 128, 16, False),
    ([500, 0, 37], [2000, 50, 0], 8, 2, 64, 64, False), ([1000], [0], 3, 1, 128, 16, False)])
def test_attend_divided(tk, dtype, new, ctx, hq, hk, d, bs, tree):
    """Caches long enough to be divided over the GPU, and units joined again; oracle in 64 bits on the GPU."""
    gen = torch.Generator().manual_seed(sum(ctx) + d)
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, d, bs, dtype)
    masks = _tree_masks(gen, new) if tree else None
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    cache, ws = tk.KVCache(c(k), c(v)), tk.KVWorkspace()
    got, lse = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), max_new=max(new), lse=True)
    ws.status()
    again = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), max_new=max(new))
    assert torch.equal(got, again)  # the order of the CTAs changes nothing
    for r, (n, x) in enumerate(zip(new, ctx)):
        if not n:
            continue
        place = torch.arange(x + n)
        rows = table[r].long()[place // bs]
        kk, vv = (c(y[rows, :, place % bs]).double() for y in (k, v))
        i, j = torch.arange(n)[:, None], place[None] - x
        seen = j <= i if masks is None else (j < 0) | ((masks[int(off[r]):int(off[r]) + n, None] >> j.clamp(min=0)) & 1 != 0)
        for h in range(hq):
            qq = c(q[int(off[r]):int(off[r]) + n, h]).double()
            s = (qq @ kk[:, h * hk // hq].T * d ** -0.5).masked_fill(~c(seen), -np.inf)
            w = torch.softmax(s, 1)
            o, a = w @ vv[:, h * hk // hq], w @ vv[:, h * hk // hq].abs()
            big = ((qq.abs() @ kk[:, h * hk // hq].abs().T).max(1).values * d ** -0.5)[:, None]
            tol = 1.02 * U[dtype] * (o.abs() + a) + 2.0 ** -15 * (1 + big) * a + 2.0 ** -24
            if dtype == torch.float16:
                tol = tol + (x + n) * 2.0 ** -24 * vv.abs().max()
            at = slice(int(off[r]), int(off[r]) + n)
            _close(got[at, h], o.cpu(), tol.cpu(), (r, h))
            err = (lse[at, h].double() - torch.logsumexp(s, 1)).abs()
            assert bool((err <= 2.0 ** -16 * (1 + big[:, 0])).all())


@pytest.mark.gpu
def test_attend_offsets_that_contradict_each_other(tk):
    """Nothing outside the buffers is touched, and the status tells."""
    gen = torch.Generator().manual_seed(12)
    q, k, v, off, lens, table = _attend_case(gen, [3, 2, 4], [20, 30, 10], 4, 2, 64, 16, torch.bfloat16)
    cache, ws = tk.KVCache(k.cuda(), v.cuda()), tk.KVWorkspace()
    for bad in ([0, 3, 1, 9], [-5, 3, 5, 9], [0, 3, 1 << 40, 9], [9, 6, 3, 0]):
        guard = torch.full((9 + 64, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.attend(q.cuda(), torch.tensor(bad, device="cuda"), lens.cuda(), table.cuda(), ws, out=guard[32:41])
        with pytest.raises(tk.TkError):
            ws.status()
        assert bool((guard[:32] == 7).all()) and bool((guard[41:] == 7).all())
    many = torch.tensor([0, 9] * 9000 + [0], device="cuda")  # requests over each other
    ln = torch.full((18000,), 9, dtype=torch.int32, device="cuda")
    cache.attend(q.cuda(), many, ln, torch.zeros(18000, 3, dtype=torch.int32, device="cuda"), ws)
    with pytest.raises(tk.TkError):
        ws.status()


@pytest.mark.gpu
def test_attend_long_cache_past_32_bits(tk):
    """Blocks more than 2^31 elements into the pool, and a request of 70,001 tokens."""
    bs, hk, d, n = 128, 2, 128, 3
    blocks = (1 << 31) // (hk * bs * d) + 600
    gen = torch.Generator(device="cuda").manual_seed(8)
    k = torch.empty(blocks, hk, bs, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    L = 70001
    used = -(-L // bs)
    table = torch.arange(blocks - 1, blocks - 1 - used, -1, dtype=torch.int32, device="cuda")[None]
    lo = blocks - used
    k[lo:].normal_(generator=gen)
    v[lo:].normal_(generator=gen)
    q = torch.randn(n, 4, d, generator=gen, device="cuda").bfloat16() * 2
    off, lens = torch.tensor([0, n], device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    cache, ws = tk.KVCache(k, v), tk.KVWorkspace()
    got = cache.attend(q, off, lens, table, ws).double()
    ws.status()
    kk = k[lo:].flip(0).transpose(0, 1).reshape(hk, -1, d)[:, :L].double()
    vv = v[lo:].flip(0).transpose(0, 1).reshape(hk, -1, d)[:, :L].double()
    for i in range(n):
        for h in range(4):
            s = kk[h // 2, :L - n + i + 1] @ q[i, h].double() * d ** -0.5
            w = torch.softmax(s, 0)
            o, a = w @ vv[h // 2, :L - n + i + 1], w @ vv[h // 2, :L - n + i + 1].abs()
            big = (kk[h // 2].abs() @ q[i, h].double().abs()).max() * d ** -0.5
            _close(got[i, h], o, (1.02 * U[torch.bfloat16] * (o.abs() + a) + 2.0 ** -15 * (1 + big) * a).cpu(), (i, h))


@pytest.mark.gpu
def test_plan_append_attend_in_a_graph(tk):
    """The three calls captured into one CUDA graph and replayed on new contents."""
    gen = torch.Generator().manual_seed(11)
    R, bs, hq, hk, d, W = 3, 16, 4, 2, 64, 8
    table0 = torch.tensor([[0, 1] + [-1] * 6, [2] + [-1] * 7, [-1] * 8], dtype=torch.int32, device="cuda")
    free = torch.arange(3, 20, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 4, 5, 9], device="cuda")
    ctx = torch.tensor([30, 3, 0], dtype=torch.int32, device="cuda")
    par = torch.tensor([-1, 0, 0, 1, -1, -1, 0, 1, 1], dtype=torch.int32, device="cuda")
    pool = torch.randn(2, 20, hk, bs, d, generator=gen).bfloat16().cuda()
    qkv = torch.randn(9, (hq + 2 * hk) * d, generator=gen).bfloat16().cuda()
    rope, cache, ws = tk.rope_table(64, d), tk.KVCache(pool[0], pool[1]), tk.KVWorkspace()
    table = table0.clone()

    def step():
        p = tk.kv_plan(off, ctx, table, free, bs, 9, parents=par)
        q = cache.append(qkv, p.positions, p.slots, hq, rope=rope)
        return cache.attend(q, off, p.lengths, table, ws, masks=p.masks)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for trial in range(3):
        qkv.copy_(torch.randn(9, (hq + 2 * hk) * d, generator=gen).bfloat16())
        table.copy_(table0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        table.copy_(table0)
        assert torch.equal(step(), got), trial

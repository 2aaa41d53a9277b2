"""The paged cache in 8 bits (KVCache over float8_e4m3fn blocks): storing rows with a scale for each block and head,
and attention over them, against plain forms in 64 bits."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_kv import SHAPES, TYPES, U, _append_oracle, _attend_case, _close, _tree_masks  # noqa: E402
from test_kv_ranges import host, host_inputs, on_cuda, tk  # noqa: E402,F401
from test_kv_window import windowed_oracle  # noqa: E402

E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -100


def to_e4m3(x):
    """Round to nearest, ties to even, of 64-bit values up to 448; infinities and NaN are NaN."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6)
    step = torch.exp2(e - 3)
    y = torch.round(a / step) * step  # of a whole number of steps
    return torch.where(torch.isfinite(x), torch.sign(x) * y, float("nan"))


def least_scale(top):
    """The least power of two, 2^-100 at least, of which `top` is no more than 448 times."""
    s = LEAST
    while top > 448 * s:
        s *= 2
    return s


def test_rounding_of_the_oracle():
    """Every e4m3 value, the middle of each two, and what lies next to that."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(E4M3).double()
    assert torch.equal(to_e4m3(v), v) and torch.equal(to_e4m3(-v), -v)
    mid = (v[1:] + v[:-1]) / 2
    even = torch.where(torch.arange(126) % 2 == 0, v[:-1], v[1:])
    assert torch.equal(to_e4m3(mid), even)
    assert torch.equal(to_e4m3(mid * (1 + 1e-9)), v[1:]) and torch.equal(to_e4m3(mid * (1 - 1e-9)), v[:-1])
    assert least_scale(0.0) == LEAST and least_scale(448.0) == 1.0 and least_scale(448.1) == 2.0 and least_scale(1.0) == 2.0 ** -8


# ------------------------------------------------------------------ refusals

def test_create8_refusals_are_host_side():
    from byte_level_bpe_gb300 import native
    lib = native.load()

    def create(k=1 << 20, v=1 << 20, ks=1 << 20, vs=1 << 21, type=1, stride=None):
        h = ctypes.c_void_p()
        st = (ctypes.c_int64 * 3)(*stride) if stride else None
        return lib.tk_kv_cache_create8(k, v, ks, vs, type, 4, 2, 16, 64, st, ctypes.byref(h))

    for bad in (dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(vs=1 << 20), dict(ks=(1 << 20) + 2), dict(type=3), dict(k=(1 << 20) + 8),
                dict(stride=(2048, 1024, 72)), dict(stride=(2048, 1024, 48))):
        assert create(**bad) == native.TK_E_ARG, bad


def test_cache_arguments(tk, host):
    x = host_inputs()
    k, s, z = (on_cuda(y) for y in (x["k"].to(E4M3), torch.ones(8, 2), torch.ones(8, 2)))
    tk.KVCache(k, k, s, z)
    tk.KVCache(k, k, s, z, torch.float16)
    assert [a[4] for n, a in host.calls if n == "tk_kv_cache_create8"] == [tk.native.TK_BF16, tk.native.TK_F16]
    seen = len(host.calls)
    for bad in (lambda: tk.KVCache(k, k), lambda: tk.KVCache(k, k, s), lambda: tk.KVCache(k, k, s, z, torch.float32),
                lambda: tk.KVCache(k, k, s, on_cuda(s.half())), lambda: tk.KVCache(k, k, s, on_cuda(torch.ones(8, 3))),
                lambda: tk.KVCache(k, k, on_cuda(torch.ones(2, 8)).t(), s), lambda: tk.KVCache(k, x["v"], s, z),
                lambda: tk.KVCache(k, k, s, s), lambda: tk.KVCache(x["k"], x["v"], s, z),
                lambda: tk.KVCache(x["k"], x["v"], dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    assert [n for n, _ in host.calls[seen:] if "free" not in n] == []
    with pytest.raises(ValueError):  # rows and queries have the cache's dtype
        tk.KVCache(k, k, s, z, torch.float16).append(x["qkv"], x["pos"], x["slots"], x["hq"])


def test_scales_that_require_a_gradient_are_refused(tk, host):
    x = host_inputs()
    k, z = on_cuda(x["k"].to(E4M3)), on_cuda(torch.ones(8, 2))
    cache, ws = tk.KVCache(k, k, on_cuda(torch.ones(8, 2).requires_grad_()), z), tk.KVWorkspace()
    calls = (lambda: cache.append(x["qkv"], x["pos"], x["slots"], x["hq"]),
             lambda: cache.attend(x["q"], x["off"], x["ctx"], x["table"], ws))
    for call in calls:
        with pytest.raises(ValueError):
            call()
        with torch.no_grad():
            call()


def test_side_streams_keep_the_scales(tk, host, monkeypatch):
    """A scale is an input of the work that a side stream has queued."""
    import contextlib
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    x = host_inputs()
    k, s, z = (on_cuda(t) for t in (x["k"].to(E4M3), torch.ones(8, 2), torch.ones(8, 2)))
    cache, ws = tk.KVCache(k, k, s, z), tk.KVWorkspace()
    for call in (lambda: cache.append(x["qkv"], x["pos"], x["slots"], x["hq"], stream="side"),
                 lambda: cache.attend(x["q"], x["off"], x["ctx"], x["table"], ws, stream="side")):
        type(s).used.clear()
        call()
        assert {s.data_ptr(), z.data_ptr()} <= {p for p, _ in type(s).used}


# -------------------------------------------------------------------- append

def store_oracle(old, scale, y, tol, slots, bs):
    """Values and scales of a pool [n, hk, bs, d] after rows y [T, hk, d] went to their slots, in 64 bits: (bytes' values
    before the rounding, their tolerance, scales). tol: how far y may be off in fp32."""
    want, near, scale = old.clone(), torch.zeros_like(old), scale.clone()
    blocks = {}
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < old.shape[0] * bs:
            blocks.setdefault(s // bs, []).append((t, s % bs))
    for b, rows in blocks.items():
        for h in range(old.shape[1]):
            v = torch.cat([y[t, h] for t, _ in rows])
            v = v[torch.isfinite(v)].abs()
            need = least_scale(float(v.max()) if v.numel() else 0.0)
            s = need if any(p == 0 for _, p in rows) else max(need, float(scale[b, h]))
            if s != float(scale[b, h]) and not any(p == 0 for _, p in rows):
                want[b, h] = to_e4m3(old[b, h] * (float(scale[b, h]) / s))
            scale[b, h] = s
            for t, p in rows:
                want[b, h, p] = y[t, h] / s
                near[b, h, p] = tol[t, h] / s
    return want, near, scale


def _e4m3_close(got, want, near, what):
    """Rounded values: half a step (2^-4, of what is under e4m3's least normal one 2^-10) and what fp32 may be off."""
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), ~torch.isfinite(want)), what
    fine = torch.isfinite(want)
    e = torch.floor(torch.log2(torch.where(fine & (want != 0), want.abs(), 1.0))).clamp(min=-6)
    tol = torch.where(near > 0, torch.exp2(e - 4) * (1 + 1e-9) + 1.1 * near, torch.zeros_like(near))
    err = torch.where(fine, (got - want).abs(), torch.zeros_like(want))
    assert bool((err <= tol.nan_to_num(posinf=0)).all()), (what, float((err - tol).max()))


CASES = [  # new tokens and cached ones of each request, heads, head_dim, rotated, neighbours, block, norm, layout
    ([1], [0], 1, 1, 16, 16, False, 16, True), ([1, 1, 1], [5, 15, 16], 4, 2, 64, 64, False, 16, True),
    ([33], [0], 7, 7, 64, 32, True, 32, True), ([3, 0, 40, 17], [30, 9, 0, 63], 20, 4, 96, 96, False, 16, False),
    ([130], [7], 8, 1, 128, 128, True, 64, True), ([70, 300], [50, 127], 12, 3, 128, 64, False, 128, True),
    ([1] * 64, list(range(64)), 32, 8, 128, 128, False, 16, True), ([3], [1], 2, 2, 256, 256, False, 16, True),
    ([19, 200], [100, 3], 6, 2, 240, 112, True, 128, True), ([11], [4], 5, 1, 80, 0, False, 16, True),
    ([2], [14], 1, 1, 48, 48, True, 16, False), ([700, 2, 900], [0, 33, 70], 3, 1, 112, 112, False, 32, True),
    # more rows times key heads than a decode step has: runs of four warps, of one row, of a block, of more than stay in registers
    ([150, 1, 1, 1, 90, 160], [0, 5, 63, 64, 70, 3], 16, 8, 128, 128, False, 64, True), ([1] * 320, [7] * 320, 8, 8, 64, 64, True, 16, True),
    ([300, 0, 40], [100, 5, 127], 8, 8, 256, 128, False, 128, True), ([200, 140], [0, 31], 10, 10, 96, 32, True, 32, False),
    ([2600], [3], 1, 1, 16, 0, False, 128, True),
    # so many that a run's heads are taken two at a time, the last key head with the first of the values
    ([1000, 240], [5, 17], 63, 63, 16, 16, True, 32, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(tk, dtype, case):
    new, ctx, hq, hk, d, rot, neighbours, bs, norm = CASES[case]
    gen = torch.Generator().manual_seed(case)
    T, wide = sum(new), (hq + 2 * hk) * d
    used = [-(-(c % bs + n) // bs) for c, n in zip(ctx, new)]
    blocks = sum(used) + 2
    ids = torch.randperm(blocks, generator=gen)
    slots, at = [], 0
    for n, c, u in zip(new, ctx, used):
        slots += [int(ids[at + (c % bs + i) // bs]) * bs + (c % bs + i) % bs for i in range(n)]
        at += u
    slots = torch.tensor(slots, dtype=torch.int64)
    if T > 40:  # rows without a place, between requests and at the end
        slots[T - 3] = -1
        slots[T - 2], slots[T - 1] = blocks * bs, 1 << 40
    pad = 8 * (T % 3)
    store = (torch.randn(T, wide + pad, generator=gen) * torch.exp(2 * torch.randn(T, 1, generator=gen))).to(dtype)
    x = store[:, :wide]
    tokens_first = d % 32 == 0  # the cache laid out [block][token][head] instead
    pool = (60 * torch.randn(2, blocks, bs, hk, d, generator=gen)).clamp(-448, 448).to(E4M3)
    kv = [pool[i].cuda().transpose(1, 2) if tokens_first else pool[i].reshape(blocks, hk, bs, d).cuda() for i in (0, 1)]
    before = [c.double().cpu() for c in kv]
    scales = torch.exp2(torch.randint(-9, 3, (2, blocks, hk), generator=gen).float())
    scales[:, ::3] *= 1.25  # the user's own need be no power of two
    on = [s.cuda().contiguous() for s in scales]
    pos = torch.randint(0, 500, (T,), generator=gen).int()
    rope = tk.rope_table(500, rot) if rot else None
    if T > 6:
        pos[5], pos[6] = -1, 500
    g = [1 + 0.3 * torch.randn(d, generator=gen) for _ in range(2)] if norm else [None, None]
    cache = tk.KVCache(kv[0], kv[1], on[0], on[1], dtype)
    q = cache.append(store.cuda()[:, :wide], pos.cuda(), slots.cuda(), hq, q_gain=g[0].cuda() if norm else None,
                     k_gain=g[1].cuda() if norm else None, rope=rope, eps=1e-5, neighbours=neighbours)
    y, size = _append_oracle(x, hq, hk, d, g[0], g[1], 1e-5, rope.cpu() if rot else None, pos, neighbours)
    tol = 2.0 ** -17 * size + 2.0 ** -25
    _close(q, y[:, :hq], (1.02 * U[dtype] * y.abs().nan_to_num() + tol)[:, :hq], "q")
    tol[:, hq + hk:] = 2.0 ** -30 * y[:, hq + hk:].abs() + 1e-300  # values are only scaled
    for i, first in enumerate((hq, hq + hk)):
        want, near, scale = store_oracle(before[i], scales[i].double(), y[:, first:first + hk], tol.nan_to_num()[:, first:first + hk], slots, bs)
        # the largest of a block within fp32's error of 448 times a power of two may go either way: not in these cases
        assert torch.equal(on[i].double().cpu(), scale), "kv"[i]
        _e4m3_close(kv[i], want, near, "kv"[i])


@pytest.mark.gpu
def test_append_of_extremes(tk):
    """Zeros, infinities, NaN, the largest and the smallest values, a block that begins anew, and nothing at all."""
    d, hq, hk, bs = 64, 1, 1, 16
    k, v = (torch.full((3, hk, bs, d), 1.0, device="cuda").to(E4M3) for _ in "kv")
    ks, vs = torch.full((3, hk), 4.0, device="cuda"), torch.full((3, hk), float("nan"), device="cuda")
    cache = tk.KVCache(k, v, ks, vs)
    T = 4
    x = torch.zeros(T, 3 * d, dtype=torch.bfloat16, device="cuda")
    x[1, d] = float("inf")
    x[1, d + 1] = float("nan")
    x[1, 2 * d:] = 3e38
    x[2, 2 * d] = 2.0 ** -126
    slots = torch.tensor([0, 17, 32, -1], device="cuda")  # blocks 0 and 2 begin, block 1 goes on
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    vs[1] = 1.0
    cache.append(x, pos, slots, hq)
    assert ks.flatten().tolist() == [LEAST, 4.0, LEAST]
    f = lambda c: c.float().cpu()  # noqa: E731
    assert bool((f(k)[0, 0, 0] == 0).all()) and bool((f(k)[0, 0, 1:] == 1).all())
    got = f(k)[1, 0, 1]
    assert bool(torch.isnan(got[:2]).all()) and bool((got[2:] == 0).all()) and bool((f(k)[1, 0, 2:] == 1).all())
    assert vs.flatten().tolist() == [LEAST, 2.0 ** 120, LEAST]
    big = f(v)[1, 0, 1] * 2.0 ** 120
    assert bool(((big - x[1, 2 * d].float().cpu()).abs() <= 2.0 ** -4 * 3e38).all())
    assert bool((f(v)[1, 0, 0] == 0).all())  # 2^-120 of the new scale
    assert bool((f(v)[2, 0, 0] == 0).all())  # 2^-26 of the least scale
    state = [c.view(torch.uint8).clone() for c in (k, v)] + [ks.clone(), vs.clone()]
    empty = cache.append(x[:0], pos[:0], slots[:0], hq)
    assert empty.shape == (0, hq, d)
    cache.append(x, pos, torch.full_like(slots, -1), hq)
    assert all(torch.equal(a, b) for a, b in zip(state, [k.view(torch.uint8), v.view(torch.uint8), ks, vs]))


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 100])
def test_append_in_any_order_of_places(tk, heads):
    """A block's rows follow one another in the call, in any order of their places: whole blocks backwards, and every other place."""
    d, bs, gen = 16, 32, torch.Generator().manual_seed(heads)
    slots = torch.tensor(list(range(63, 31, -1)) + list(range(97, 128, 2)) + [5], dtype=torch.int64)
    T = len(slots)
    x = (torch.randn(T, 3 * heads * d, generator=gen) * torch.exp(2 * torch.randn(T, 1, generator=gen))).half()
    pool = (60 * torch.randn(2, 5, heads, bs, d, generator=gen)).clamp(-448, 448).to(E4M3).cuda()
    before, scales = pool.double().cpu(), torch.exp2(torch.randint(-9, 0, (2, 5, heads), generator=gen).float())
    on = [s.cuda().contiguous() for s in scales]
    tk.KVCache(pool[0], pool[1], *on, torch.float16).append(x.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"), slots.cuda(), heads)
    y = x.double().view(T, 3, heads, d)
    for i in (0, 1):
        want, near, scale = store_oracle(before[i], scales[i].double(), y[:, 1 + i], 2.0 ** -30 * y[:, 1 + i].abs() + 1e-300, slots, bs)
        assert torch.equal(on[i].double().cpu(), scale)
        _e4m3_close(pool[i], want, near, i)


@pytest.mark.gpu
def test_append_goes_by_no_order(tk):
    """The same call twice gives the same bits, alone and captured."""
    d, hk, bs, T = 128, 4, 32, 900
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(T, 3 * hk * d, generator=gen, device="cuda").bfloat16()
    slots, pos = torch.arange(T, device="cuda") + 5, torch.arange(T, device="cuda").int()
    rope, gain = tk.rope_table(T, d), torch.rand(d, generator=gen, device="cuda")
    start = (60 * torch.randn(2, 30, hk, bs, d, generator=gen, device="cuda")).clamp(-448, 448).to(E4M3).view(torch.uint8)
    pool, scales = start.clone(), torch.full((2, 30, hk), 2.0 ** -9, device="cuda")
    cache = tk.KVCache(pool[0].view(E4M3), pool[1].view(E4M3), scales[0], scales[1])

    def step():
        return cache.append(x, pos, slots, hk, q_gain=gain, k_gain=gain, rope=rope)

    q = step()
    want = pool.clone(), scales.clone(), q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = step()
    for _ in range(3):
        pool.copy_(start)
        scales.fill_(2.0 ** -9)
        graph.replay()
        assert torch.equal(pool, want[0]) and torch.equal(scales, want[1]) and torch.equal(q, want[2])


@pytest.mark.gpu
def test_append_in_pieces(tk):
    """A prompt stored at once and token by token: the same scales, and values no more than the repeated roundings apart."""
    d, hk, bs, T = 128, 2, 32, 70
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn(T, 3 * hk * d, generator=gen) * torch.exp(torch.randn(T, 1, generator=gen))).bfloat16().cuda()
    pools = []
    for cuts in ([0, T], list(range(T + 1)), [0, 5, 40, 69, 70]):
        k, v = (torch.zeros(4, hk, bs, d, device="cuda").to(E4M3) for _ in "kv")
        ks, vs = (torch.zeros(4, hk, device="cuda") for _ in "kv")
        cache = tk.KVCache(k, v, ks, vs)
        slots = torch.arange(T, device="cuda") + bs  # blocks 1 to 3
        for a, b in zip(cuts, cuts[1:]):
            cache.append(x[a:b], torch.zeros(b - a, dtype=torch.int32, device="cuda"), slots[a:b].contiguous(), hk)
        pools.append((v.float() * vs[..., None, None], vs.clone(), ks.clone()))
    want = x[:, 2 * hk * d:].view(T, hk, d).float()
    for value, vs, ks in pools:
        assert torch.equal(vs, pools[0][1]) and torch.equal(ks, pools[0][2]) and bool((vs[0] == 0).all())
        got = value[1:].transpose(1, 2).reshape(-1, hk, d)[:T]
        # a value is rounded at most once in e4m3's normal range, and once more for each scale under which it is below it
        step = vs[1:].repeat_interleave(bs, 0)[:T, :, None] * 2.0 ** -9
        assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + step).all())


# -------------------------------------------------------------------- attend

def _in_8_bits(x, scale):
    """[n, hk, bs, d] with NaN -> (bytes, values in 64 bits)"""
    y = to_e4m3((x.double() / scale.double()[..., None, None]).clamp(-448, 448))
    return y.to(torch.float32).to(E4M3), y * scale.double()[..., None, None]


def case8(gen, new, ctx, hq, hk, d, bs, dtype, spread=1.0, **kw):
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, d, bs, dtype, **kw)
    scales = [torch.exp2(torch.round(spread * torch.randn(k.shape[:2], generator=gen)) - 7) for _ in "kv"]
    scales[0] = scales[0] * 1.3  # no power of two
    factor = scales[1] * 2.0 ** 7
    (k8, k), (v8, v) = _in_8_bits(k.double(), scales[0]), _in_8_bits(v.double() * factor[..., None, None].double(), scales[1])
    return q, (k8, v8, *scales), k, v, off, lens, table


def check8(tk, q, eight, k, v, off, lens, table, masks=None, scale=None, max_new=None, window=None, sinks=0, ws=None, want=None):
    dtype, d = q.dtype, q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o, lse, a, big = want or windowed_oracle(q, k, v, off, lens, table, scale, masks, window, sinks)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    k8, v8, ks, vs = (c(x) for x in eight)
    cache = tk.KVCache(k8, v8, ks, vs, dtype)
    ws = ws or tk.KVWorkspace()
    kind = dict(masks=c(masks), scale=scale, window=window, sinks=sinks)
    got, got_lse = cache.attend(c(q), c(off), c(lens), c(table), ws, max_new=max_new, lse=True, **kind)
    ws.status()
    # the result's rounding; the weights' to fp16 (half a step, and those lost below 2^-31 of the largest scaled one);
    # fp32 sums and exponents of scores as large as `big`
    n = float(lens.max()) if len(lens) else 0.0
    tol = 1.02 * U[dtype] * o.abs() + (1.02 * 2.0 ** -11 + 2.0 ** -15 * (1 + big[..., None])) * a + 2.0 ** -24
    tol = tol + n * 2.0 ** -24 * v[~torch.isnan(v)].abs().max().double()
    tol = tol.nan_to_num()  # of results that are NaN
    _close(got, o, tol, "out")
    fin = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got_lse.cpu()), torch.isneginf(lse))
    assert bool(((got_lse.cpu().double() - lse).abs()[fin] <= (2.0 ** -16 * (1 + big))[fin]).all())
    again = cache.attend(c(q), c(off), c(lens), c(table), ws, max_new=max_new, **kind)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))  # the same bits
    _close(cache.attend(c(q), c(off), c(lens), c(table), ws, **kind), o, tol, "no max_new")
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attend(tk, dtype, d, tree, shape):
    new, ctx, hq, hk, bs = SHAPES[shape]
    gen = torch.Generator().manual_seed(300 * shape + d)
    case = case8(gen, new, ctx, hq, hk, d, bs, dtype)
    check8(tk, *case, masks=_tree_masks(gen, new) if tree else None, max_new=max(new))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,ctx,hq,hk,d,bs", [([300], [0], 2, 1, 64, 16), ([129, 257, 1], [77, 0, 400], 4, 2, 128, 64),
                                                ([40], [1300], 8, 1, 128, 128)])
def test_attend_chunks_of_prompts(tk, dtype, new, ctx, hq, hk, d, bs):
    gen = torch.Generator().manual_seed(sum(new))
    check8(tk, *case8(gen, new, ctx, hq, hk, d, bs, dtype), max_new=max(new))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,hq", [([1, 1], 3), ([9, 2], 3), ([40, 64], 3)])
def test_attend_scales_far_apart(tk, d, new, hq):
    """Values' scales of neighbouring blocks up to 2^40 apart, zeros among them, and queries from 2^-30 to 2^30."""
    gen = torch.Generator().manual_seed(d + sum(new))
    q, (k8, v8, ks, vs), k, v, off, lens, table = case8(gen, new, [200, 333], hq, 1, d, 16, torch.bfloat16, poison=False)
    e = torch.randint(-20, 21, vs.shape, generator=gen).float()
    e[::5] = -float("inf")
    new_vs = torch.exp2(e)
    v = v8.double() * new_vs.double()[..., None, None]
    f = torch.exp2(torch.randint(-30, 31, (q.shape[0], hq, 1), generator=gen).float())
    q = (q.float() * f).bfloat16()
    # scores of the large queries are large too: their scale brings them back
    for lo, hi in ((-31, 0), (0, 31)):
        part = ((f >= 2.0 ** lo) & (f < 2.0 ** hi))
        check8(tk, torch.where(part, q, 0), (k8, v8, ks, new_vs), k, v, off, lens, table, scale=d ** -0.5 * (1.0 if lo < 0 else 2.0 ** -26),
               max_new=max(new))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [1, 4, 24])
@pytest.mark.parametrize("ctx", [0, 100, 120, 256])
def test_attend_hidden_nonfinite(tk, d, hq, ctx):
    """NaN in keys and values that a row does not see have no influence on it; seen ones have."""
    gen = torch.Generator().manual_seed(ctx + d)
    n = 9
    q, (k8, v8, ks, vs), k, v, off, lens, table = case8(gen, [n, 1], [ctx, 40], hq, 1, d, 16, torch.bfloat16)
    place = ctx + 6  # seen by the last three new tokens only
    b, s = int(table[0, place // 16]), place % 16
    for pool, bytes_, cols in ((v, v8, [3, d - 1]),):
        pool[b, 0, s, cols] = float("nan")
        bytes_.view(torch.uint8)[b, 0, s, cols] = 0x7f
    got = check8(tk, q, (k8, v8, ks, vs), k, v, off, lens, table, max_new=n)
    assert not bool(torch.isnan(got[:6]).any()) and bool(torch.isnan(got[6:9][:, :, [3, d - 1]]).all())
    k[b, 0, s, 0] = float("nan")
    k8.view(torch.uint8)[b, 0, s, 0] = 0xff
    got = check8(tk, q, (k8, v8, ks, vs), k, v, off, lens, table, max_new=n)
    assert not bool(torch.isnan(got[:6]).any()) and bool(torch.isnan(got[6:9]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,ctx,hq,hk,d,bs,tree", [
    ([1], [9000], 1, 1, 64, 16, False), ([1], [5000], 8, 1, 128, 16, False), ([5], [7000], 4, 1, 128, 64, True),
    ([1, 1, 1], [4000, 10, 2500], 2, 2, 64, 128, False), ([33], [3000], 4, 2, 128, 32, True), ([90], [2500], 4, 1, 64, 64, False)])
def test_attend_divided(tk, dtype, new, ctx, hq, hk, d, bs, tree):
    """Long caches, divided over workers that one of them joins."""
    gen = torch.Generator().manual_seed(sum(ctx))
    case = case8(gen, new, ctx, hq, hk, d, bs, dtype)
    check8(tk, *case, masks=_tree_masks(gen, new) if tree else None, max_new=max(new))


@pytest.mark.gpu
@pytest.mark.parametrize("hi", [2, 30])
def test_attend_many_requests(tk, hi):
    """More requests than a block has threads; empty ones among them."""
    gen = torch.Generator().manual_seed(6)
    R = 1500 if hi == 2 else 300
    new = torch.randint(0, hi, (R,), generator=gen).tolist()
    ctx = torch.randint(0, 60, (R,), generator=gen).tolist()
    check8(tk, *case8(gen, new, ctx, 2, 1, 64, 16, torch.float16), max_new=hi)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 40])
def test_long_cache_past_32_bits(tk, n):
    """Blocks more than 2^32 elements into the pool, stored there and read, by a request of 70,001 tokens; with a window too."""
    bs, hk, d = 128, 2, 128
    blocks = (1 << 32) // (hk * bs * d) + 600
    gen = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.empty(blocks, hk, bs, d, dtype=E4M3, device="cuda") for _ in "kv")
    ks, vs = (torch.full((blocks, hk), float("nan"), device="cuda") for _ in "kv")
    L = 70001
    used = -(-L // bs)
    table = torch.arange(blocks - 1, blocks - 1 - used, -1, dtype=torch.int32, device="cuda")[None]
    place = torch.arange(L, device="cuda")
    slots = table[0].long()[place // bs] * bs + place % bs
    qkv = torch.randn(L, (4 + 2 * hk) * d, generator=gen, device="cuda").bfloat16()
    cache, ws = tk.KVCache(k, v, ks, vs), tk.KVWorkspace()
    q = cache.append(qkv, place.int(), slots, 4)[-n:].contiguous()
    assert torch.equal(q, qkv[-n:, :4 * d].view(n, 4, d))
    off, lens = torch.tensor([0, n], device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    lo = blocks - used
    values = [(x[lo:].float() * s[lo:, :, None, None]).flip(0).transpose(0, 1).reshape(hk, -1, d)[:, :L].double() for x, s in ((k, ks), (v, vs))]
    x = qkv.view(L, -1, d).transpose(0, 1).double()
    for got, want in zip(values, (x[4:6], x[6:8])):
        assert float((got - want).norm() / want.norm()) < 2.0 ** -4
    for window in (None, 5000):
        got = cache.attend(q, off, lens, table, ws, max_new=n, window=window, sinks=0 if window is None else 7).double()
        ws.status()
        for i in range(0, n, 13):
            own = L - n + i
            seen = place <= own
            if window is not None:
                seen &= (place > own - window) | (place < 7)
            for h in range(4):
                kk, vv = (y[h // 2, seen] for y in values)
                s = kk @ q[i, h].double() * d ** -0.5
                w = torch.softmax(s, 0)
                o, a = w @ vv, w @ vv.abs()
                big = (kk.abs() @ q[i, h].double().abs()).max() * d ** -0.5
                _close(got[i, h], o, (1.02 * U[torch.bfloat16] * o.abs() + (2.0 ** -11 + 2.0 ** -15 * (1 + big)) * a + 2.0 ** -20).cpu(), (i, h))


@pytest.mark.gpu
def test_attend_padding_limits_and_bad_blocks(tk):
    """Tokens of no request give zeros, requests outside the limits too, blocks outside the cache read as zeros."""
    gen = torch.Generator().manual_seed(1)
    d, hq = 64, 4
    q, (k8, v8, ks, vs), k, v, off, lens, table = case8(gen, [2, 3, 1], [20, 40, 33], hq, 2, d, 16, torch.bfloat16)
    table[2, 0], table[2, 1] = -5, 1 << 30
    kz, vz = (torch.cat([x, torch.zeros_like(x[:1])]) for x in (k, v))
    tz = table.clone()
    tz[2, :2] = len(k)
    want, lse, _, _ = windowed_oracle(q, kz, vz, off, lens, tz, d ** -0.5, None, None, 0)
    big = torch.randn(10, hq, d, generator=gen).bfloat16()
    big[2:8] = q
    cache = tk.KVCache(k8.cuda(), v8.cuda(), ks.cuda(), vs.cuda())
    ws = tk.KVWorkspace()
    for max_new in (3, None):
        out, got_lse = cache.attend(big.cuda(), off.cuda() + 2, lens.cuda(), table.cuda(), ws, max_new=max_new, lse=True)
        ws.status()
        assert bool((out[:2] == 0).all()) and bool((out[8:] == 0).all()) and bool(torch.isneginf(got_lse[:2]).all())
        assert float((out[2:8].double().cpu() - want).abs().max()) < 0.02
        assert float((got_lse[2:8].double().cpu() - lse).abs().max()) < 1e-3
    out, got_lse = cache.attend(big.cuda(), off.cuda() + 2, lens.cuda(), table.cuda(), ws, max_new=2, lse=True)
    with pytest.raises(tk.TkError) as e:
        ws.status()
    assert e.value.code == tk.native.TK_E_LIMIT
    assert bool((out[4:7] == 0).all()) and bool(torch.isneginf(got_lse[4:7]).all()) and bool((out[2:4] != 0).any())
    # offsets that decrease
    bad = torch.tensor([0, 4, 2, 6], device="cuda")
    out = cache.attend(big.cuda(), bad, lens.cuda(), table.cuda(), ws)
    with pytest.raises(tk.TkError):
        ws.status()
    assert bool((out == 0).all())


@pytest.mark.gpu
def test_layouts_streams_and_graphs(tk):
    """Blocks laid out [token][head], rows apart, a side stream, a captured graph and two workspaces at once."""
    gen = torch.Generator().manual_seed(9)
    new, ctx, hq, hk, d, bs = [2, 5, 1], [300, 17, 900], 8, 2, 128, 32
    q, (k8, v8, ks, vs), k, v, off, lens, table = case8(gen, new, ctx, hq, hk, d, bs, torch.float16)
    plain = check8(tk, q, (k8, v8, ks, vs), k, v, off, lens, table, max_new=5)
    kt, vt = (x.cuda().view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(E4M3) for x in (k8, v8))
    cache, ws = tk.KVCache(kt, vt, ks.cuda(), vs.cuda(), torch.float16), tk.KVWorkspace()
    wide = torch.zeros(len(q), hq + 3, d, dtype=q.dtype, device="cuda")
    wide[:, :hq] = q.cuda()
    args = (off.cuda(), lens.cuda(), torch.cat([table, table], 1).cuda()[:, :table.shape[1]])
    assert torch.equal(cache.attend(wide[:, :hq], *args, ws, max_new=5), plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws2 = tk.KVWorkspace()
    other = cache.attend(wide[:, :hq], *args, ws2, max_new=5, stream=side)
    same = cache.attend(wide[:, :hq], *args, ws, max_new=5)
    side.synchronize()
    assert torch.equal(other, plain) and torch.equal(same, plain)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(plain)
    with torch.cuda.graph(graph):
        cache.attend(wide[:, :hq], *args, ws, max_new=5, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, plain)
    ws.status()


@pytest.mark.gpu
def test_from_plan_to_attention(tk):
    """Prompts, then single tokens: placed, stored in 8 bits and read, against the same in 16 bits."""
    d, hq, hk, bs, R = 64, 4, 2, 16, 3
    gen = torch.Generator("cuda").manual_seed(0)
    i32 = torch.int32
    blocks = 64
    table = torch.zeros(R, 12, dtype=i32, device="cuda")
    free = torch.randperm(blocks, generator=gen, device="cuda").to(i32)
    k8, v8 = (torch.zeros(blocks, hk, bs, d, device="cuda").to(E4M3) for _ in "kv")
    ks, vs = (torch.full((blocks, hk), float("nan"), device="cuda") for _ in "kv")  # nothing there yet
    k, v = (torch.zeros(blocks, hk, bs, d, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    eight, sixteen, ws = tk.KVCache(k8, v8, ks, vs), tk.KVCache(k, v), tk.KVWorkspace()
    rope, gains = tk.rope_table(256, d), torch.rand(2, d, generator=gen, device="cuda") + 0.5
    lengths, cursor = torch.zeros(R, dtype=i32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    for counts in ([40, 7, 93], [1, 1, 1], [1, 1, 1], [0, 5, 1], [1, 1, 1]):
        off = torch.tensor([0] + np.cumsum(counts).tolist(), device="cuda")
        T = sum(counts)
        plan = tk.kv_plan(off, lengths, table, free, bs, T, cursor=cursor)
        lengths, cursor = plan.lengths, plan.info[:1]
        qkv = torch.randn(T, (hq + 2 * hk) * d, generator=gen, device="cuda").bfloat16()
        outs = []
        for cache in (eight, sixteen):
            q = cache.append(qkv, plan.positions, plan.slots, hq, q_gain=gains[0], k_gain=gains[1], rope=rope)
            outs.append(cache.attend(q, off, plan.lengths, table, ws, max_new=max(counts)).float())
        ws.status()
        # a value is off by 2^-4 of itself at most and of random sign: a few per cent of the results' size
        assert float((outs[0] - outs[1]).norm() / outs[1].norm()) < 0.08

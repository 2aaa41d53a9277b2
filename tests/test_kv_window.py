"""Attention with a window and first tokens that stay visible (KVCache.attend with window and sinks), against a plain form
in 64 bits."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_kv import TYPES, U, _attend_case, _close, _tree_masks  # noqa: E402
from test_kv_ranges import host, host_inputs, tk  # noqa: E402,F401


def sees(place, i, n, L, mask, window, sinks):
    """Whether new token i of n sees `place` of L, one at a time."""
    ctx = L - n
    if mask is None:
        own = ctx + i
        if place > own:
            return False
        limited = True
    else:
        own = ctx + bin(mask & ((1 << n) - 1) & ~(1 << i)).count("1")
        if place >= ctx and not (mask >> (place - ctx)) & 1:
            return False
        limited = place < ctx
    return window is None or not limited or place < sinks or place > own - window


def windowed_oracle(q, k, v, off, lens, table, scale, masks=None, window=None, sinks=0):
    """(o, lse, A, S) in 64 bits as test_kv's; k, v [blocks, hk, bs, d] of any type."""
    T, hq, d = q.shape
    hk, bs = k.shape[1], k.shape[2]
    o, a = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64)
    lse = torch.full((T, hq), -np.inf, dtype=torch.float64)
    big = torch.zeros(T, hq, dtype=torch.float64)
    for r in range(len(lens)):
        n, L = int(off[r + 1] - off[r]), int(lens[r])
        place = torch.arange(L)
        rows = table[r].long()[place // bs]
        kk, vv = (x[rows, :, place % bs].double().view(L, hk, d) for x in (k, v))
        for i in range(n):
            t = int(off[r]) + i
            mask = None if masks is None else int(masks[t]) & (2 ** 64 - 1)
            seen = torch.tensor([sees(j, i, n, L, mask, window, sinks) for j in range(L)], dtype=torch.bool)
            if not bool(seen.any()):
                continue
            ks, vs = (x[seen].repeat_interleave(hq // hk, 1) for x in (kk, vv))  # [seen, hq, d]
            s = torch.einsum("jhd,hd->hj", ks, q[t].double()) * scale
            lse[t] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[t][:, None])
            o[t], a[t] = torch.einsum("hj,jhd->hd", w, vs), torch.einsum("hj,jhd->hd", w, vs.abs())
            big[t] = torch.einsum("jhd,hd->hj", ks.abs(), q[t].double().abs()).amax(1) * scale
    return o, lse, a, big


def check(tk, q, k, v, off, lens, table, masks=None, max_new=None, window=None, sinks=0):
    dtype, d = q.dtype, q.shape[2]
    scale = d ** -0.5
    o, lse, a, big = windowed_oracle(q, k, v, off, lens, table, scale, masks, window, sinks)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    cache, ws = tk.KVCache(c(k), c(v)), tk.KVWorkspace()
    kind = dict(masks=c(masks), window=window, sinks=sinks)
    got, got_lse = cache.attend(c(q), c(off), c(lens), c(table), ws, max_new=max_new, lse=True, **kind)
    ws.status()
    n = float(lens.max()) if len(lens) else 0.0
    tol = 1.02 * U[dtype] * (o.abs() + a) + 2.0 ** -15 * (1 + big[..., None]) * a + 2.0 ** -24
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -24 * v[torch.isfinite(v)].abs().max().double()
    tol = tol.nan_to_num()  # of results that are NaN
    _close(got, o, tol, "out")
    fin = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got_lse.cpu()), torch.isneginf(lse))
    assert bool(((got_lse.cpu().double() - lse).abs()[fin] <= (2.0 ** -16 * (1 + big))[fin]).all())
    again = cache.attend(c(q), c(off), c(lens), c(table), ws, max_new=max_new, **kind)
    assert torch.equal(again.view(torch.int16), got.view(torch.int16))  # the same bits
    _close(cache.attend(c(q), c(off), c(lens), c(table), ws, **kind), o, tol, "no max_new")
    return got


def test_refusals(tk, host):
    x = host_inputs()
    cache, ws = tk.KVCache(x["k"], x["v"]), tk.KVWorkspace()
    call = lambda **kw: cache.attend(x["q"], x["off"], x["ctx"], x["table"], ws, **kw)  # noqa: E731
    with pytest.raises(ValueError):
        call(sinks=4)
    call(window=7, sinks=2)
    assert host.calls[-1][0] == "tk_kv_attend_window" and host.calls[-1][1][14:16] == (7, 2)
    call()
    assert host.calls[-1][0] == "tk_kv_attend"


def test_refusals_of_the_library():
    from byte_level_bpe_gb300 import native
    lib = native.load()

    def call(window, sinks, mask=None):
        return lib.tk_kv_attend_window(None, None, None, 0, 1, None, 0, 0, 0, None, None, 0, 0, mask, window, sinks, 1.0, None, None, None)

    for window, sinks, mask, what in ((0, 0, None, b"window"), (-3, 0, None, b"window"), (5, -1, None, b"sinks"), (63, 0, 1 << 20, b"64"),
                                      (64, 0, 1 << 20, b"null"), (1, 0, None, b"null")):
        assert call(window, sinks, mask) == native.TK_E_ARG and what in lib.tk_last_error(), (window, sinks, mask)
    assert ctypes.sizeof(ctypes.c_int64) == 8


def test_oracle_without_a_window():
    """A window that covers everything is none."""
    from test_kv import attend_oracle
    gen = torch.Generator().manual_seed(0)
    new = [3, 5]
    q, k, v, off, lens, table = _attend_case(gen, new, [20, 2], 4, 2, 64, 16, torch.bfloat16)
    for masks in (None, _tree_masks(gen, new)):
        want = attend_oracle(q, k, v, off, lens, table, 0.125, masks)
        for window in (None, 23):
            got = windowed_oracle(q, k, v, off, lens, table, 0.125, masks, window)
            assert all(torch.allclose(x, y, rtol=1e-12, atol=1e-12) for x, y in zip(got, want))


WINDOWS = [(64, 0), (64, 4), (65, 1), (127, 16), (128, 130), (200, 64), (1000, 3), (2 ** 31 - 2, 1), (1 << 40, 1 << 40)]
SHAPES = [([1, 1, 1], [0, 199, 700], 4, 2, 16), ([3, 0, 17], [5, 9, 600], 4, 2, 64), ([64, 1, 33], [130, 1000, 2], 8, 1, 32),
          ([2] * 12, list(range(0, 720, 60)), 2, 2, 16), ([7, 40], [1500, 64], 5, 5, 128), ([64], [500], 20, 4, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window(tk, dtype, tree, shape, window, sinks):
    new, ctx, hq, hk, bs = SHAPES[shape]
    gen = torch.Generator().manual_seed(100 * shape + window % 97)
    d = 128 if (shape + window) % 2 else 64
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, d, bs, dtype)
    check(tk, q, k, v, off, lens, table, _tree_masks(gen, new) if tree else None, max(new), window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (33, 5), (150, 17)])
@pytest.mark.parametrize("new,ctx,hq,hk,d,bs", [([300], [0], 2, 1, 64, 16), ([129, 257, 1], [77, 0, 400], 4, 2, 128, 64), ([1, 1], [0, 90], 4, 1, 64, 16)])
def test_short_windows_of_chunks(tk, window, sinks, new, ctx, hq, hk, d, bs):
    """Windows shorter than a chunk, down to the token alone: it is its own value."""
    gen = torch.Generator().manual_seed(window + sum(new))
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, d, bs, torch.bfloat16)
    got = check(tk, q, k, v, off, lens, table, None, max(new), window, sinks)
    if (window, sinks) == (1, 0):
        place = ctx[0] + new[0] - 1
        assert torch.equal(got[new[0] - 1, 0].cpu(), v[table[0, place // bs].long(), 0, place % bs])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new,ctx,hq,tree", [([1], [500], 4, False), ([30], [500], 2, False), ([40], [700], 8, False), ([40], [700], 8, True),
                                             ([5], [130], 6, True)])
def test_nonfinite_outside_the_window(tk, dtype, new, ctx, hq, tree):
    """Keys and values outside every row's window may hold anything; those inside some rows' reach these alone."""
    gen = torch.Generator().manual_seed(new[0] + hq)
    window, sinks, bs, d = 100, 5, 16, 128
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, 1, d, bs, dtype)
    masks = _tree_masks(gen, new) if tree else None
    low = ctx[0] + 1 - window  # of the first token
    for place, what in ((sinks, np.nan), (low - 1, np.inf), (low - 2, np.nan), (low // 2, -np.inf)):
        b, s = int(table[0, place // bs]), place % bs
        k[b, 0, s], v[b, 0, s] = float("nan"), what
    got = check(tk, q, k, v, off, lens, table, masks, max(new), window, sinks)
    assert bool(torch.isfinite(got).all())
    # an infinite value that the first token sees and the last does not
    b, s = int(table[0, low // bs]), low % bs
    v[b, 0, s, 1] = float("inf")
    got = check(tk, q, k, v, off, lens, table, masks, max(new), window, sinks)
    assert bool(torch.isinf(got[0, :, 1]).all())
    if new[0] > 1 and not tree:
        assert bool(torch.isfinite(got[1:]).all())


@pytest.mark.gpu
def test_masks_that_show_nothing(tk):
    """A row whose mask is empty still sees its window of the context; without context it gives 0."""
    gen = torch.Generator().manual_seed(5)
    q, k, v, off, lens, table = _attend_case(gen, [3, 2], [0, 200], 4, 2, 64, 16, torch.bfloat16)
    masks = torch.tensor([0, 2, 0, 0, 3], dtype=torch.int64)
    got = check(tk, q, k, v, off, lens, table, masks, 3, 64, 2)
    assert bool((got[0] == 0).all()) and bool((got[2] == 0).all()) and bool((got[3] != 0).any())


@pytest.mark.gpu
@pytest.mark.parametrize("new,ctx,hq,hk", [([1], [9000], 4, 1), ([20, 1], [5000, 3000], 8, 2), ([600], [3000], 4, 1)])
def test_divided(tk, new, ctx, hq, hk):
    """Windows long enough to be divided over workers."""
    gen = torch.Generator().manual_seed(new[0])
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, 64, 64, torch.bfloat16)
    check(tk, q, k, v, off, lens, table, None, max(new), 2500, 70)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("window,sinks", [(64, 0), (65, 1), (128, 130), (200, 64), (1000, 3), (2 ** 31 - 2, 1)])
def test_window_in_8_bits(tk, dtype, tree, shape, window, sinks):
    from test_kv8 import case8, check8
    new, ctx, hq, hk, bs = SHAPES[shape]
    gen = torch.Generator().manual_seed(100 * shape + window % 97)
    case = case8(gen, new, ctx, hq, hk, 128 if (shape + window) % 2 else 64, bs, dtype)
    check8(tk, *case, masks=_tree_masks(gen, new) if tree else None, max_new=max(new), window=window, sinks=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (33, 5), (150, 17)])
def test_short_windows_in_8_bits(tk, window, sinks):
    from test_kv8 import case8, check8
    gen = torch.Generator().manual_seed(window)
    check8(tk, *case8(gen, [129, 60, 1], [77, 0, 400], 4, 2, 128, 64, torch.bfloat16), max_new=129, window=window, sinks=sinks)


@pytest.mark.gpu
def test_nonfinite_outside_the_window_in_8_bits(tk):
    from test_kv8 import case8, check8
    gen = torch.Generator().manual_seed(8)
    window, sinks, bs = 100, 5, 16
    for new, hq in ((1, 4), (30, 2)):
        q, eight, k, v, off, lens, table = case8(gen, [new], [500], hq, 1, 128, bs, torch.bfloat16)
        low = 501 - window
        for place, cols in ((sinks, slice(None)), (low - 1, slice(None)), (low - 2, slice(3, 9)), (low, slice(1, 2))):
            b, s = int(table[0, place // bs]), place % bs
            for x, x8 in ((k, eight[0]), (v, eight[1])):
                if place == low and x is k:
                    continue
                x[b, 0, s, cols] = float("nan")
                x8.view(torch.uint8)[b, 0, s, cols] = 0x7f
        got = check8(tk, q, eight, k, v, off, lens, table, max_new=new, window=window, sinks=sinks)
        assert bool(torch.isnan(got[0, :, 1]).all()) and not bool(torch.isnan(got[0, :, 2:]).any()) and not bool(torch.isnan(got[1:]).any())

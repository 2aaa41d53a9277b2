"""Corners of the paged cache in 8 bits (KVCache over float8_e4m3fn blocks), against plain forms in 64 bits."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_kv import TYPES, U, _attend_case, _close, _tree_masks  # noqa: E402
from test_kv8 import E4M3, case8, check8  # noqa: E402
from test_kv_ranges import host, host_inputs, on_cuda, tk  # noqa: E402,F401
from test_kv_window import sees  # noqa: E402


@pytest.mark.parametrize("shift", [-28, -4, 4, 28])
def test_scales_that_overlap_are_refused(shift):
    """Of 4 blocks of 2 heads: a block's scale of the values would be another's of the keys."""
    from byte_level_bpe_gb300 import native
    lib, h = native.load(), ctypes.c_void_p()
    for apart, what in ((shift, b"overlap"), (0, b"overlap")):
        rc = lib.tk_kv_cache_create8(1 << 20, 1 << 21, 1 << 22, (1 << 22) + apart, 1, 4, 2, 16, 64, None, ctypes.byref(h))
        assert rc == native.TK_E_ARG and what in lib.tk_last_error()


def test_views_of_scales_that_overlap_are_refused(tk, host):
    x = host_inputs()
    k, both = on_cuda(x["k"].to(E4M3)), on_cuda(torch.ones(20, 2))
    for a, b in ((0, 1), (7, 0), (5, 5)):
        with pytest.raises(ValueError):
            tk.KVCache(k, k, both[a:a + 8], both[b:b + 8])
    assert [n for n, _ in host.calls if "free" not in n] == []
    tk.KVCache(k, k, both[:8], both[8:16])
    tk.KVCache(k, k, both[8:16], both[:8])
    assert [n for n, _ in host.calls if "free" not in n] == ["tk_kv_cache_create8"] * 2


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,most", [(4, 4), (8, 2), (2, 8), (5, 3)])
def test_ragged_units_of_up_to_16_rows(tk, dtype, d, group, most):
    """Units of 1 to 8 rows and of 9 to 16 one after the other in every worker: a piece is not asked for its rows any more
    when the next ones may be in its place."""
    gen = torch.Generator().manual_seed(10 * group + d)
    new = torch.randint(0, most + 1, (420,), generator=gen).tolist()
    new[0] = most
    ctx = torch.randint(0, 40, (420,), generator=gen).tolist()
    q, eight, k, v, off, lens, table = case8(gen, new, ctx, 2 * group, 2, d, 16, dtype)
    got = check8(tk, q, eight, k, v, off, lens, table, max_new=most)
    c = [x.cuda() for x in eight]
    cache, ws, args = tk.KVCache(*c, dtype), tk.KVWorkspace(), [x.cuda() for x in (q, off, lens, table)]
    for _ in range(50):
        assert torch.equal(cache.attend(*args, ws, max_new=most), got)
    ws.status()


@pytest.mark.gpu
@pytest.mark.parametrize("T,heads", [(1, 1), (40, 2), (3000, 1)])
@pytest.mark.parametrize("eps", [1e-6, 2.0 ** -57, 1e-20, 1e-37])
def test_append_of_zero_keys_with_a_norm(tk, T, heads, eps):
    """0 / sqrt(0 + eps) is 0, however small eps is; rows of zeros beside others too."""
    d, bs = 64, 16
    blocks = T // bs + 2
    k, v = (torch.full((blocks, heads, bs, d), 1.0, device="cuda").to(E4M3) for _ in "kv")
    ks, vs = (torch.full((blocks, heads), 4.0, device="cuda") for _ in "kv")
    cache = tk.KVCache(k, v, ks, vs)
    x = torch.zeros(T, 3 * heads * d, dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, device="cuda") + bs
    gain = torch.full((d,), 2.0, device="cuda")
    q = cache.append(x, pos, slots, heads, q_gain=gain, k_gain=gain, eps=eps)
    rows = lambda y: y.float().transpose(1, 2).flatten(0, 1)[bs:bs + T]  # noqa: E731
    assert bool((q == 0).all()) and bool((rows(k) == 0).all()) and bool((rows(v) == 0).all())
    used = slice(1, (T + bs - 1) // bs + 1)
    assert bool((ks[used] == 2.0 ** -100).all()) and bool((vs[used] == 2.0 ** -100).all()) and bool((ks[0] == 4).all())
    x[::3] = 0.5
    cache.append(x, pos, slots, heads, q_gain=gain, k_gain=gain, eps=eps)
    got = (k.float() * ks[..., None, None]).transpose(1, 2).flatten(0, 1)[bs:bs + T]
    # 0.5 / sqrt(0.25 + eps) * 2: eps at most 1e-6
    assert bool(((got[::3] - 2).abs() <= 2.0 ** -4 * 2).all())
    got[::3] = 0
    assert bool((got == 0).all())


# What a result may be off by, from the kernels' formulas: o = sum w_j v8_j / sum p_j, p_j = exp(s_j), W_j = p_j vs_j.
#   The product's weight is W_j in fp16, relative to a maximum M of the row's own W that is within 2^8 of the largest, at 2^7: half
#   a step is 2^-11 of it, or, of one that is subnormal there, 2^-25 of M / 2^7: 2^-32 of the row's largest W.
#   Exponents, of scores as large as `big` and log2 of scales up to 2^7, and sums are fp32's: 2^-15 (1 + big) of the sum of |W_j v8_j|.
#   The result is rounded once, and fp16's least step is 2^-24.
def exact_rows(q, eight, off, lens, table, scale, masks=None, window=None, sinks=0):
    """(o, tolerance, lse, big) in 64 bits of nothing but the places that a row sees."""
    k8, v8, ks, vs = (x.double() for x in eight)
    T, hq, d = q.shape
    hk, bs = k8.shape[1], k8.shape[2]
    o, tol = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64)
    lse, big = torch.full((T, hq), -float("inf"), dtype=torch.float64), torch.zeros(T, hq, dtype=torch.float64)
    for r in range(len(lens)):
        n, L = int(off[r + 1] - off[r]), int(lens[r])
        for i in range(n):
            t = int(off[r]) + i
            mask = None if masks is None else int(masks[t]) & (2 ** 64 - 1)
            seen = torch.tensor([j for j in range(L) if sees(j, i, n, L, mask, window, sinks)], dtype=torch.long)
            if not len(seen):
                continue
            b, place = table[r].long()[seen // bs], seen % bs
            for h in range(hq):
                g = h // (hq // hk)
                kk, vv = k8[b, g, place] * ks[b, g, None], v8[b, g, place]
                s = kk @ q[t, h].double() * scale
                lse[t, h] = torch.logsumexp(s, 0)
                w = torch.exp(s - lse[t, h]) * vs[b, g]
                o[t, h] = w @ vv
                big[t, h] = float((kk.abs() @ q[t, h].double().abs()).max()) * scale
                tol[t, h] = ((1.02 * 2.0 ** -11 + 2.0 ** -15 * (1 + big[t, h])) * (w @ vv.abs()) + 1.02 * 2.0 ** -32 * w.max() * vv.abs().sum(0)
                             + 1.02 * U[q.dtype] * o[t, h].abs() + (2.0 ** -25 if q.dtype == torch.float16 else 2.0 ** -134))
    return o, tol, lse, big


def exactly(tk, q, eight, off, lens, table, masks=None, max_new=None, window=None, sinks=0):
    scale = q.shape[2] ** -0.5
    o, tol, lse, big = exact_rows(q, eight, off, lens, table, scale, masks, window, sinks)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    cache, ws = tk.KVCache(*(c(x) for x in eight), q.dtype), tk.KVWorkspace()
    got, got_lse = cache.attend(c(q), c(off), c(lens), c(table), ws, masks=c(masks), max_new=max_new, lse=True, window=window, sinks=sinks)
    ws.status()
    _close(got, o, tol, "out")
    fin = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got_lse.cpu()), torch.isneginf(lse))
    assert bool(((got_lse.cpu().double() - lse).abs()[fin] <= (2.0 ** -16 * (1 + big))[fin]).all())
    return got


def spread_case(gen, new, ctx, hq, hk, d, bs, dtype):
    """Blocks that all have values of every size and the value scale 2^-16; of blocks with a larger one `loud` makes values that
    a 16-bit result can hold."""
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, hq, hk, d, bs, dtype, poison=False)
    k8, v8 = k.float().to(E4M3), (40 * v.float()).clamp(-448, 448).to(E4M3)
    ks, vs = torch.full(k.shape[:2], 0.7), torch.full(k.shape[:2], 2.0 ** -16)
    return q, (k8, v8, ks, vs), off, lens, table


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(1, 4), (3, 5), (30, 1), (150, 2)])
@pytest.mark.parametrize("scales", [(2.0 ** 127, 1.9 * 2.0 ** 127, 2.0 ** 126), (2.0 ** 127, 1.0, 2.0 ** -120), (2.0 ** -110, 1.5 * 2.0 ** -120, 0.0)])
def test_largest_and_smallest_scales(tk, d, n, group, scales):
    """Scales of every finite size, where the result is finite."""
    gen = torch.Generator().manual_seed(n)
    q, eight, off, lens, table = spread_case(gen, [n, 1], [1700, 20], group, 1, d, 16, torch.bfloat16)
    eight[1].copy_((0.01 * torch.randn(eight[1].shape, generator=gen)).clamp(-0.0625, 0.0625).to(E4M3))
    eight[3].copy_(torch.tensor(scales)[torch.randint(0, 3, eight[3].shape, generator=gen)])
    exactly(tk, q, eight, off, lens, table, max_new=n)


def loud(gen, eight, b, scale):
    _, v8, _, vs = eight
    v8[b] = torch.exp2(-8 + 4 * torch.rand(v8[b].shape, generator=gen)).to(E4M3)
    vs[b] = scale


ROWS = [(8, 1), (2, 4), (16, 1), (3, 5), (40, 2), (64, 2), (200, 1), (90, 4)]  # new tokens, query heads a key head


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", ROWS)
@pytest.mark.parametrize("ctx", [0, 14, 60, 3005])
def test_scales_of_later_blocks(tk, dtype, d, n, group, ctx):
    """A block that a chunk's later tokens begin has no influence on the earlier ones, whatever its scale."""
    gen = torch.Generator().manual_seed(n + ctx)
    q, eight, off, lens, table = spread_case(gen, [n, 1], [ctx, 33], group, 1, d, 16, dtype)
    for i, place in enumerate((ctx + 1, ctx + n // 2, ctx + n - 1)):
        if place // 16 > ctx // 16:
            loud(gen, eight, int(table[0, place // 16]), 2.0 ** (5 + 7 * i))
    exactly(tk, q, eight, off, lens, table, max_new=n)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(8, 1), (5, 3), (30, 2), (64, 4)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (70, 3)])
def test_scales_of_drafted_tokens_that_a_mask_hides(tk, d, n, group, window, sinks):
    gen = torch.Generator().manual_seed(n)
    q, eight, off, lens, table = spread_case(gen, [n, 2], [121, 0], group, 1, d, 16, torch.bfloat16)
    masks = _tree_masks(gen, [n, 2])
    for i in range(n):  # what lies in the last block is seen by few
        if 121 + i >= (120 + n) // 16 * 16:
            loud(gen, eight, int(table[0, (121 + i) // 16]), 2.0 ** 30)
    exactly(tk, q, eight, off, lens, table, masks, n, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(1, 4)] + ROWS)
@pytest.mark.parametrize("bad", [1e38, 3.4e38, float("inf"), float("nan")])
def test_scales_outside_the_window(tk, dtype, d, n, group, bad):
    """Blocks that lie between the first tokens and the window may have any scales, unset ones too; a block that the window
    leaves behind has no more influence."""
    gen = torch.Generator().manual_seed(n)
    window, sinks, ctx = 100, 5, 516
    q, eight, off, lens, table = spread_case(gen, [n, 1], [ctx, 33], group, 1, d, 16, dtype)
    low = ctx + 1 - window
    for b in range((sinks + 15) // 16, low // 16):
        for s in eight[2:]:
            s[int(table[0, b])] = bad
    if n > 1:
        loud(gen, eight, int(table[0, low // 16]), 2.0 ** 19)
    exactly(tk, q, eight, off, lens, table, None, n, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(1, 1), (1, 8), (2, 6), (9, 1), (20, 1), (50, 2), (150, 2)])
@pytest.mark.parametrize("ctx", [300, 4000])
def test_large_scales_of_small_weights(tk, d, n, group, ctx):
    """Scores and scales of blocks far apart: what counts is their product, whichever of the two is large."""
    gen = torch.Generator().manual_seed(n + group)
    q, eight, off, lens, table = spread_case(gen, [n], [ctx], group, 1, d, 16, torch.bfloat16)
    k8, v8, ks, vs = eight
    q[..., 0] = d ** 0.5  # scores are 0.7 times a key's first element, and something
    q[..., 1:] *= 0.2
    at = torch.randint(0, 4, (len(k8),), generator=gen)
    k8[..., 0] = torch.tensor([0.0, -20.0, -60.0, -88.0])[at][:, None, None].to(E4M3)
    vs[:, 0] = torch.exp2(torch.tensor([-30.0, -5.0, 0.0, 30.0, 60.0])[torch.randint(0, 5, (len(k8),), generator=gen)])
    exactly(tk, q, eight, off, lens, table, max_new=n)
    # one block has nearly all of the weight and the least scale
    first = int(table[0, 2])
    k8[..., 0] = torch.full(k8.shape[:3], -60.0).to(E4M3)
    k8[first, :, :, 0] = torch.zeros(k8.shape[1:3]).to(E4M3)
    vs[:] = 2.0 ** 30
    vs[first] = 1.0
    exactly(tk, q, eight, off, lens, table, max_new=n)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(3, 1), (4, 4), (20, 2), (64, 4)])
@pytest.mark.parametrize("window", [None, 64])
def test_rows_that_see_nothing(tk, d, n, group, window):
    """Empty masks without context give 0 and -infinity, beside rows that see some, whatever the scales of what is hidden."""
    gen = torch.Generator().manual_seed(n)
    q, eight, off, lens, table = spread_case(gen, [n, 2, n], [0, 50, 33], group, 1, d, 16, torch.bfloat16)
    masks = _tree_masks(gen, [n, 2, n])
    masks[:n:2] = 0  # of the first request
    masks[n + 2] = 0
    if n == 3:
        for s in eight[2:]:
            s[int(table[0, 0])] = 3.4e38
        masks[:n] = 0
    got = exactly(tk, q, eight, off, lens, table, masks, n, window, 2 if window else 0)
    assert bool((got[:n:2] == 0).all()) and bool((got[n + 2] != 0).any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(4, 2), (3, 5), (30, 1), (150, 2)])
def test_queries_that_are_not_finite(tk, dtype, d, n, group):
    """They make their own row's result NaN or what they make it, and leave the bits of every other row."""
    gen = torch.Generator().manual_seed(n)
    q, eight, off, lens, table = spread_case(gen, [n, 1], [700, 30], group, 1, d, 16, dtype)
    want = exactly(tk, q, eight, off, lens, table, max_new=n)
    bad = q.clone()
    bad[1, 0, 5], bad[2, group - 1, 0], bad[n, 0, 1] = float("inf"), float("nan"), -float("inf")
    cache, ws = tk.KVCache(*(x.cuda() for x in eight), dtype), tk.KVWorkspace()
    got = cache.attend(bad.cuda(), off.cuda(), lens.cuda(), table.cuda(), ws, max_new=n)
    ws.status()
    rows = torch.ones(n + 1, group, dtype=torch.bool)
    rows[1, 0] = rows[2, group - 1] = rows[n, 0] = False
    assert torch.equal(got[rows.cuda()], want[rows.cuda()]) and bool(torch.isnan(got[2, group - 1]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n,group", [(1, 4), (3, 5), (30, 2)])
def test_scales_of_zero(tk, n, group):
    """Keys' scales of 0 make all scores 0, values' the results."""
    gen = torch.Generator().manual_seed(n)
    q, eight, off, lens, table = spread_case(gen, [n, 1], [300, 30], group, 1, 128, 16, torch.bfloat16)
    eight[2].zero_()
    exactly(tk, q, eight, off, lens, table, max_new=n)
    eight[2].fill_(0.7)
    eight[3].zero_()
    assert bool((exactly(tk, q, eight, off, lens, table, max_new=n) == 0).all())

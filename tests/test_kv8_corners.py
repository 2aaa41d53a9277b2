"""Corners of the paged cache in 8 bits (KVCache over float8_e4m3fn blocks), against plain forms in 64 bits."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_kv import TYPES  # noqa: E402
from test_kv8 import E4M3, case8, check8  # noqa: E402
from test_kv_ranges import host, host_inputs, on_cuda, tk  # noqa: E402,F401


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

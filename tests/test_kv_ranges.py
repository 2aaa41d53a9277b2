"""Ranges and misuse of the paged cache calls (tk_kv_*): what must hold past the ordinary cases."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_kv import U, _attend_case, _close  # noqa: E402


@pytest.fixture(scope="module")
def tk():
    import byte_level_bpe_gb300 as tk
    return tk


class OnCuda(torch.Tensor):
    """A tensor of the host that says it is on cuda:0: for what the calls check before they reach the library."""
    is_cuda = property(lambda self: True)

    used = []

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.used.append((self.data_ptr(), stream))


def on_cuda(x):
    return x.as_subclass(OnCuda)


class Stream:
    """A side stream, for calls without a GPU."""
    cuda_stream = 4096


class Library:
    """In libtk's place: notes the calls and their arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def host(monkeypatch):
    """The calls without a GPU. host.device is the current one."""
    from byte_level_bpe_gb300 import kv, native
    lib = Library()
    lib.device = 0
    monkeypatch.setattr(kv, "_T", torch)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(kv, "_current_device", lambda: lib.device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: lib.device)
    monkeypatch.setattr(native, "load", lambda: lib)
    return lib


def host_inputs(R=3, T=6, W=4, hq=4, hk=2, d=64, bs=16):
    i32, i64 = torch.int32, torch.int64
    z = lambda *s, t=torch.bfloat16: on_cuda(torch.zeros(*s, dtype=t))  # noqa: E731
    return dict(off=z(R + 1, t=i64), ctx=z(R, t=i32), table=z(R, W, t=i32), free=z(8, t=i32), pos=z(T, t=i32),
                slots=z(T, t=i64), qkv=z(T, (hq + 2 * hk) * d), q=z(T, hq, d), k=z(8, hk, bs, d), v=z(8, hk, bs, d), T=T, hq=hq)


def test_tensors_of_another_device_are_refused(tk, host):
    """A kernel would start on the current device, ordered after nothing on the tensors'."""
    x = host_inputs()
    tk.kv_plan(x["off"], x["ctx"], x["table"], x["free"], 16, x["T"])
    cache, ws = tk.KVCache(x["k"], x["v"]), tk.KVWorkspace()
    ws.status()
    assert [name for name, _ in host.calls] == ["tk_kv_plan", "tk_kv_cache_create", "tk_kv_workspace_create", "tk_kv_status"]
    host.device = 1
    for bad in (lambda: tk.kv_plan(x["off"], x["ctx"], x["table"], x["free"], 16, x["T"]), lambda: tk.KVCache(x["k"], x["v"]),
                ws.status):
        with pytest.raises(ValueError):
            bad()
    assert len(host.calls) == 4
    host.device = 0
    del cache


def test_rows_that_overlap_are_refused(tk, host):
    """Expanded (stride 0) and overlapping tensors: packed rows in their place would lie past their storage."""
    x = host_inputs()
    cache, ws = tk.KVCache(x["k"], x["v"]), tk.KVWorkspace()
    seen = len(host.calls)

    def calls(table, qkv, q):
        return (lambda: tk.kv_plan(x["off"], x["ctx"], table, x["free"], 16, x["T"]),
                lambda: cache.attend(x["q"], x["off"], x["ctx"], table, ws),
                lambda: cache.append(qkv, x["pos"], x["slots"], x["hq"]), lambda: cache.attend(q, x["off"], x["ctx"], x["table"], ws))

    for bad in calls(x["table"][:1].expand(3, 4), x["qkv"][:1].expand(6, -1), x["q"][:1].expand(6, -1, -1)) + calls(
            x["table"].as_strided((3, 4), (2, 1)), x["qkv"].as_strided((6, 512), (64, 1)), x["q"].as_strided((6, 4, 64), (64, 64, 1))):
        with pytest.raises(ValueError):
            bad()
    assert len(host.calls) == seen
    # rows further apart are passed on, of a single or empty row no stride is taken from torch
    wide = on_cuda(torch.zeros(3, 9, dtype=torch.int32))[:, :4]
    one = x["table"][:1].expand(1, 4).as_strided((1, 4), (0, 1))
    tk.kv_plan(x["off"], x["ctx"], wide, x["free"], 16, x["T"])
    tk.kv_plan(x["off"][:2], x["ctx"][:1], one, x["free"], 16, x["T"])
    tk.kv_plan(x["off"], x["ctx"], wide[:, :0], x["free"], 16, x["T"])
    assert [args[6:8] for _, args in host.calls[seen:]] == [(9, 4), (4, 4), (0, 0)]


@pytest.mark.parametrize("out,over", [("len", "ctx"), ("info", "cur"), ("pos", "par"), ("slot", "off"), ("req", "free"), ("mask", "off"),
                                      ("len", "off")])
@pytest.mark.parametrize("shift", [-16, 0, 16])
def test_plan_outputs_over_inputs_are_refused(tk, out, over, shift):
    """In place, one CTA would write the lengths or the cursor that another has yet to read."""
    if (over, shift) == ("cur", 16):
        shift = -24  # one value: behind the first of the four
    names = ("off", "ctx", "table", "free", "cur", "par", "pos", "slot", "req", "len", "mask", "info")
    at = {name: (i + 1) << 20 for i, name in enumerate(names)}
    at[out] = at[over] + shift
    rc = tk.native.load().tk_kv_plan(at["off"], at["ctx"], 9, 40, 16, at["table"], 4, 4, at["free"], 8, at["cur"], at["par"],
                                     at["pos"], at["slot"], at["req"], at["len"], at["mask"], at["info"], None)
    assert rc == tk.native.TK_E_ARG and b"overlaps" in tk.native.load().tk_last_error()


def test_inputs_that_require_a_gradient_are_refused(tk, host):
    """A loss over the outputs would train nothing, without a word."""
    x = host_inputs()
    cache, ws = tk.KVCache(x["k"], x["v"]), tk.KVWorkspace()
    seen = len(host.calls)
    qkv, q = (on_cuda(x[name].clone().requires_grad_()) for name in ("qkv", "q"))
    gain = on_cuda(torch.ones(64).requires_grad_())
    calls = (lambda: cache.append(qkv, x["pos"], x["slots"], 4), lambda: cache.append(x["qkv"], x["pos"], x["slots"], 4, q_gain=gain),
             lambda: cache.append(x["qkv"], x["pos"], x["slots"], 4, k_gain=gain),
             lambda: cache.attend(q, x["off"], x["ctx"], x["table"], ws))
    for bad in calls:
        with pytest.raises(ValueError):
            bad()
    assert len(host.calls) == seen
    with torch.no_grad():
        for fine in calls:
            fine()
    assert len(host.calls) == seen + 4


def test_stream_argument_owns_the_outputs_and_keeps_the_inputs(tk, host, monkeypatch):
    """Without a GPU: outputs are allocated with the stream current, and every tensor touched is recorded on it."""
    x, side = host_inputs(), Stream()
    cache, ws = tk.KVCache(x["k"], x["v"]), tk.KVWorkspace()
    current, allocated, empty = [None], [], torch.empty

    class use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *e):
            current.pop()

    from byte_level_bpe_gb300 import kv
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(kv, "_raw_stream", lambda index: getattr(current[-1], "cuda_stream", 0))
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (allocated.append(current[-1]), empty(*a, **k))[1])
    gain, rope = on_cuda(torch.ones(64)), on_cuda(torch.ones(5, 32, 2))
    par, masks, cur = on_cuda(torch.zeros(6, dtype=torch.int32)), x["slots"], x["slots"][:1]
    out = on_cuda(torch.zeros_like(x["q"]))
    for call, inputs in (
            (lambda s: tk.kv_plan(x["off"], x["ctx"], x["table"], x["free"], 16, 6, parents=par, cursor=cur, stream=s),
             (x["off"], x["ctx"], x["table"], x["free"], par, cur)),
            (lambda s: cache.append(x["qkv"], x["pos"], x["slots"], 4, q_gain=gain, k_gain=gain, rope=rope, stream=s),
             (x["qkv"], x["pos"], x["slots"], gain, rope, x["k"], x["v"])),
            (lambda s: cache.append(x["qkv"], x["pos"], x["slots"], 4, out=out, stream=s), (x["qkv"], x["slots"], out)),
            (lambda s: cache.attend(x["q"], x["off"], x["ctx"], x["table"], ws, masks=masks, lse=True, stream=s),
             (x["q"], x["off"], x["ctx"], x["table"], masks, x["k"], x["v"])),
            (lambda s: cache.attend(x["q"], x["off"], x["ctx"], x["table"], ws, out=out, stream=s), (x["q"], out))):
        for stream in (None, side):
            OnCuda.used.clear()
            allocated.clear()
            call(stream)
            assert all(a is stream for a in allocated)
            assert host.calls[-1][1][-1] == (4096 if stream else 0)  # where the kernel goes
            for i in inputs:
                assert ((i.data_ptr(), side) in OnCuda.used) == (stream is side)


@pytest.mark.gpu
def test_stream_argument(tk):
    """The calls on a side stream give the same results; their outputs are that stream's, and inputs that are
    let go meanwhile are not handed out again before it is done."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    z = torch.zeros
    off, ctx = torch.tensor([0, 3, 9], device="cuda"), torch.tensor([20, 0], dtype=torch.int32, device="cuda")
    qkv = torch.randn(9, 8 * 64, generator=gen, device="cuda").bfloat16()
    free, rope, side = torch.arange(2, 30, dtype=torch.int32, device="cuda"), tk.rope_table(64, 64), torch.cuda.Stream()
    busy = torch.randn(8192, 8192, device="cuda").bfloat16()

    product = torch.empty_like(busy)

    def step(stream):
        table = z(2, 4, dtype=torch.int32, device="cuda")
        table[0, 1] = 1
        cache, ws = tk.KVCache(*z(2, 30, 2, 16, 64, dtype=torch.bfloat16, device="cuda")), tk.KVWorkspace()
        rows = qkv.clone()
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                for _ in range(300):  # some 200 ms
                    torch.mm(busy, busy, out=product)
        p = tk.kv_plan(off, ctx, table, free, 16, 9, stream=stream)
        q = cache.append(rows, p.positions, p.slots, 4, rope=rope, stream=stream)
        at, size = rows.data_ptr(), rows.shape
        del rows
        if stream is not None:
            again = torch.empty(size, dtype=torch.bfloat16, device="cuda")
            assert not side.query() and again.data_ptr() != at
        o = cache.attend(q, off, p.lengths, table, ws, stream=stream)
        ws.status(stream)
        return [p.positions, p.slots, p.info, q, o]

    want, got = step(None), step(side)
    for w, g in zip(want, got):
        assert torch.equal(w, g)
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"]}
    assert [owner[g.data_ptr()] for g in got] == [side.cuda_stream] * 5


def guarded_plan(tk, off, ctx, T, bs=16, W=3, parents=None, free=20):
    """kv_plan over a table between guard rows and columns. Returns the plan and the table; nothing outside it is written."""
    R = len(ctx)
    big = torch.full((R + 2, W + 4), 77, dtype=torch.int32, device="cuda")
    table = big[1:-1, 2:2 + W]
    table[:] = 1000 + torch.arange(R * W, device="cuda").view(R, W)
    ids = torch.full((free + 64,), 1 << 29, dtype=torch.int32, device="cuda")
    ids[32:32 + free] = torch.arange(free, device="cuda")
    i64 = torch.tensor(off, dtype=torch.int64, device="cuda")
    i32 = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    par = None if parents is None else torch.tensor(parents, dtype=torch.int32, device="cuda")
    p = tk.kv_plan(i64, i32, table, ids[32:32 + free], bs, T, parents=par)
    after = table.clone()
    table[:] = 77
    assert bool((big == 77).all())
    return p, after


@pytest.mark.gpu
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("T", [9, 3000])
@pytest.mark.parametrize("off,who", [([9, 6, 3, 0], 0), ([-5, 3, 5, 9], 0), ([0, 3, 1 << 62, 9], 2), ([0, 9, 0, 9], 1),
                                     ([-(1 << 63), (1 << 63) - 1, (1 << 63) - 1, (1 << 63) - 1], 0), ([0, 9, 8, 9], 1),
                                     ([0] + [9, 0] * 1000, 1)])
def test_plan_offsets_that_contradict_each_other(tk, off, who, T, tree):
    """Nothing is placed, nothing outside the buffers is written, and the status tells of the first."""
    R = len(off) - 1
    p, table = guarded_plan(tk, off, [2] * R, T, parents=[-1] * T if tree else None)
    assert p.info.tolist() == [0, 0, tk.native.TK_E_LIMIT, who]
    assert bool((table == 1000 + torch.arange(R * 3, device="cuda").view(R, 3)).all())
    assert bool((p.slots == -1).all()) and bool((p.requests == -1).all()) and bool((p.lengths == 2).all())


@pytest.mark.gpu
@pytest.mark.parametrize("end", [(1 << 63) - 1, (1 << 62), (1 << 32) + 5, (1 << 31) - 128 - 2, (1 << 31) - 1])
@pytest.mark.parametrize("ctx", [2, 16, (1 << 31) - 1])
def test_plan_more_tokens_than_positions(tk, end, ctx):
    """A request whose end is past 31 bits, or 63, is not placed, however its sums would wrap."""
    p, table = guarded_plan(tk, [0, end], [ctx], 5000)
    assert p.info.tolist() == [0, 0, tk.native.TK_E_LIMIT, 0] and p.lengths.tolist() == [ctx]
    assert table.tolist() == [[1000, 1001, 1002]] and bool((p.slots == -1).all())


@pytest.mark.gpu
def test_plan_with_fewer_tokens_than_the_offsets(tk):
    """Requests whose tokens got no slot are not reported as stored."""
    p, table = guarded_plan(tk, [0, 5, 30, 31], [2, 2, 2], 29)
    assert p.info.tolist() == [0, 0, tk.native.TK_E_LIMIT, 1] and p.lengths.tolist() == [7, 2, 2]
    assert p.slots.tolist() == [16 * 1000 + 2 + i for i in range(5)] + [-1] * 24
    p, table = guarded_plan(tk, [0, 5, 30, 31], [2, 16, 2], 30)
    assert p.info.tolist() == [2, 2, tk.native.TK_E_LIMIT, 2] and p.lengths.tolist() == [7, 41, 2]
    assert p.slots.tolist() == [16 * 1000 + 2 + i for i in range(5)] + list(range(25))


@pytest.mark.gpu
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("first", [1, 3, 4, 7, 2048, 5001])
def test_plan_tokens_before_the_first_request(tk, first, tree):
    """Offsets may be a part of a longer batch's: what comes before them has no slot."""
    n = [9, 0, 40, 3]
    ctx = [20, 5, 0, 31]
    off = np.cumsum([first] + n)
    T = int(off[-1]) + 6
    par = np.full(T, -1, np.int32)
    p, table = guarded_plan(tk, off.tolist(), ctx, T, W=4, parents=par.tolist() if tree else None)
    q, same = guarded_plan(tk, (off - first).tolist(), ctx, T - first, W=4, parents=par[first:].tolist() if tree else None)
    assert torch.equal(table, same) and torch.equal(p.info, q.info) and torch.equal(p.lengths, q.lengths)
    for name, none in (("positions", 0), ("slots", -1), ("requests", -1), ("masks", 0)):
        x, y = getattr(p, name), getattr(q, name)
        if x is not None:
            assert bool((x[:first] == none).all()), name
            assert torch.equal(x[first:], y), name


@pytest.mark.gpu
@pytest.mark.parametrize("first,last", [(-5, 9), (-(1 << 63), 9), (0, 12), (0, (1 << 63) - 1), (-1, 1 << 40)])
def test_attend_offsets_past_the_tokens(tk, first, last):
    """A request that reaches outside the tokens gives zeros; it writes no other one's rows."""
    gen = torch.Generator().manual_seed(5)
    new, ctx = [3, 2, 1, 3], [20, 30, 10, 300]
    q, k, v, off, lens, table = _attend_case(gen, new, ctx, 4, 2, 64, 16, torch.bfloat16)
    q, k, v, off, lens, table = (x.cuda() for x in (q, k, v, off, lens, table))
    cache, ws = tk.KVCache(k, v), tk.KVWorkspace()
    want = cache.attend(q, off, lens, table, ws)
    ws.status()
    bad = off.clone()
    bad[0], bad[-1] = first, last
    got, lse = cache.attend(q, bad, lens, table, ws, lse=True)
    with pytest.raises(tk.TkError) as e:
        ws.status()
    assert e.value.code == tk.native.TK_E_LIMIT
    for r, (a, b) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        if (r == 0 and first < 0) or (r == 3 and last > 9):
            assert bool((got[a:b] == 0).all()) and bool(torch.isneginf(lse[a:b]).all())
        else:
            assert torch.equal(got[a:b], want[a:b])


@pytest.mark.gpu
@pytest.mark.parametrize("first,behind", [(0, 1), (2, 0), (3, 500), (700, 0)])
@pytest.mark.parametrize("d,dtype,max_new", [(64, torch.bfloat16, 3), (128, torch.float16, 40), (128, torch.bfloat16, None)])
def test_attend_padding_is_zero(tk, first, behind, d, dtype, max_new):
    """Tokens before the first and after the last request, as padded batches have them; a batch of them alone."""
    gen = torch.Generator().manual_seed(6)
    q, k, v, off, lens, table = (x.cuda() for x in _attend_case(gen, [3, 0, 2], [20, 30, 500], 4, 2, d, 16, dtype))
    cache, ws = tk.KVCache(k, v), tk.KVWorkspace()
    # as many tokens: the variants, chosen by the bound on a request's, sum in other orders
    same = torch.cat([q, torch.zeros(first + behind, 4, d, dtype=dtype, device="cuda")])
    want, want_lse = (x[:5] for x in cache.attend(same, off, lens, table, ws, max_new=max_new, lse=True))
    none = float("nan")
    wide = torch.full((first + 5 + behind, 4, d), none, dtype=dtype, device="cuda")
    wide[first:first + 5] = q
    got, lse = cache.attend(wide, off + first, lens, table, ws, max_new=max_new, lse=True, out=torch.full_like(wide, none))
    ws.status()
    assert torch.equal(got[first:first + 5], want) and torch.equal(lse[first:first + 5], want_lse)
    for a, b in ((0, first), (first + 5, first + 5 + behind)):
        assert bool((got[a:b] == 0).all()) and bool(torch.isneginf(lse[a:b]).all())
    got, lse = cache.attend(wide, off[:1], lens[:0], table[:0], ws, max_new=max_new, lse=True, out=torch.full_like(wide, none))
    ws.status()
    assert bool((got == 0).all()) and bool(torch.isneginf(lse).all())
    got, lse = cache.attend(wide, off.flip(0), lens, table, ws, max_new=max_new, lse=True, out=torch.full_like(wide, none))
    with pytest.raises(tk.TkError):
        ws.status()
    assert bool((got == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.gpu
def test_attend_offsets_that_decrease(tk):
    """Many requests over the same tokens ask for work without end: none of it is done."""
    R, T, bs = 4001, 1 << 20, 128
    W = T // bs
    z = torch.zeros
    cache, ws = tk.KVCache(*z(2, 4, 1, bs, 64, dtype=torch.bfloat16, device="cuda")), tk.KVWorkspace()
    q = z(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, T] * ((R + 1) // 2), device="cuda")
    lens, table = torch.full((R,), T, dtype=torch.int32, device="cuda"), z(R, W, dtype=torch.int32, device="cuda")
    cache.attend(q, off, lens, table, ws)
    with pytest.raises(tk.TkError) as e:
        ws.status()
    assert e.value.code == tk.native.TK_E_LIMIT
    off = torch.cat([torch.arange(200, device="cuda"), torch.arange(R - 199, device="cuda")])  # one step back, far on
    cache.attend(q, off, lens, table, ws)
    with pytest.raises(tk.TkError) as e:
        ws.status()


@pytest.mark.gpu
@pytest.mark.parametrize("scale,taken", [(1e-38, True), (9e37, True), (2.5e38, False), (float("inf"), False)])
def test_attend_scales(tk, scale, taken):
    """Scores of 0 have equal weights at any scale; one that is infinite in base 2 is refused."""
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    cache, ws = tk.KVCache(k, v), tk.KVWorkspace()
    off, lens = torch.tensor([0, 2], device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None]
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    if taken:
        assert bool((cache.attend(q, off, lens, table, ws, scale=scale) == 1).all())
    else:
        with pytest.raises(tk.TkError):
            cache.attend(q, off, lens, table, ws, scale=scale)


@pytest.mark.gpu
def test_new_workspace_is_clear_on_any_stream(tk):
    """Its counters are cleared on the legacy stream; torch's side streams do not wait for that one."""
    L, bs = 20000, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = torch.randn(2, L // bs + 1, 1, bs, 64, generator=gen, device="cuda").bfloat16()
    q = torch.randn(3, 2, 64, generator=gen, device="cuda").bfloat16()
    table = torch.arange(L // bs + 1, dtype=torch.int32, device="cuda")[None]
    off, lens = torch.tensor([0, 3], device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    cache, first = tk.KVCache(k, v), tk.KVWorkspace()
    want = cache.attend(q, off, lens, table, first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    work = torch.randn(8192, 8192, device="cuda").bfloat16()
    for _ in range(40):  # some 20 ms
        work = (work @ work).clamp(-1, 1)
    done = torch.cuda.Event()
    done.record()
    ws = tk.KVWorkspace()
    assert done.query()  # the stream on which it was cleared is past that
    with torch.cuda.stream(side):
        got = cache.attend(q, off, lens, table, ws)
        ws.status()
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hk,n", [(2, 1, 1), (64, 1, 1), (16, 1, 20)])
@pytest.mark.parametrize("below", [9.0, 15.0, 18.0])
@pytest.mark.parametrize("at", [0, 17321])
@pytest.mark.parametrize("R", [1, 320])
def test_attend_one_strong_key(tk, dtype, hq, hk, n, below, at, R):
    """One key of value 0 takes nearly all the weight; the others, e^-below each, carry the output. (Many requests, here
    over one request's blocks, are not divided over the GPU: the key then stands against all others at once.)

    As in test_kv, |err| <= 1.02 u (|o| + A) + 2^-15 (1 + S) A, and in fp16 each weight is off by at most half a
    subnormal step, 2^-25, of a row whose largest weight is at least 2^7: n 2^-32 max|v| in all, and half a
    step of the result, 2^-25.
    """
    L, bs, d = 40000, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(at + n)
    k = torch.zeros(L // bs, hk, bs, d, device="cuda")
    k[..., 1:] = 0.02 * torch.randn(L // bs, hk, bs, d - 1, generator=gen, device="cuda")
    v = 1 + 0.5 * torch.rand(L // bs, hk, bs, d, generator=gen, device="cuda")
    k[at // bs, :, at % bs] = 0
    k[at // bs, :, at % bs, 0] = below
    v[at // bs, :, at % bs] = 0
    k, v = k.to(dtype), v.to(dtype)
    q = torch.randn(R * n, hq, d, generator=gen, device="cuda")
    q[..., 0] = 1
    q = q.to(dtype)
    table = torch.arange(L // bs, dtype=torch.int32, device="cuda").repeat(R, 1)
    off, lens = torch.arange(R + 1, device="cuda") * n, torch.full((R,), L, dtype=torch.int32, device="cuda")
    cache, ws = tk.KVCache(k, v), tk.KVWorkspace()
    got, got_lse = cache.attend(q, off, lens, table, ws, scale=1.0, max_new=n, lse=True)
    ws.status()
    q, got, got_lse = q[-n:], got[-n:], got_lse[-n:]  # the last request's
    kk, vv = (x.transpose(0, 1).reshape(hk, L, d).double()[0] for x in (k, v))
    seen = torch.arange(L, device="cuda")[None] <= L - n + torch.arange(n, device="cuda")[:, None]
    s = torch.einsum("nhd,ld->nhl", q.double(), kk).masked_fill(~seen[:, None], -np.inf)
    w = torch.softmax(s, 2)
    o, a = w @ vv, w @ vv.abs()
    big = torch.einsum("nhd,ld->nhl", q.double().abs(), kk.abs()).amax(2)[..., None]
    tol = 1.02 * U[dtype] * (o.abs() + a) + 2.0 ** -15 * (1 + big) * a
    if dtype == torch.float16:
        tol = tol + L * 2.0 ** -32 * vv.max() + 2.0 ** -25
    _close(got, o.cpu(), tol.cpu())
    assert bool(((got_lse.double() - torch.logsumexp(s, 2)).abs() <= 2.0 ** -16 * (1 + big[..., 0])).all())


@pytest.mark.gpu
def test_requests_of_several_segments(tk, full_table):
    """A prompt of typed segments is one request: the encode's offsets are gathered at the requests' first segments."""
    import workloads
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import draft_tree_step as ex
    tokenizer = tk.Tokenizer(full_table, workloads.SPECIALS)
    prompts = [[("What is a page?", False), ("<|endoftext|>", True), ("A block of", False)], "1, 2, 3,",
               [("x" * 700, False), ("", False), (" and so on", False)]]
    model = ex.Model(100277, 512)
    batch, first = ex.prefill(model, tokenizer, prompts, 64, 512)
    model.workspace.status()
    sizes = [sum(tokenizer.encode(t, a).numel() for t, a in ([(p, False)] if isinstance(p, str) else p)) for p in prompts]
    assert batch.lengths.tolist() == sizes and batch.lengths.shape == (3,)
    for p, want in zip(prompts, first.tolist()):
        alone, got = ex.prefill(model, tokenizer, [p], 64, 512)
        assert got.tolist() == [want]
    tokenizer.close()

"""From the encode's device offsets to a paged key/value cache.

    plan = kv_plan(offsets, context, table, free, block_size, n_tokens)   # place the new tokens
    q = cache.append(qkv, plan.positions, plan.slots, q_heads, ...)       # norm, rotate, store
    out = cache.attend(q, offsets, plan.lengths, table, workspace)        # read the cache

`offsets` is what `encode_device` / `encode_segments` returned (or the
offsets of drafted trees); nothing here copies to the host or waits for the
device. Every step runs in libtk's kernels (include/tk.h, tk_kv_*): the calls
raise without a GPU.
"""
from typing import NamedTuple

from . import native


def _torch():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("byte_level_bpe_gb300 needs a CUDA device (no CPU fallback)")
    return torch


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _stream(torch, stream, device):
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _vector(x, name, dtype, n, device):
    _need(x.dtype == dtype and x.dim() == 1 and x.numel() == n and x.is_contiguous() and x.device == device,
          f"{name} must be a contiguous {dtype} vector of {n} on {device}")
    return x.data_ptr()


class KVPlan(NamedTuple):
    positions: object  # int32[T]
    slots: object      # int64[T], -1 = not placed
    requests: object   # int32[T]
    lengths: object    # int32[R]: tokens in the cache afterwards
    info: object       # int64[4]: cursor, blocks asked for, status, request (tk_kv_plan)
    masks: object      # int64[T] for drafted trees, else None


def kv_plan(offsets, context, table, free, block_size, n_tokens, parents=None, cursor=None, stream=None):
    """Places every request's new tokens in the cache's blocks (tk_kv_plan).

    offsets int64[R+1], context int32[R] (tokens cached already), table
    int32[R, W] (filled in place behind ceil(context / block_size) blocks),
    free int32[n] block ids, n_tokens = the new tokens (offsets[R], or more:
    the rest is padding), parents int32[T] for drafted trees, cursor: one
    int64 on the device, e.g. an earlier plan's info[:1]."""
    torch = _torch()
    dev = table.device
    R, T = context.numel(), int(n_tokens)
    _need(table.dim() == 2 and table.shape[0] == R and table.dtype == torch.int32 and table.is_cuda
          and (table.shape[1] < 2 or table.stride(1) == 1), "table must be int32[R, W] on the GPU, rows contiguous")
    _need(free.dim() == 1, "free must be a vector")
    i32, i64 = torch.int32, torch.int64
    p_off = _vector(offsets, "offsets", i64, R + 1, dev)
    p_ctx = _vector(context, "context", i32, R, dev)
    p_free = _vector(free, "free", i32, free.numel(), dev)
    p_par = _vector(parents, "parents", i32, T, dev) if parents is not None else None
    p_cur = _vector(cursor, "cursor", i64, 1, dev) if cursor is not None else None
    # one allocation, cut at multiples of 16 bytes: slots, masks, info, positions, requests, lengths
    t4 = (T + 3) & ~3
    words = torch.empty((3 if parents is not None else 2) * t4 + 4 + (R + 1) // 2, dtype=i64, device=dev)
    slots, rest = words[:T], words[t4:]
    masks = None
    if parents is not None:
        masks, rest = rest[:T], rest[t4:]
    info, small = rest[:4], rest[4:].view(i32)
    positions, requests, lengths = small[:T], small[t4:t4 + T], small[2 * t4:2 * t4 + R]
    stride = table.stride(0) if R > 1 else table.shape[1]
    native.tk_kv_plan(p_off, p_ctx, R, T, block_size, table.data_ptr(), max(stride, table.shape[1]), table.shape[1],
                      p_free, free.numel(), p_cur, p_par, positions.data_ptr(), slots.data_ptr(),
                      requests.data_ptr(), lengths.data_ptr(), masks.data_ptr() if masks is not None else None,
                      info.data_ptr(), _stream(torch, stream, dev))
    return KVPlan(positions, slots, requests, lengths, info, masks)


def rope_table(n_positions, rot_dim, theta=10000.0, device="cuda"):
    """(cos, sin) float32[n_positions, rot_dim/2, 2] of the angles position *
    theta^(-2i / rot_dim), computed in 64 bits: the table that `append` takes."""
    torch = _torch()
    freq = theta ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    angle = torch.arange(n_positions, device=device, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()


class KVWorkspace:
    """Scratch of one `attend` in flight (tk_kv_workspace): one per stream."""

    def __init__(self):
        _torch()
        self._h = None
        self._h = native.tk_kv_workspace_create()

    def status(self, stream=None):
        """Waits for the stream; raises TkError for the first request that an
        attend on this workspace could not take (tk_kv_status)."""
        torch = _torch()
        native.tk_kv_status(self._h, _stream(torch, stream, None))

    def close(self):
        if self._h is not None:
            native.tk_kv_workspace_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """The paged cache of one layer over caller-owned tensors k, v
    [n_blocks, kv_heads, block_size, head_dim] (bfloat16 or float16; any
    strides that are multiples of 8 elements, the last dimension contiguous)."""

    def __init__(self, k, v):
        torch = _torch()
        types = {torch.bfloat16: native.TK_BF16, torch.float16: native.TK_F16}
        _need(k.is_cuda and k.dim() == 4 and k.dtype in types, "k must be a 4-dimensional bf16 or fp16 GPU tensor")
        _need(v.device == k.device and v.shape == k.shape and v.dtype == k.dtype and v.stride() == k.stride(),
              "v must have k's device, shape, type and strides")
        _need(k.stride(3) == 1, "the last dimension must be contiguous")
        self._h = None
        self.k, self.v, self.device, self.dtype = k, v, k.device, k.dtype
        self.n_blocks, self.kv_heads, self.block_size, self.head_dim = k.shape
        # the stride of a dimension of one element is arbitrary in torch
        d = self.head_dim
        packed = (self.kv_heads * self.block_size * d, self.block_size * d, d)
        stride = [s if n > 1 else p for s, n, p in zip(k.stride(), k.shape, packed)]
        self._h = native.tk_kv_cache_create(k.data_ptr(), v.data_ptr(), types[k.dtype], self.n_blocks, self.kv_heads,
                                            self.block_size, d, stride)

    def append(self, qkv, positions, slots, q_heads, q_gain=None, k_gain=None, rope=None, eps=1e-6,
               neighbours=False, out=None, stream=None):
        """qkv [T, (q_heads + 2 kv_heads) * head_dim] -> queries [T, q_heads,
        head_dim], normed and rotated; keys (normed, rotated) and values are
        stored at `slots` (tk_kv_append). gains float32[head_dim], rope
        float32[n, rot_dim / 2, 2] (`rope_table`)."""
        torch = _torch()
        dev, d = self.device, self.head_dim
        _need(qkv.dim() == 2 and qkv.dtype == self.dtype and qkv.device == dev
              and qkv.shape[1] == (q_heads + 2 * self.kv_heads) * d and qkv.stride(1) == 1,
              f"qkv must be {self.dtype}[T, (q_heads + 2 kv_heads) * head_dim] on {dev}, rows contiguous")
        T = qkv.shape[0]
        f32 = torch.float32
        p_qg = _vector(q_gain, "q_gain", f32, d, dev) if q_gain is not None else None
        p_kg = _vector(k_gain, "k_gain", f32, d, dev) if k_gain is not None else None
        p_rope, n_rope, rot, p_pos = None, 0, 0, None
        if rope is not None:
            _need(rope.dim() == 3 and rope.shape[2] == 2 and rope.dtype == f32 and rope.is_contiguous()
                  and rope.device == dev, f"rope must be a contiguous float32[n, rot_dim / 2, 2] on {dev}")
            p_rope, n_rope, rot = rope.data_ptr(), rope.shape[0], 2 * rope.shape[1]
            p_pos = _vector(positions, "positions", torch.int32, T, dev)
        p_slot = _vector(slots, "slots", torch.int64, T, dev)
        if out is None:
            out = torch.empty((T, q_heads, d), dtype=self.dtype, device=dev)
        else:
            _need(out.shape == (T, q_heads, d) and out.dtype == self.dtype and out.is_contiguous() and out.device == dev,
                  "out must be a contiguous tensor [T, q_heads, head_dim] of the cache's type")
        native.tk_kv_append(self._h, qkv.data_ptr(), max(qkv.stride(0), qkv.shape[1]) if T > 1 else qkv.shape[1], T,
                            q_heads, p_qg, p_kg, eps, p_rope, n_rope, rot, neighbours, p_pos, p_slot, out.data_ptr(),
                            _stream(torch, stream, dev))
        return out

    def attend(self, q, offsets, lengths, table, workspace, masks=None, scale=None, max_new=None, lse=False,
               out=None, stream=None):
        """q [T, q_heads, head_dim] -> out of the same shape: each request's new
        tokens over its cache (tk_kv_attend). masks int64[T] as `kv_plan` makes
        them for drafted trees, None = each token sees those before it. scale
        defaults to head_dim^-0.5; max_new: no request has more new tokens
        (T if not given). lse=True also returns float32[T, q_heads]."""
        torch = _torch()
        dev, d = self.device, self.head_dim
        _need(q.dim() == 3 and q.shape[2] == d and q.dtype == self.dtype and q.device == dev and q.stride(2) == 1
              and (q.stride(1) == d or q.shape[1] == 1),
              f"q must be {self.dtype}[T, q_heads, head_dim] on {dev}, the heads of a token contiguous")
        T, hq = q.shape[0], q.shape[1]
        R = lengths.numel()
        _need(table.dim() == 2 and table.shape[0] == R and table.dtype == torch.int32 and table.device == dev
              and (table.shape[1] < 2 or table.stride(1) == 1), f"table must be int32[R, W] on {dev}, rows contiguous")
        p_off = _vector(offsets, "offsets", torch.int64, R + 1, dev)
        p_len = _vector(lengths, "lengths", torch.int32, R, dev)
        p_mask = _vector(masks, "masks", torch.int64, T, dev) if masks is not None else None
        if out is None:
            out = torch.empty((T, hq, d), dtype=self.dtype, device=dev)
        else:
            _need(out.shape == q.shape and out.dtype == self.dtype and out.is_contiguous() and out.device == dev,
                  "out must be a contiguous tensor of q's shape and type")
        sums = torch.empty((T, hq), dtype=torch.float32, device=dev) if lse else None
        W = table.shape[1]
        native.tk_kv_attend(self._h, workspace._h, q.data_ptr(), q.stride(0) if T > 1 else hq * d, hq, p_off, R, T,
                            T if max_new is None else max_new, p_len, table.data_ptr(),
                            max(table.stride(0), W) if R > 1 else W, W, p_mask, d ** -0.5 if scale is None else scale,
                            out.data_ptr(), sums.data_ptr() if lse else None, _stream(torch, stream, dev))
        return (out, sums) if lse else out

    def close(self):
        if self._h is not None:
            native.tk_kv_cache_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

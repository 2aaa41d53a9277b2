"""From the encode's device offsets to a paged key/value cache.

    plan = kv_plan(offsets, context, table, free, block_size, n_tokens)   # place the new tokens
    q = cache.append(qkv, plan.positions, plan.slots, q_heads, ...)       # norm, rotate, store
    out = cache.attend(q, offsets, plan.lengths, table, workspace)        # read the cache

`offsets` has an entry where each request's tokens begin, and the end: what
`encode_device` / `encode_segments` returned if a request is one segment. The
encode counts segments, so for requests of several it is `offsets[first]`, with
first = the number of each request's first segment and, last, of all segments
(an index tensor on the device). For drafted trees it is theirs. Nothing here
copies to the host or waits for the device. Every step runs in libtk's kernels
(include/tk.h, tk_kv_*): the calls raise without a GPU.

A call queues its work on the current stream, or on the one given as `stream`: then
it is as if that one were current (outputs are its own, the caller orders it
after what wrote the inputs), and the inputs' memory is not handed out again
before its work is done.
"""
from typing import NamedTuple

from . import native


_T = None  # torch, once a CUDA device has been seen
_raw_stream = None
_current_device = None


def _torch():
    global _T, _raw_stream, _current_device
    if _T is None:
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("byte_level_bpe_gb300 needs a CUDA device (no CPU fallback)")
        # the current device's index and its current stream's handle without the objects around them,
        # where torch has that
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
        _T = torch
    return _T


# These calls take a few microseconds on the GPU for a decode step, so the checks
# are written for few Python operations: devices are compared as indices.

def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _need_current(index):
    """Kernels and handles go to the current device, so it has to be the tensors'."""
    if _current_device() != index:
        raise ValueError(f"the tensors are on cuda:{index}, which is not the current device")


def _no_gradient(name):
    """There is no backward pass: a result without a gradient must not pass for one that has it."""
    if _T.is_grad_enabled():
        raise ValueError(f"{name} has no gradient: call it under torch.no_grad(), or detach its inputs")


def _on(stream, call, *used):
    """The call with `stream` as the current one; `used` are the tensors its work touches."""
    with _torch().cuda.stream(stream):
        result = call()
    for x in used:
        if x is not None:
            x.record_stream(stream)
    return result


def _vector(x, name, dtype, n, index):
    if x.dtype is not dtype or x.shape != (n,) or x.get_device() != index or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on cuda:{index}")
    return x.data_ptr()


def _row_stride(stride, rows, width, name):
    """Elements from a row to the next; of one row or empty ones torch's stride says nothing."""
    if rows < 2 or width == 0:
        return width
    if stride < width:
        raise ValueError(f"the rows of {name} must not overlap (an expanded tensor is not taken)")
    return stride


def _table(table, R, dtype, index):
    """(address, row stride, width) of a block table."""
    if table.dim() != 2 or table.dtype is not dtype or table.get_device() != index or index < 0 or table.shape[0] != R:
        raise ValueError("table must be int32[R, W] on the GPU, like the other tensors")
    stride, unit = table.stride()
    W = table.shape[1]
    if unit != 1 and W > 1:
        raise ValueError("the rows of table must be contiguous")
    return table.data_ptr(), _row_stride(stride, R, W, "table"), W


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
    the rest is padding; with fewer, requests that end past it are not placed),
    parents int32[T] for drafted trees, cursor: one int64 on the device, e.g. an
    earlier plan's info[:1]. info tells whether all were placed; the attention's
    rows of one that was not mean nothing."""
    if stream is not None:
        return _on(stream, lambda: kv_plan(offsets, context, table, free, block_size, n_tokens, parents, cursor),
                   offsets, context, table, free, parents, cursor)
    torch = _torch()
    index = table.get_device()
    i32, i64 = torch.int32, torch.int64
    R, T = context.numel(), n_tokens
    p_table, stride, W = _table(table, R, i32, index)
    _need_current(index)
    p_off = _vector(offsets, "offsets", i64, R + 1, index)
    p_ctx = _vector(context, "context", i32, R, index)
    n_free = free.numel()
    p_free = _vector(free, "free", i32, n_free, index)
    p_cur = _vector(cursor, "cursor", i64, 1, index) if cursor is not None else None
    # an allocation each: on the host they are cheaper than views of a common one
    empty, device = torch.empty, table.device
    positions, slots = empty(T, dtype=i32, device=device), empty(T, dtype=i64, device=device)
    requests, lengths = empty(T, dtype=i32, device=device), empty(R, dtype=i32, device=device)
    info = empty(4, dtype=i64, device=device)
    p_par, masks, p_mask = None, None, None
    if parents is not None:
        p_par = _vector(parents, "parents", i32, T, index)
        masks = empty(T, dtype=i64, device=device)
        p_mask = masks.data_ptr()
    rc = native.load().tk_kv_plan(p_off, p_ctx, R, T, block_size, p_table, stride, W, p_free, n_free, p_cur, p_par,
                                  positions.data_ptr(), slots.data_ptr(), requests.data_ptr(), lengths.data_ptr(), p_mask,
                                  info.data_ptr(), _raw_stream(index))
    if rc:
        native.check(rc, "tk_kv_plan")
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
        self._h = None
        self._index = _torch().cuda.current_device()
        self._h = native.tk_kv_workspace_create()

    def status(self, stream=None):
        """Waits for the stream; raises TkError for the first request that an
        attend on this workspace could not take (tk_kv_status)."""
        _need_current(self._index)
        native.tk_kv_status(self._h, stream.cuda_stream if stream is not None else _raw_stream(self._index))

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
        self._index = k.get_device()
        _need_current(self._index)
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
        if stream is not None:
            return _on(stream, lambda: self.append(qkv, positions, slots, q_heads, q_gain, k_gain, rope, eps, neighbours, out),
                       qkv, positions, slots, q_gain, k_gain, rope, out, self.k, self.v)
        torch = _torch()
        index, d = self._index, self.head_dim
        T, width = qkv.shape  # a ValueError if there are not two dimensions
        row, unit = qkv.stride()
        if (qkv.dtype is not self.dtype or qkv.get_device() != index or width != (q_heads + 2 * self.kv_heads) * d
                or unit != 1):
            raise ValueError(f"qkv must be {self.dtype}[T, (q_heads + 2 kv_heads) * head_dim] on cuda:{index}, "
                             "rows contiguous")
        if (qkv.requires_grad or (q_gain is not None and q_gain.requires_grad)
                or (k_gain is not None and k_gain.requires_grad) or (rope is not None and rope.requires_grad)):
            _no_gradient("append")
        f32 = torch.float32
        p_qg = _vector(q_gain, "q_gain", f32, d, index) if q_gain is not None else None
        p_kg = _vector(k_gain, "k_gain", f32, d, index) if k_gain is not None else None
        p_rope, n_rope, rot, p_pos = None, 0, 0, None
        if rope is not None:
            n_rope, rot, two = rope.shape
            if two != 2 or rope.dtype is not f32 or not rope.is_contiguous() or rope.get_device() != index:
                raise ValueError(f"rope must be a contiguous float32[n, rot_dim / 2, 2] on cuda:{index}")
            p_rope, rot = rope.data_ptr(), 2 * rot
            p_pos = _vector(positions, "positions", torch.int32, T, index)
        p_slot = _vector(slots, "slots", torch.int64, T, index)
        if out is None:
            out = torch.empty((T, q_heads, d), dtype=self.dtype, device=self.device)
        elif (out.shape != (T, q_heads, d) or out.dtype is not self.dtype or not out.is_contiguous()
              or out.get_device() != index):
            raise ValueError("out must be a contiguous tensor [T, q_heads, head_dim] of the cache's type")
        rc = native.load().tk_kv_append(self._h, qkv.data_ptr(), _row_stride(row, T, width, "qkv"), T, q_heads, p_qg,
                                        p_kg, eps, p_rope, n_rope, rot, 1 if neighbours else 0, p_pos, p_slot,
                                        out.data_ptr(), _raw_stream(index))
        if rc:
            native.check(rc, "tk_kv_append")
        return out

    def attend(self, q, offsets, lengths, table, workspace, masks=None, scale=None, max_new=None, lse=False,
               out=None, stream=None):
        """q [T, q_heads, head_dim] -> out of the same shape: each request's new
        tokens over its cache (tk_kv_attend). masks int64[T] as `kv_plan` makes
        them for drafted trees, None = each token sees those before it. scale
        defaults to head_dim^-0.5; max_new: no request has more new tokens
        (T if not given; it chooses the kernel, so give it: a decode step with
        max_new=1 can be a quarter faster). lse=True also returns
        float32[T, q_heads]. Tokens of no request, and rows that see nothing, give
        0 and an lse of -inf; so do requests outside the call's limits, of which
        only workspace.status() tells."""
        if stream is not None:
            return _on(stream, lambda: self.attend(q, offsets, lengths, table, workspace, masks, scale, max_new, lse, out),
                       q, offsets, lengths, table, masks, out, self.k, self.v)
        torch = _torch()
        index, d = self._index, self.head_dim
        T, hq, width = q.shape  # a ValueError if there are not three dimensions
        step, head, unit = q.stride()
        if (width != d or q.dtype is not self.dtype or q.get_device() != index or unit != 1
                or (head != d and hq > 1)):
            raise ValueError(f"q must be {self.dtype}[T, q_heads, head_dim] on cuda:{index}, the heads of a token contiguous")
        if q.requires_grad or self.k.requires_grad or self.v.requires_grad:
            _no_gradient("attend")
        R = lengths.numel()
        p_table, stride, W = _table(table, R, torch.int32, index)
        p_off = _vector(offsets, "offsets", torch.int64, R + 1, index)
        p_len = _vector(lengths, "lengths", torch.int32, R, index)
        p_mask = _vector(masks, "masks", torch.int64, T, index) if masks is not None else None
        if out is None:
            out = torch.empty((T, hq, d), dtype=self.dtype, device=self.device)
        elif out.shape != q.shape or out.dtype is not self.dtype or not out.is_contiguous() or out.get_device() != index:
            raise ValueError("out must be a contiguous tensor of q's shape and type")
        sums = torch.empty((T, hq), dtype=torch.float32, device=self.device) if lse else None
        rc = native.load().tk_kv_attend(self._h, workspace._h, q.data_ptr(), _row_stride(step, T, hq * d, "q"), hq, p_off, R, T,
                                        T if max_new is None else max_new, p_len, p_table, stride, W, p_mask,
                                        d ** -0.5 if scale is None else scale, out.data_ptr(),
                                        sums.data_ptr() if lse else None, _raw_stream(index))
        if rc:
            native.check(rc, "tk_kv_attend")
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

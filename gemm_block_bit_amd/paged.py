"""Rotary positions, the paged key-value cache and its attention: the binding
of gbb_rope*, gbb_paged_attention* and gbb_cache_evict* (include/gbb.h states
what each computes).

A decoding step around the quantized products:

    qkv = gemm_mixed_w(...)                                    # [T][(Hq + 2 Hkv) D]
    q = rope_append(cache, qkv, Hq, positions, slots, table)   # k, v -> cache
    o = paged_attention(cache, q, block_table, lengths, max_len)
    y = gemm_mixed_w(..., o.view(T, -1))

Every call enqueues on torch's current stream of the cache's (or x's) device.
Calls of several threads on one stream are as good as one after the other.  rope
takes part in torch's differentiation; the other calls' results have no gradient.
"""
from __future__ import annotations

import ctypes

import numpy as np

from .binding import _check, _dev_ptr, _given, _kept, _np_ptr, _on, _PagedCache, _RopeScaling, _torch, lib

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "yarn": 3}
_dtype_codes: dict = {}


def _dtype_code(dtype) -> int:
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.float8_e4m3fn: 3})
    code = _dtype_codes.get(dtype)
    if code is None:
        raise TypeError(f"{dtype} is not supported (float16, bfloat16, float32 or float8_e4m3fn)")
    return code


def _layout(layout: str) -> int:
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
    return _LAYOUTS[layout]


def _ptr(t, dtype, device: int, name: str, shape=None):
    """Address of a contiguous tensor of `dtype` on GPU `device`.  These
    checks are on the path of calls that take a few microseconds, so the
    messages are left to _refuse."""
    if getattr(t, "dtype", None) is not dtype or t.get_device() != device or not t.is_contiguous() or \
            (shape is not None and t.shape != shape):
        _refuse(t, dtype, device, name, shape)
    return t.data_ptr()


def _refuse(t, dtype, device, name, shape):
    _dev_ptr(t, dtype, name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on GPU {device}")


def _device_of(t, name) -> int:
    try:
        device = t.get_device()
    except AttributeError:
        device = -1
    if device < 0:
        raise TypeError(f"{name} must be a torch tensor on a GPU")
    return device


_int32 = _float32 = _raw_stream = _current_device = _capturing = _grad_enabled = _written = None


def _resolve() -> None:
    """What every call needs of torch, looked up once.  The stream as a
    hipStream_t is taken by the accessor that torch's own generated code uses
    (the public one builds two Python objects for every call, 2 us)."""
    global _int32, _float32, _raw_stream, _current_device, _capturing, _grad_enabled, _written
    torch = _torch()
    _float32, _capturing = torch.float32, torch.cuda.is_current_stream_capturing
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    # _written: a tensor's version, by which torch sees that a saved one changed
    _grad_enabled, _written = torch.is_grad_enabled, torch.autograd.graph.increment_version
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _int32 = torch.int32


# ----------------------------------------------------------------------------
# rotary positions
# ----------------------------------------------------------------------------
def rope_table(rot: int, n_pos: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               original_len: float = 0.0, low: float | None = None, high: float | None = None,
               attention: float = 1.0) -> np.ndarray:
    """float32 [n_pos][rot/2][2] of (cos, sin) on the host (see
    gbb_rope_table); scaling is plain, linear, bands or yarn.  low and high
    default to what each is published with: bands 1 and 4 wave lengths in
    original_len, yarn 1 and 32 turns.  attention is left to the caller (yarn
    is published with 0.1 ln factor + 1)."""
    if low is None:
        low = 1.0
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    table = np.empty((max(0, n_pos), max(0, rot) // 2, 2), np.float32)
    s = _RopeScaling(_SCALINGS[scaling], factor, original_len, low, high, attention)
    _check(lib().gbb_rope_table(rot, n_pos, float(base), ctypes.byref(s), _np_ptr(table)))
    return table


def _table(table, device):
    p = _ptr(table, _float32, device, "table")
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2:
        raise ValueError("table must be float32 [n_pos][rot/2][2]")
    return p, shape[0], 2 * shape[1]


def rope(x, positions, table, layout: str = "half", transpose: bool = False, out=None):
    """x [T][H][D] (float16, bfloat16 or float32; the last dimension
    contiguous) with its first 2 * table.shape[1] elements rotated to int32
    positions [T].  out: where to write (x itself for in place), else a new
    contiguous tensor.  transpose: the transposed rotation, which is the
    gradient with respect to x; where x requires one, the result takes part in
    torch's differentiation (the table has no gradient)."""
    if _int32 is None:
        _resolve()
    device = _device_of(x, "x")
    if x.requires_grad and _grad_enabled():
        return _differentiable().apply(x, positions, table, layout, transpose, out)
    if _current_device() != device:
        return _on(device, rope, x, positions, table, layout, transpose, out)
    shape, xs = x.shape, x.stride()
    if len(shape) != 3 or xs[2] != 1:
        raise ValueError("x must be [T][H][D] with contiguous heads")
    T, H, D = shape
    if out is None:
        y = x.new_empty(T, H, D)
    else:
        y = out
        if y.dtype != x.dtype or y.shape != x.shape or y.stride(2) != 1:
            raise ValueError("out must be like x, with contiguous heads")
        if y.get_device() != device:
            raise ValueError(f"out is on {y.device}, not on {x.device}")
    tp, n_pos, rot = _table(table, device)
    ys = y.stride()
    _check(lib().gbb_rope(x.data_ptr(), xs[0], xs[1], y.data_ptr(), ys[0], ys[1], _dtype_code(x.dtype), T, H, D,
                          _ptr(positions, _int32, device, "positions", (T,)), tp, n_pos, rot, _layout(layout),
                          int(transpose), _raw_stream(device)))
    if out is not None:
        _written(out)
    return y


_Rope = None


def _differentiable():
    """The rotation as a torch.autograd.Function, made at its first use."""
    global _Rope
    if _Rope is not None:
        return _Rope
    torch = _torch()

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, table, layout, transpose, out):
            ctx.layout, ctx.transpose = layout, transpose
            ctx.save_for_backward(positions, table)
            if out is not None:
                ctx.mark_dirty(out)
            return rope(x, positions, table, layout, transpose, out)   # torch runs this without gradients

        @staticmethod
        def backward(ctx, g):
            positions, table = ctx.saved_tensors
            if g.stride(2) != 1:
                g = g.contiguous()
            return rope(g, positions, table, ctx.layout, not ctx.transpose), None, None, None, None, None

    _Rope = Rope
    return Rope


# ----------------------------------------------------------------------------
# the cache
# ----------------------------------------------------------------------------
class PagedCache:
    """A gbb_paged_cache over torch tensors: k and v [pages][kv heads][page]
    [head size] (float16, bfloat16 or float8_e4m3fn with float32 k_scale and
    v_scale [kv heads]); for eviction also float32 weights and int32
    positions [pages][kv heads][page].  The tensors are kept referenced and
    must keep their storage."""

    def __init__(self, k, v, k_scale=None, v_scale=None, weights=None, positions=None):
        _resolve()
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages][kv heads][page][head size] of one dtype")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.weights, self.positions = weights, positions
        self.device, self.dtype = k.device, k.dtype
        self.num_pages, self.kv_heads, self.page, self.head_dim = k.shape
        code = _dtype_code(k.dtype)
        if code == 2:
            raise TypeError("a cache holds float16, bfloat16 or float8_e4m3fn")
        self._index = _device_of(k, "k")

        def ptr(t, dtype, name, shape):
            return None if t is None else _ptr(t, dtype, self._index, name, shape)

        one, slots = (self.kv_heads,), tuple(k.shape[:3])
        self._c = _PagedCache(ptr(k, k.dtype, "k", None), ptr(v, v.dtype, "v", None),
                              ptr(k_scale, _float32, "k_scale", one), ptr(v_scale, _float32, "v_scale", one),
                              ptr(weights, _float32, "weights", slots), ptr(positions, _int32, "positions", slots),
                              code, self.num_pages, self.page, self.kv_heads, self.head_dim)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, page: int, kv_heads: int, head_dim: int, dtype=None, device="cuda",
              tracked: bool = False, k_scale=None, v_scale=None):
        """A new cache (its k and v zero); tracked: with weights and
        positions, for eviction."""
        torch = _torch()
        dtype = torch.float16 if dtype is None else dtype
        shape = (num_pages, kv_heads, page, head_dim)
        k, v = torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device)
        w = torch.zeros(shape[:3], dtype=torch.float32, device=device) if tracked else None
        p = torch.full(shape[:3], -1, dtype=torch.int32, device=device) if tracked else None
        return cls(k, v, k_scale, v_scale, w, p)


_ws_cache: dict = {}
_E_SPACE = -5


def _with_workspace(kind: str, device: int, given, call, args, need):
    """call(*args, workspace, bytes, stream), on the current GPU, with the
    caller's workspace, or with a buffer kept per use, device and stream (apart
    from the buffer of the gemm calls, which has to stay zero), one call at a
    time.  need() is only asked when a call says that the buffer is too small.
    A call that is captured in a graph gets a buffer of the graph's own, whose
    counters are cleared in every replay: one that is kept would be shared with
    calls outside the graph."""
    stream = _raw_stream(device)
    if given is not None:
        _check(call(*args, *_given(given, device), stream))
        return
    if _capturing():
        buf = _buffer(kind, max(need(), 16), device)
        _check(call(*args, buf.data_ptr(), buf.numel(), stream))
        return
    kept = _kept(_ws_cache, (kind, device, stream))
    with kept.lock:
        if kept.buf is None:
            kept.buf = _buffer(kind, 1 << 20, device)
        st = call(*args, kept.buf.data_ptr(), kept.buf.numel(), stream)
        if st == _E_SPACE:
            kept.buf = _buffer(kind, need(), device)
            st = call(*args, kept.buf.data_ptr(), kept.buf.numel(), stream)
        _check(st)


# bytes at a workspace's start that have to be zero before its first use
_CLEARED = {"attention": 16384, "evict": 0}


def _buffer(kind: str, nbytes: int, device: int):
    torch = _torch()
    buf = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
    if _CLEARED[kind]:
        buf[:_CLEARED[kind]].zero_()
    return buf


def rope_append(cache: PagedCache, qkv, q_heads: int, positions, slots, table, layout: str = "half", out=None):
    """Rotates the q and k heads of qkv [T][(q_heads + 2 kv heads) head size]
    (rows may be strided), writes k and v to the cache's int32 slots [T] and
    returns q [T][q_heads][head size] (see gbb_rope_append)."""
    device = cache._index
    if _current_device() != device:
        return _on(device, rope_append, cache, qkv, q_heads, positions, slots, table, layout, out)
    if _device_of(qkv, "qkv") != device:
        raise ValueError(f"qkv is on {qkv.device}, not on GPU {device}")
    D = cache.head_dim
    width = (q_heads + 2 * cache.kv_heads) * D
    shape, stride = qkv.shape, qkv.stride()
    if len(shape) != 2 or shape[1] != width or stride[1] != 1:
        raise ValueError(f"qkv must be [T][{width}] with contiguous rows")
    T = shape[0]
    if out is None:
        q = qkv.new_empty(T, q_heads, D)
        qp = q.data_ptr()
    else:
        q = out
        qp = _ptr(q, qkv.dtype, device, "out", (T, q_heads, D))
    tp, n_pos, rot = _table(table, device)
    _check(lib().gbb_rope_append(
        cache._ref, qkv.data_ptr(), stride[0] if T > 1 else width, _dtype_code(qkv.dtype), T, q_heads,
        _ptr(positions, _int32, device, "positions", (T,)), _ptr(slots, _int32, device, "slots", (T,)), tp,
        n_pos, rot, _layout(layout), qp, _raw_stream(device)))
    return q


def paged_attention_workspace(cache: PagedCache, batch: int, q_heads: int, max_len: int,
                              with_weights: bool = False) -> int:
    """Bytes of paged_attention's workspace (with_weights: of a call with
    weights_out).  A new one's first 16384 have to be zero: torch.zeros."""
    return _on(cache._index, lib().gbb_paged_attention_workspace, cache._ref, batch, q_heads, max_len,
               int(with_weights))


def paged_attention(cache: PagedCache, q, block_table, lengths, max_len: int, scale: float | None = None, out=None,
                    lse=None, weights_out=None, workspace=None):
    """Attention of one new token per sequence, q [B][q_heads][head size],
    over the first lengths[b] <= max_len slots of the pages block_table[b]
    (int32 [B] and [B][pages]); scale defaults to head size ** -0.5.  lse:
    float32 [B][q_heads] to fill.  weights_out: where to write the cache's
    weights with this step's added (cache.weights itself for in place).
    workspace: paged_attention_workspace bytes that were zero when they were
    new (torch.zeros, not empty: outputs would stay unwritten), else the
    binding's own.  Returns [B][q_heads][head size] (see gbb_paged_attention)."""
    device, D = cache._index, cache.head_dim
    if _current_device() != device:
        return _on(device, paged_attention, cache, q, block_table, lengths, max_len, scale, out, lse, weights_out, workspace)
    if _device_of(q, "q") != device:
        raise ValueError(f"q is on {q.device}, not on GPU {device}")
    shape, stride = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != D or stride[2] != 1 or (stride[1] != D and shape[1] != 1):
        raise ValueError(f"q must be [B][q_heads][{D}] with contiguous tokens")
    B, q_heads, _ = shape
    if out is None:
        o = q.new_empty(B, q_heads, D)
        op = o.data_ptr()
    else:
        o = out
        op = _ptr(o, q.dtype, device, "out", shape)
    bt, table_shape = _ptr(block_table, _int32, device, "block_table"), block_table.shape
    if len(table_shape) != 2 or table_shape[0] != B:
        raise ValueError(f"block_table must be int32 [{B}][pages]")
    w = None
    if weights_out is not None:
        if cache.weights is None:
            raise ValueError("the cache has no weights")
        w = _ptr(weights_out, _float32, device, "weights_out", cache.weights.shape)
    args = (cache._ref, q.data_ptr(), stride[0], _dtype_code(q.dtype), B, q_heads, bt, table_shape[1],
            _ptr(lengths, _int32, device, "lengths", (B,)), max_len, D ** -0.5 if scale is None else scale,
            op, _ptr(lse, _float32, device, "lse", (B, q_heads)) if lse is not None else None, w)
    _with_workspace("attention", device, workspace, lib().gbb_paged_attention, args,
                    lambda: paged_attention_workspace(cache, B, q_heads, max_len, w is not None))
    return o


def cache_evict_workspace(cache: PagedCache, batch: int, max_len: int, budget: int) -> int:
    """Bytes of cache_evict's workspace, which may hold anything."""
    return lib().gbb_cache_evict_workspace(cache._ref, batch, max_len, budget)


def cache_evict(cache: PagedCache, block_table, lengths, max_len: int, budget: int, recent: int, weights_out=None,
                positions_out=None, lengths_out=None, workspace=None):
    """Cuts every sequence longer than budget to budget slots: per kv head
    the `recent` newest positions and the slots of the largest weight (see
    gbb_cache_evict).  weights_out, positions_out: default in place.  Returns
    the new lengths, int32 [B] (lengths_out if given)."""
    if cache.weights is None or cache.positions is None:
        raise ValueError("eviction needs a cache with weights and positions")
    device = cache._index
    if _current_device() != device:
        return _on(device, cache_evict, cache, block_table, lengths, max_len, budget, recent, weights_out, positions_out,
                   lengths_out, workspace)
    bt = _ptr(block_table, _int32, device, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B][pages]")
    B, pages = block_table.shape
    lp = _ptr(lengths, _int32, device, "lengths", (B,))
    n = lengths_out if lengths_out is not None else lengths.new_empty(B)
    shape = cache.weights.shape
    w = cache._c.weights if weights_out is None else _ptr(weights_out, _float32, device, "weights_out", shape)
    p = cache._c.positions if positions_out is None else _ptr(positions_out, _int32, device, "positions_out", shape)
    args = (cache._ref, B, bt, pages, lp, max_len, budget, recent,
            _ptr(n, _int32, device, "lengths_out", (B,)), w, p)
    _with_workspace("evict", device, workspace, lib().gbb_cache_evict, args,
                    lambda: cache_evict_workspace(cache, B, max_len, budget))
    return n

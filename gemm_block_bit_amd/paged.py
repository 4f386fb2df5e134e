"""Rotary positions, norms of heads, the paged key-value cache and its
attention: the binding of gbb_rope*, gbb_norm_rope*, gbb_paged_attention* and
gbb_cache_* (include/gbb.h states what each computes).

A decoding step around the quantized products:

    qkv = gemm_mixed_w(...)                                    # [T][(Hq + 2 Hkv) D]
    q = rope_append(cache, qkv, Hq, positions, slots, table)   # k, v -> cache
    o = paged_attention(cache, q, block_table, lengths, max_len)
    y = gemm_mixed_w(..., o.view(T, -1))

and with prompts or drafted tokens, any number of new ones per sequence:

    o = paged_attention_tokens(cache, q, starts, block_table, lengths, max_len, tree=tree)
    lengths = cache_keep(cache, block_table, lengths, drafted, kept, counts)

Every call enqueues on torch's current stream of the cache's (or x's) device.
Calls of several threads on one stream are as good as one after the other.  rope
and norm_rope take part in torch's differentiation; the other calls' results have
no gradient.
"""
from __future__ import annotations

import ctypes
import operator

import numpy as np

from .binding import (_AttentionOptions, _check, _dev_ptr, _given, _kept, _np_ptr, _on, _PagedCache, _RopeScaling,
                      _torch, lib)

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "yarn": 3}
_INT_MAX = 2 ** 31 - 1
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


_section_arrays: dict = {}


def _axes(positions, sections, device, tokens):
    """(address of positions, number of axes, host array of the sections or
    None): positions [T], or [axes][T] with sections."""
    if sections is None:
        return _ptr(positions, _int32, device, "positions", (tokens,)), 1, None
    array = _section_arrays.get(sections) if type(sections) is tuple else None
    if array is None:
        sections = tuple(operator.index(n) for n in sections)
        if not 1 <= len(sections) <= 4:
            raise ValueError(f"sections must have 1 to 4 axes ({len(sections)})")
        array = _section_arrays.setdefault(sections, (ctypes.c_int * len(sections))(*sections))
    return _ptr(positions, _int32, device, "positions", (len(array), tokens)), len(array), array


def _heads(x, name="x"):
    """(shape, strides) of x [T][H][D] with contiguous heads."""
    shape, strides = x.shape, x.stride()
    if len(shape) != 3 or strides[2] != 1:
        raise ValueError(f"{name} must be [T][H][D] with contiguous heads")
    return shape, strides


def _output_like(x, out, device):
    if out is None:
        return x.new_empty(*x.shape)
    if out.dtype != x.dtype or out.shape != x.shape or out.stride(2) != 1:
        raise ValueError("out must be like x, with contiguous heads")
    if out.get_device() != device:
        raise ValueError(f"out is on {out.device}, not on {x.device}")
    return out


def rope(x, positions, table, layout: str = "half", transpose: bool = False, out=None, sections=None):
    """x [T][H][D] (float16, bfloat16 or float32; the last dimension
    contiguous) with its first 2 * table.shape[1] elements rotated to int32
    positions [T].  out: where to write (x itself for in place), else a new
    contiguous tensor.  transpose: the transposed rotation, which is the
    gradient with respect to x; where x requires one, the result takes part in
    torch's differentiation (the table has no gradient).  sections: the pairs
    of each of 1 to 4 axes, in order (their sum is table.shape[1]); positions
    is then [axes][T]."""
    if _int32 is None:
        _resolve()
    device = _device_of(x, "x")
    if x.requires_grad and _grad_enabled():
        return _differentiable().apply(x, positions, table, layout, transpose, out, sections)
    if _current_device() != device:
        return _on(device, rope, x, positions, table, layout, transpose, out, sections)
    shape, xs = _heads(x)
    T, H, D = shape
    y = _output_like(x, out, device)
    tp, n_pos, rot = _table(table, device)
    ys = y.stride()
    if sections is None:
        _check(lib().gbb_rope(x.data_ptr(), xs[0], xs[1], y.data_ptr(), ys[0], ys[1], _dtype_code(x.dtype), T, H, D,
                              _ptr(positions, _int32, device, "positions", (T,)), tp, n_pos, rot, _layout(layout),
                              int(transpose), _raw_stream(device)))
    else:
        pp, axes, counts = _axes(positions, sections, device, T)
        _check(lib().gbb_rope_axes(x.data_ptr(), xs[0], xs[1], y.data_ptr(), ys[0], ys[1], _dtype_code(x.dtype), T, H,
                                   D, pp, axes, counts, tp, n_pos, rot, _layout(layout), int(transpose),
                                   _raw_stream(device)))
    if out is not None:
        _written(out)
    return y


_Rope = _NormRope = None


def _differentiable():
    """The rotation as a torch.autograd.Function, made at its first use."""
    global _Rope
    if _Rope is not None:
        return _Rope
    torch = _torch()

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, table, layout, transpose, out, sections):
            ctx.layout, ctx.transpose, ctx.sections = layout, transpose, sections
            ctx.save_for_backward(positions, table)
            if out is not None:
                ctx.mark_dirty(out)
            return rope(x, positions, table, layout, transpose, out, sections)   # torch runs this without gradients

        @staticmethod
        def backward(ctx, g):
            positions, table = ctx.saved_tensors
            if g.stride(2) != 1:
                g = g.contiguous()
            gx = rope(g, positions, table, ctx.layout, not ctx.transpose, None, ctx.sections)
            return gx, None, None, None, None, None, None

    _Rope = Rope
    return Rope


def _weight(weight, x, device, D, name="weight"):
    """(address, dtype code) of a norm's weight [D], float32 or of x's dtype."""
    if weight is None:
        return None, 2
    dtype = getattr(weight, "dtype", None)
    if dtype is not _float32 and dtype is not x.dtype:
        raise TypeError(f"{name} must be float32 or {x.dtype}")
    return _ptr(weight, dtype, device, name, (D,)), _dtype_code(dtype)


def norm_rope(x, weight, positions, table, eps: float = 1e-6, layout: str = "half", sections=None, out=None):
    """Every head of x [T][H][D] divided by its root mean square (with eps) and
    times weight [D] (float32 or x's dtype; None: ones), then rotated as rope
    does, in one pass and with one rounding.  Takes part in torch's
    differentiation with respect to x and weight, but not twice; then `out` must
    not be given."""
    if _int32 is None:
        _resolve()
    device = _device_of(x, "x")
    if (x.requires_grad or getattr(weight, "requires_grad", False)) and _grad_enabled():
        if out is not None:
            raise ValueError("out is for calls without a gradient")
        return _differentiable_norm().apply(x, weight, positions, table, eps, layout, sections)
    if _current_device() != device:
        return _on(device, norm_rope, x, weight, positions, table, eps, layout, sections, out)
    shape, xs = _heads(x)
    T, H, D = shape
    y = _output_like(x, out, device)
    ys = y.stride()
    tp, n_pos, rot = _table(table, device)
    wp, wd = _weight(weight, x, device, D)
    pp, axes, counts = _axes(positions, sections, device, T)
    _check(lib().gbb_norm_rope(x.data_ptr(), xs[0], xs[1], y.data_ptr(), ys[0], ys[1], _dtype_code(x.dtype), T, H, D,
                               wp, wd, eps, pp, axes, counts, tp, n_pos, rot, _layout(layout), _raw_stream(device)))
    if out is not None:
        _written(out)
    return y


def _norm_rope_grad(x, weight, dy, positions, table, eps, layout, sections, needs_x, needs_weight):
    device = x.get_device()
    if _current_device() != device:
        return _on(device, _norm_rope_grad, x, weight, dy, positions, table, eps, layout, sections, needs_x, needs_weight)
    if dy.stride(2) != 1:
        dy = dy.contiguous()
    T, H, D = x.shape
    dx = x.new_empty(T, H, D) if needs_x else None
    dw = weight.new_empty(D) if needs_weight else None
    xs, gs = x.stride(), dy.stride()
    tp, n_pos, rot = _table(table, device)
    wp, wd = _weight(weight, x, device, D)
    pp, axes, counts = _axes(positions, sections, device, T)
    need = lib().gbb_norm_rope_grad_workspace(T, H, D) if needs_weight else 0
    ws = x.new_empty(need, dtype=_torch().uint8) if need else None
    _check(lib().gbb_norm_rope_grad(
        x.data_ptr(), xs[0], xs[1], dy.data_ptr(), gs[0], gs[1], dx.data_ptr() if needs_x else None, H * D, D,
        _dtype_code(x.dtype), T, H, D, wp, wd, eps, pp, axes, counts, tp, n_pos, rot, _layout(layout),
        dw.data_ptr() if needs_weight else None, ws.data_ptr() if need else None, need, _raw_stream(device)))
    return dx, dw


def _differentiable_norm():
    """norm_rope as a torch.autograd.Function, made at its first use."""
    global _NormRope
    if _NormRope is not None:
        return _NormRope
    torch = _torch()

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, positions, table, eps, layout, sections):
            ctx.eps, ctx.layout, ctx.sections = eps, layout, sections
            ctx.save_for_backward(x, weight, positions, table)
            return norm_rope(x, weight, positions, table, eps, layout, sections)   # torch runs this without gradients

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, g):
            x, weight, positions, table = ctx.saved_tensors
            dx, dw = _norm_rope_grad(x, weight, g, positions, table, ctx.eps, ctx.layout, ctx.sections,
                                     ctx.needs_input_grad[0], ctx.needs_input_grad[1])
            return dx, dw, None, None, None, None, None

    _NormRope = NormRope
    return NormRope


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


def rope_append(cache: PagedCache, qkv, q_heads: int, positions, slots, table, layout: str = "half", out=None,
                q_norm=None, k_norm=None, eps: float = 1e-6, sections=None):
    """Rotates the q and k heads of qkv [T][(q_heads + 2 kv heads) head size]
    (rows may be strided), writes k and v to the cache's int32 slots [T] and
    returns q [T][q_heads][head size] (see gbb_rope_append).  q_norm, k_norm:
    weights [head size] (both float32 or both qkv's dtype) of a norm of every q
    and k head before its rotation, as norm_rope.  sections: of positions
    [axes][T], as rope; the cache keeps those of the first axis (see
    gbb_norm_rope_append)."""
    device = cache._index
    if _current_device() != device:
        return _on(device, rope_append, cache, qkv, q_heads, positions, slots, table, layout, out, q_norm, k_norm, eps,
                   sections)
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
    if q_norm is not None or k_norm is not None or sections is not None:
        (qw, qd), (kw, kd) = _weight(q_norm, qkv, device, D, "q_norm"), _weight(k_norm, qkv, device, D, "k_norm")
        if (qw is None) != (kw is None) or qd != kd:
            raise ValueError("q_norm and k_norm must be given together, of one dtype")
        pp, axes, counts = _axes(positions, sections, device, T)
        _check(lib().gbb_norm_rope_append(
            cache._ref, qkv.data_ptr(), stride[0] if T > 1 else width, _dtype_code(qkv.dtype), T, q_heads, qw, kw, qd,
            eps, pp, axes, counts, _ptr(slots, _int32, device, "slots", (T,)), tp, n_pos, rot, _layout(layout), qp,
            _raw_stream(device)))
        return q
    _check(lib().gbb_rope_append(
        cache._ref, qkv.data_ptr(), stride[0] if T > 1 else width, _dtype_code(qkv.dtype), T, q_heads,
        _ptr(positions, _int32, device, "positions", (T,)), _ptr(slots, _int32, device, "slots", (T,)), tp,
        n_pos, rot, _layout(layout), qp, _raw_stream(device)))
    return q


def paged_attention_workspace(cache: PagedCache, batch: int, q_heads: int, max_len: int,
                              with_weights: bool = False, window: int = 0) -> int:
    """Bytes of paged_attention's workspace (with_weights: of a call with
    weights_out).  A new one's first 16384 have to be zero: torch.zeros."""
    return _on(cache._index, lib().gbb_paged_attention_options_workspace, cache._ref, batch, q_heads, max_len,
               int(with_weights), min(window, _INT_MAX))


def _options(device, q_heads, softcap, slopes, window, first=None, prefix=None, tree=None, tokens=0, batch=0):
    """A gbb_attention_options, or None where nothing is asked for."""
    if not softcap and slopes is None and not window and first is None and prefix is None and tree is None:
        return None
    words, window = 0, min(window, _INT_MAX)
    if tree is not None:
        p, shape = _ptr(tree, _int32, device, "tree"), tree.shape
        if len(shape) != 2 or shape[0] != tokens:
            raise ValueError(f"tree must be int32 [{tokens}][words]")
        tree, words = p, shape[1]
    return ctypes.byref(_AttentionOptions(
        softcap, None if slopes is None else _ptr(slopes, _float32, device, "slopes", (q_heads,)), window,
        None if first is None else _ptr(first, _int32, device, "first", (tokens,)),
        None if prefix is None else _ptr(prefix, _int32, device, "prefix", (batch,)), tree, words))


def paged_attention(cache: PagedCache, q, block_table, lengths, max_len: int, scale: float | None = None, out=None,
                    lse=None, weights_out=None, workspace=None, softcap: float = 0.0, slopes=None, window: int = 0):
    """Attention of one new token per sequence, q [B][q_heads][head size],
    over the first lengths[b] <= max_len slots of the pages block_table[b]
    (int32 [B] and [B][pages]); scale defaults to head size ** -0.5.  lse:
    float32 [B][q_heads] to fill.  weights_out: where to write the cache's
    weights with this step's added (cache.weights itself for in place).
    workspace: paged_attention_workspace bytes that were zero when they were
    new (torch.zeros, not empty: outputs would stay unwritten), else the
    binding's own.  softcap: scores s become softcap * tanh(s / softcap).
    slopes: float32 [q_heads], a score then loses slope * distance from the
    newest slot.  window: only so many of the newest slots take part.  Returns
    [B][q_heads][head size] (see gbb_paged_attention and its options)."""
    device, D = cache._index, cache.head_dim
    if _current_device() != device:
        return _on(device, paged_attention, cache, q, block_table, lengths, max_len, scale, out, lse, weights_out,
                   workspace, softcap, slopes, window)
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
            _ptr(lengths, _int32, device, "lengths", (B,)), max_len, D ** -0.5 if scale is None else scale)
    outs = (op, _ptr(lse, _float32, device, "lse", (B, q_heads)) if lse is not None else None, w)
    options = _options(device, q_heads, softcap, slopes, window)
    if options is None:
        call, args = lib().gbb_paged_attention, args + outs
    else:
        call, args = lib().gbb_paged_attention_options, args + (options,) + outs
    _with_workspace("attention", device, workspace, call, args,
                    lambda: paged_attention_workspace(cache, B, q_heads, max_len, w is not None, window))
    return o


def paged_attention_tokens_workspace(cache: PagedCache, tokens: int, batch: int, q_heads: int, max_len: int,
                                     window: int = 0, tree_words: int = 0) -> int:
    """Bytes of paged_attention_tokens' workspace (tree_words: tree.shape[1]).
    A new one's first 16384 have to be zero: torch.zeros."""
    return _on(cache._index, lib().gbb_paged_attention_tokens_workspace, cache._ref, tokens, batch, q_heads, max_len,
               min(window, _INT_MAX), tree_words)


def paged_attention_tokens(cache: PagedCache, q, starts, block_table, lengths, max_len: int,
                           scale: float | None = None, out=None, lse=None, workspace=None, softcap: float = 0.0,
                           slopes=None, window: int = 0, first=None, prefix=None, tree=None):
    """Attention of several new tokens per sequence: q [T][q_heads][head size],
    of which tokens starts[b] ... starts[b + 1] - 1 (int32 [B + 1]) are sequence
    b's, in the last of its lengths[b] <= max_len slots of the pages
    block_table[b].  A token sees the slots up to its own; with `prefix` (int32
    [B]) those below prefix[b] too; with `tree` (int32 [T][words]) all before the
    new ones, and new token j of its sequence where bit j % 32 of word j // 32
    of its row is set.  `first` (int32 [T]) is the first slot that a token sees,
    `window` how near a slot has to be.  softcap and slopes as paged_attention,
    with distances counted along a tree.  lse: float32 [T][q_heads] to fill.
    workspace: paged_attention_tokens_workspace bytes, otherwise as
    paged_attention's.  Returns [T][q_heads][head size]; tokens outside all
    sequences are left as they are (see gbb_paged_attention_tokens)."""
    device, D = cache._index, cache.head_dim
    if _current_device() != device:
        return _on(device, paged_attention_tokens, cache, q, starts, block_table, lengths, max_len, scale, out, lse,
                   workspace, softcap, slopes, window, first, prefix, tree)
    if _device_of(q, "q") != device:
        raise ValueError(f"q is on {q.device}, not on GPU {device}")
    shape, stride = q.shape, q.stride()
    if len(shape) != 3 or shape[2] != D or stride[2] != 1 or (stride[1] != D and shape[1] != 1):
        raise ValueError(f"q must be [T][q_heads][{D}] with contiguous tokens")
    T, q_heads, _ = shape
    bt, table_shape = _ptr(block_table, _int32, device, "block_table"), block_table.shape
    if len(table_shape) != 2:
        raise ValueError("block_table must be int32 [B][pages]")
    B = table_shape[0]
    if out is None:
        o = q.new_empty(T, q_heads, D)
        op = o.data_ptr()
    else:
        o = out
        op = _ptr(o, q.dtype, device, "out", shape)
    options = _options(device, q_heads, softcap, slopes, window, first, prefix, tree, T, B)
    args = (cache._ref, q.data_ptr(), stride[0], _dtype_code(q.dtype), T, B,
            q_heads, _ptr(starts, _int32, device, "starts", (B + 1,)), bt, table_shape[1],
            _ptr(lengths, _int32, device, "lengths", (B,)), max_len, D ** -0.5 if scale is None else scale, options, op,
            _ptr(lse, _float32, device, "lse", (T, q_heads)) if lse is not None else None)
    words = 0 if tree is None else tree.shape[1]
    _with_workspace("attention", device, workspace, lib().gbb_paged_attention_tokens, args,
                    lambda: paged_attention_tokens_workspace(cache, T, B, q_heads, max_len, window, words))
    return o


def cache_keep(cache: PagedCache, block_table, lengths, drafted, kept, counts, lengths_out=None):
    """Keeps of the last drafted[b] of lengths[b] slots those numbered
    kept[b][: counts[b]] (rising; int32 [B], [B], [B][most] and [B]), moved to
    the front of them in place, and returns the new lengths, int32 [B]
    (lengths_out if given; see gbb_cache_keep)."""
    device = cache._index
    if _current_device() != device:
        return _on(device, cache_keep, cache, block_table, lengths, drafted, kept, counts, lengths_out)
    bt = _ptr(block_table, _int32, device, "block_table")
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B][pages]")
    B, pages = block_table.shape
    kp = _ptr(kept, _int32, device, "kept")
    if kept.dim() != 2 or kept.shape[0] != B:
        raise ValueError(f"kept must be int32 [{B}][most]")
    lp = _ptr(lengths, _int32, device, "lengths", (B,))
    n = lengths_out if lengths_out is not None else lengths.new_empty(B)
    _check(lib().gbb_cache_keep(cache._ref, B, bt, pages, lp, _ptr(drafted, _int32, device, "drafted", (B,)), kp,
                                kept.shape[1], _ptr(counts, _int32, device, "counts", (B,)),
                                _ptr(n, _int32, device, "lengths_out", (B,)), _raw_stream(device)))
    return n


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

"""Rotary positions, the paged key-value cache and its attention: the binding
of gbb_rope*, gbb_paged_attention* and gbb_cache_evict* (include/gbb.h states
what each computes).

A decoding step around the quantized products:

    qkv = gemm_mixed_w(...)                                    # [T][(Hq + 2 Hkv) D]
    q = rope_append(cache, qkv, Hq, positions, slots, table)   # k, v -> cache
    o = paged_attention(cache, q, block_table, lengths, max_len)
    y = gemm_mixed_w(..., o.view(T, -1))

Every call enqueues on torch's current stream of the cache's (or x's) device.
"""
from __future__ import annotations

import ctypes

import numpy as np

from .binding import _check, _dev_ptr, _np_ptr, _PagedCache, _RopeScaling, _stream, _torch, lib

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


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _ints(t, shape, name):
    p = _dev_ptr(t, _torch().int32, name)
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be int32 {list(shape)}, got {list(t.shape)}")
    return p


# ----------------------------------------------------------------------------
# rotary positions
# ----------------------------------------------------------------------------
def rope_table(rot: int, n_pos: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
               original_len: float = 0.0, low: float = 1.0, high: float = 4.0, attention: float = 1.0) -> np.ndarray:
    """float32 [n_pos][rot/2][2] of (cos, sin) on the host (see
    gbb_rope_table); scaling is plain, linear, bands or yarn."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    table = np.empty((max(0, n_pos), max(0, rot) // 2, 2), np.float32)
    s = _RopeScaling(_SCALINGS[scaling], factor, original_len, low, high, attention)
    _check(lib().gbb_rope_table(rot, n_pos, float(base), ctypes.byref(s), _np_ptr(table)))
    return table


def _table(table, device):
    p = _dev_ptr(table, _torch().float32, "table")
    if table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be float32 [n_pos][rot/2][2]")
    _same_device(device, table=table)
    return p, table.shape[0], 2 * table.shape[1]


def rope(x, positions, table, layout: str = "half", transpose: bool = False, out=None):
    """x [T][H][D] (float16, bfloat16 or float32; the last dimension
    contiguous) with its first 2 * table.shape[1] elements rotated to int32
    positions [T].  out: where to write (x itself for in place), else a new
    contiguous tensor.  transpose: the transposed rotation, which is the
    gradient with respect to x."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise TypeError("x must be a torch tensor on a GPU")
    if x.dim() != 3 or x.stride(2) != 1:
        raise ValueError("x must be [T][H][D] with contiguous heads")
    T, H, D = x.shape
    y = out if out is not None else torch.empty((T, H, D), dtype=x.dtype, device=x.device)
    if y.dtype != x.dtype or y.shape != x.shape or y.stride(2) != 1:
        raise ValueError("out must be like x, with contiguous heads")
    _same_device(x.device, out=y, positions=positions)
    tp, n_pos, rot = _table(table, x.device)
    xs, ys = x.stride(), y.stride()
    _check(lib().gbb_rope(x.data_ptr(), xs[0], xs[1], y.data_ptr(), ys[0], ys[1], _dtype_code(x.dtype), T, H, D,
                          _ints(positions, (T,), "positions"), tp, n_pos, rot, _layout(layout), int(transpose),
                          _stream(x)))
    return y


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
        torch = _torch()
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [pages][kv heads][page][head size] of one dtype")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.weights, self.positions = weights, positions
        self.device, self.dtype = k.device, k.dtype
        self.num_pages, self.kv_heads, self.page, self.head_dim = k.shape
        _same_device(k.device, v=v, k_scale=k_scale, v_scale=v_scale, weights=weights, positions=positions)
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and tuple(t.shape) != (self.kv_heads,):
                raise ValueError(f"{name} must be float32 [{self.kv_heads}]")
        for name, t in (("weights", weights), ("positions", positions)):
            if t is not None and t.shape != k.shape[:3]:
                raise ValueError(f"{name} must be {list(k.shape[:3])}")

        def ptr(t, dtype, name):
            return None if t is None else _dev_ptr(t, dtype, name)

        code = _dtype_code(k.dtype)
        if code == 2:
            raise TypeError("a cache holds float16, bfloat16 or float8_e4m3fn")
        self._c = _PagedCache(ptr(k, k.dtype, "k"), ptr(v, v.dtype, "v"), ptr(k_scale, torch.float32, "k_scale"),
                              ptr(v_scale, torch.float32, "v_scale"), ptr(weights, torch.float32, "weights"),
                              ptr(positions, torch.int32, "positions"), code, self.num_pages, self.page,
                              self.kv_heads, self.head_dim)
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

    def _state(self, t, like, name):
        """Pointer of an output like the cache's weights or positions."""
        if t.shape != like.shape:
            raise ValueError(f"{name} must be {list(like.shape)}")
        _same_device(self.device, **{name: t})
        return _dev_ptr(t, like.dtype, name)


_ws_cache: dict = {}


def _workspace(kind: str, device, nbytes: int):
    """A device buffer per use, device and stream, zero when it is new.  Kept
    apart from the buffer of the gemm calls, which has to stay zero."""
    torch = _torch()
    if nbytes == 0:
        return None
    key = (kind, device, torch.cuda.current_stream(device).cuda_stream)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def rope_append(cache: PagedCache, qkv, q_heads: int, positions, slots, table, layout: str = "half", out=None):
    """Rotates the q and k heads of qkv [T][(q_heads + 2 kv heads) head size]
    (rows may be strided), writes k and v to the cache's int32 slots [T] and
    returns q [T][q_heads][head size] (see gbb_rope_append)."""
    torch = _torch()
    if not isinstance(qkv, torch.Tensor) or qkv.device.type != "cuda":
        raise TypeError("qkv must be a torch tensor on a GPU")
    width = (q_heads + 2 * cache.kv_heads) * cache.head_dim
    if qkv.dim() != 2 or qkv.shape[1] != width or qkv.stride(1) != 1:
        raise ValueError(f"qkv must be [T][{width}] with contiguous rows")
    T = qkv.shape[0]
    q = out if out is not None else torch.empty((T, q_heads, cache.head_dim), dtype=qkv.dtype, device=qkv.device)
    if tuple(q.shape) != (T, q_heads, cache.head_dim):
        raise ValueError(f"out must be [{T}][{q_heads}][{cache.head_dim}]")
    _same_device(cache.device, qkv=qkv, out=q, positions=positions, slots=slots)
    tp, n_pos, rot = _table(table, cache.device)
    stride = qkv.stride(0) if T > 1 else width
    _check(lib().gbb_rope_append(cache._ref, qkv.data_ptr(), stride, _dtype_code(qkv.dtype), T, q_heads,
                                 _ints(positions, (T,), "positions"), _ints(slots, (T,), "slots"), tp, n_pos, rot,
                                 _layout(layout), _dev_ptr(q, qkv.dtype, "out"), _stream(qkv)))
    return q


def paged_attention_workspace(cache: PagedCache, batch: int, q_heads: int, max_len: int,
                              with_weights: bool = False) -> int:
    return lib().gbb_paged_attention_workspace(cache._ref, batch, q_heads, max_len, int(with_weights))


def paged_attention(cache: PagedCache, q, block_table, lengths, max_len: int, scale: float | None = None, out=None,
                    lse=None, weights_out=None, workspace=None):
    """Attention of one new token per sequence, q [B][q_heads][head size],
    over the first lengths[b] <= max_len slots of the pages block_table[b]
    (int32 [B] and [B][pages]); scale defaults to head size ** -0.5.  lse:
    float32 [B][q_heads] to fill.  weights_out: where to write the cache's
    weights with this step's added (cache.weights itself for in place).
    Returns [B][q_heads][head size] (see gbb_paged_attention)."""
    torch = _torch()
    if not isinstance(q, torch.Tensor) or q.device.type != "cuda":
        raise TypeError("q must be a torch tensor on a GPU")
    if q.dim() != 3 or q.shape[2] != cache.head_dim or q.stride(2) != 1 or q.stride(1) != cache.head_dim:
        raise ValueError(f"q must be [B][q_heads][{cache.head_dim}] with contiguous tokens")
    B, q_heads = q.shape[0], q.shape[1]
    o = out if out is not None else torch.empty((B, q_heads, cache.head_dim), dtype=q.dtype, device=q.device)
    if o.shape != q.shape:
        raise ValueError(f"out must be {list(q.shape)}")
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError(f"block_table must be int32 [{B}][pages]")
    _same_device(cache.device, q=q, out=o, block_table=block_table, lengths=lengths, lse=lse, workspace=workspace)
    if lse is not None and tuple(lse.shape) != (B, q_heads):
        raise ValueError(f"lse must be float32 [{B}][{q_heads}]")
    w = None
    if weights_out is not None:
        if cache.weights is None:
            raise ValueError("the cache has no weights")
        w = cache._state(weights_out, cache.weights, "weights_out")
    L = lib()
    ws = workspace
    if ws is None:
        ws = _workspace("attention", cache.device,
                        L.gbb_paged_attention_workspace(cache._ref, B, q_heads, max_len, int(w is not None)))
    _check(L.gbb_paged_attention(
        cache._ref, q.data_ptr(), q.stride(0), _dtype_code(q.dtype), B, q_heads,
        _dev_ptr(block_table, torch.int32, "block_table"), block_table.shape[1], _ints(lengths, (B,), "lengths"),
        max_len, cache.head_dim ** -0.5 if scale is None else scale, _dev_ptr(o, q.dtype, "out"),
        _dev_ptr(lse, torch.float32, "lse") if lse is not None else None, w,
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0, _stream(q)))
    return o


def cache_evict_workspace(cache: PagedCache, batch: int, max_len: int, budget: int) -> int:
    return lib().gbb_cache_evict_workspace(cache._ref, batch, max_len, budget)


def cache_evict(cache: PagedCache, block_table, lengths, max_len: int, budget: int, recent: int, weights_out=None,
                positions_out=None, lengths_out=None, workspace=None):
    """Cuts every sequence longer than budget to budget slots: per kv head
    the `recent` newest positions and the slots of the largest weight (see
    gbb_cache_evict).  weights_out, positions_out: default in place.  Returns
    the new lengths, int32 [B] (lengths_out if given)."""
    torch = _torch()
    if cache.weights is None or cache.positions is None:
        raise ValueError("eviction needs a cache with weights and positions")
    B = block_table.shape[0]
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B][pages]")
    n = lengths_out if lengths_out is not None else torch.empty((B,), dtype=torch.int32, device=cache.device)
    _same_device(cache.device, block_table=block_table, lengths=lengths, lengths_out=n, workspace=workspace)
    w = cache._c.weights if weights_out is None else cache._state(weights_out, cache.weights, "weights_out")
    p = cache._c.positions if positions_out is None else cache._state(positions_out, cache.positions, "positions_out")
    L = lib()
    ws = workspace
    if ws is None:
        ws = _workspace("evict", cache.device, L.gbb_cache_evict_workspace(cache._ref, B, max_len, budget))
    _check(L.gbb_cache_evict(
        cache._ref, B, _dev_ptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        _ints(lengths, (B,), "lengths"), max_len, budget, recent, _ints(n, (B,), "lengths_out"), w, p,
        ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0, _stream(cache.k)))
    return n

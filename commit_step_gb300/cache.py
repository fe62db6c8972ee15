"""The paged 8-bit key/value cache of a block decoder: appending tokens,
attending over them, and evicting the least attended (``dllm_cache_append``,
``dllm_cache_attention``, ``dllm_cache_evict``)."""
from __future__ import annotations

import ctypes as C
import threading
from typing import Optional

import torch

from . import _F32, _I32, _MASK, _arg, _check, _lib, _need_cuda

_I64x3 = C.c_int64 * 3
_BF16 = (torch.bfloat16,)


class _CacheStruct(C.Structure):
    """Mirror of ``dllm_kv_cache``."""

    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("num_pages", C.c_int64), ("page_size", C.c_int32), ("heads", C.c_int32), ("head_dim", C.c_int32)]


class KVCache:
    """A pool of pages of e4m3 keys and values with one scale per page and head.

    ``k`` and ``v``: (num_pages, heads, page_size, head_dim) float8_e4m3fn;
    ``k_scale`` and ``v_scale``: (num_pages, heads) float32.  A cached value
    is its code times its page's scale.  The caller deals the pages out in
    page tables, (B, width) int32 tensors.
    """

    def __init__(self, num_pages: int, page_size: int, heads: int, head_dim: int, device=None):
        dev = device or "cuda"
        shape = (num_pages, heads, page_size, head_dim)
        k = torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        v = torch.zeros(shape, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        self._hold(k, v, torch.ones((num_pages, heads), device=dev), torch.ones((num_pages, heads), device=dev))

    @classmethod
    def from_tensors(cls, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor) -> "KVCache":
        """A cache over existing pools (float8_e4m3fn, or uint8 holding the codes)."""
        self = cls.__new__(cls)
        self._hold(k, v, k_scale, v_scale)
        return self

    def _hold(self, k, v, k_scale, v_scale) -> None:
        _need_cuda(k, v, k_scale, v_scale)
        if k.dim() != 4:
            raise ValueError("k must be (num_pages, heads, page_size, head_dim)")
        pages, heads, page_size, head_dim = k.shape
        codes = (torch.float8_e4m3fn, torch.uint8)
        _arg(k, "k", k.numel(), codes, k.device)
        _arg(v, "v", k.numel(), codes, k.device)
        if v.shape != k.shape:
            raise ValueError("k and v must have one shape")
        _arg(k_scale, "k_scale", pages * heads, _F32, k.device)
        _arg(v_scale, "v_scale", pages * heads, _F32, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.head_dim = pages, heads, page_size, head_dim
        self.device, self.index = k.device, k.get_device()
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages,
                                    page_size, heads, head_dim)
        self._ref = C.byref(self._struct)


def _at(t, name: str, numel: int, dtypes, index: int, device) -> int:
    """The address of a tensor that passes ``_arg``'s checks (a call's cost on
    the host is mostly these checks, so the usual case is decided here)."""
    try:
        if t.get_device() == index and t.dtype in dtypes and t.numel() == numel and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if t is None:
        raise ValueError(f"{name} is needed")
    _arg(t, name, numel, dtypes, device)
    raise ValueError(f"{name} is not a tensor this call can use")


def _at_or_none(t, name: str, numel: int, dtypes, index: int, device):
    return None if t is None else _at(t, name, numel, dtypes, index, device)


def _table(cache: KVCache, table: torch.Tensor, name: str = "page_table"):
    """(B, width, address) of a page table."""
    if not torch.is_tensor(table) or table.dim() != 2:
        raise ValueError(f"{name} must be a (B, width) int32 tensor")
    B, width = table.shape
    return B, width, _at(table, name, B * width, _I32, cache.index, cache.device)


def _strided(t, name: str, shape, device):
    """The three outer strides of a bf16 (B, L, heads, head_dim) tensor."""
    if not torch.is_tensor(t) or t.dtype != torch.bfloat16 or t.dim() != 4:
        raise TypeError(f"{name} must be a 4-D bfloat16 tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}; the cache is on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    sb, sl, sh, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"{name} needs unit stride over its last dimension")
    # (a dimension of one element has no stride that matters)
    return _I64x3(sb if shape[0] > 1 else 0, sl if shape[1] > 1 else 0, sh if shape[2] > 1 else 0)


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _raw_stream(stream, index: int) -> int:
    """The stream a call runs on: the given one, or the device's current one.  The
    library launches on the current device, so that has to be the tensors' device
    (another one's default stream has the same handle, and no use for their
    addresses)."""
    current = torch._C._cuda_getDevice()
    if current != index:
        raise ValueError(f"the tensors are on cuda:{index}; the current device is cuda:{current}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"the tensors are on cuda:{index}; the stream is on {stream.device}")
    return stream.cuda_stream


def cache_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
                 count: Optional[torch.Tensor] = None, stream=None) -> None:
    """Writes the keys and values of L new tokens per sequence, (B, L, heads,
    head_dim) bf16 of any outer strides, at positions start[b] .. start[b] +
    L - 1 (the first count[b] of them when ``count`` is given)."""
    B, width, table = _table(cache, page_table)
    if not torch.is_tensor(k) or k.dim() != 4:
        raise TypeError("k must be a 4-D bfloat16 tensor")
    L, dev, idx = k.shape[1], cache.device, cache.index
    shape = (B, L, cache.heads, cache.head_dim)
    ks, vs = _strided(k, "k", shape, dev), _strided(v, "v", shape, dev)
    _check(_lib.dllm_cache_append(cache._ref, k.data_ptr(), v.data_ptr(), ks, vs, B, L, table, width,
                                  _at(start, "start", B, _I32, idx, dev),
                                  _at_or_none(count, "count", B, _I32, idx, dev), _raw_stream(stream, idx)),
           "dllm_cache_append")


_NEED = {}


def _attention_need(L: int, Hq: int, cache: KVCache) -> int:
    """The bytes of workspace that L queries of Hq heads per sequence need, however
    many sequences there are.  Kept by all that the library's answer depends on:
    a size asked for by a call that is empty or refused must answer no other."""
    size = (cache.index, L, Hq, cache.heads, cache.head_dim)
    need = _NEED.get(size)
    if need is None:
        need = _NEED[size] = int(_lib.dllm_cache_attention_workspace_size(1, L, Hq, cache.heads, cache.head_dim))
    return need


_KEPT = threading.local()


def _attention_ws(L: int, Hq: int, cache: KVCache, raw: int) -> torch.Tensor:
    """A workspace for a call on the current stream.  A call's launches pass its
    parts on through it, so it is kept for later calls of the same host thread on
    the same stream only: those of another thread may be enqueued in between.  A
    call that is captured gets memory of its graph's, which is not kept, and no
    kept one, which a later call may replace.  (Allocated anew for every call,
    large blocks cost the host 2 to 5 of its 16 us for a single token.)"""
    need = _attention_need(L, Hq, cache)
    if torch.cuda.is_current_stream_capturing():
        return _empty((need,), torch.uint8, cache.device, None)
    try:
        kept = _KEPT.ws
    except AttributeError:
        kept = _KEPT.ws = {}
    ws = kept.get((cache.index, raw))
    if ws is None or ws.numel() < need:
        ws = kept[(cache.index, raw)] = _empty((need,), torch.uint8, cache.device, None)
    return ws


def cache_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, lens: torch.Tensor,
                    scale: Optional[float] = None, key_mask: Optional[torch.Tensor] = None,
                    weights: Optional[torch.Tensor] = None, decay: float = 1.0, out=None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """Attention of q (B, L, Hq, head_dim) bf16 over each sequence's first
    lens[b] cached tokens.  Returns (out bf16 like q, contiguous; lse (B, L,
    Hq) float32).

    ``scale`` defaults to 1 / sqrt(head_dim).  ``key_mask``: (B, width *
    page_size) uint8 / bool, 0 for tokens that are not attended.  ``weights``:
    (B, heads, width * page_size) float32, updated in place to decay * weights
    + the probability each token drew.  ``out``: preallocated (out, lse).
    ``ws``: a workspace of the caller's, not in use by another call; zeroed, it
    tells ``workspace_fault`` afterwards whether a wait ran out.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_attention(q, cache, page_table, lens, scale, key_mask, weights, decay, out, ws)
    B, width, table = _table(cache, page_table)
    if not torch.is_tensor(q) or q.dim() != 4:
        raise TypeError("q must be a 4-D bfloat16 tensor")
    L, Hq = q.shape[1], q.shape[2]
    dev, idx, heads, D = cache.device, cache.index, cache.heads, cache.head_dim
    strides = _strided(q, "q", (B, L, Hq, D), dev)
    cap = width * cache.page_size
    if out is None:
        o, lse = _empty((B, L, Hq, D), torch.bfloat16, dev, None), _empty((B, L, Hq), torch.float32, dev, None)
        out_at, lse_at = o.data_ptr(), lse.data_ptr()
    else:
        o, lse = out
        out_at = _at(o, "out", B * L * Hq * D, _BF16, idx, dev)
        lse_at = _at(lse, "lse", B * L * Hq, _F32, idx, dev)
    raw = _raw_stream(None, idx)
    if ws is None:
        ws = _attention_ws(L, Hq, cache, raw)
    elif not torch.is_tensor(ws):
        raise TypeError("ws must be a tensor")
    else:
        _arg(ws, "ws", ws.numel(), (ws.dtype,), dev)
    _check(_lib.dllm_cache_attention(cache._ref, q.data_ptr(), strides, B, L, Hq, table, width,
                                     _at(lens, "lens", B, _I32, idx, dev),
                                     _at_or_none(key_mask, "key_mask", B * cap, _MASK, idx, dev),
                                     0 if key_mask is None else cap, D ** -0.5 if scale is None else scale, out_at,
                                     lse_at, _at_or_none(weights, "weights", B * heads * cap, _F32, idx, dev), decay,
                                     ws.data_ptr(), ws.numel(), raw), "dllm_cache_attention")
    return o, lse


def cache_evict(cache: KVCache, page_table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor, budget: int,
                dst_table: torch.Tensor, keep_first: int = 0, keep_last: int = 0, out=None, stream=None):
    """Copies, per sequence and head, the ``budget`` tokens to keep (the first
    keep_first, the last keep_last, and the largest ``weights`` of the rest)
    into the pages of ``dst_table`` (other pages than ``page_table``'s).
    Returns (keep (B, heads, budget) int32: the old positions in order, -1
    behind the last; lens (B) int32; weights like ``weights``, moved along).
    ``out``: those three, preallocated."""
    B, width, table = _table(cache, page_table)
    B2, dst_width, dst = _table(cache, dst_table, "dst_table")
    if B2 != B:
        raise ValueError("page_table and dst_table must have one row per sequence")
    budget, dev, idx, heads = int(budget), cache.device, cache.index, cache.heads
    cap, kept = width * cache.page_size, max(budget, 0)
    if out is None:
        out = (_empty((B, heads, kept), torch.int32, dev, stream), _empty((B,), torch.int32, dev, stream),
               _empty((B, heads, cap), torch.float32, dev, stream))
    keep, lens_out, weights_out = out
    _check(_lib.dllm_cache_evict(cache._ref, table, width, _at(lens, "lens", B, _I32, idx, dev), B,
                                 _at(weights, "weights", B * heads * cap, _F32, idx, dev), budget, int(keep_first),
                                 int(keep_last), dst, dst_width, _at(keep, "keep", B * heads * kept, _I32, idx, dev),
                                 _at(lens_out, "lens_out", B, _I32, idx, dev),
                                 _at(weights_out, "weights_out", B * heads * cap, _F32, idx, dev),
                                 _raw_stream(stream, idx)), "dllm_cache_evict")
    return keep, lens_out, weights_out

"""The 4-bit key/value cache: append, read, attention of new tokens, gathered
attention weight, eviction.  Binding of the fp4attn_kv_* calls, whose
declarations in ``include/fp4attn.h`` define layouts and results; every check
that needs no look at device memory is made here, before the call.

One step of generation::

    cache = empty_kv_cache(num_pages, heads, D, "cuda")
    lens += 1                                     # tokens, the new one included
    kv_append(k, v, cache, table, lens)           # k, v: [B, heads, D]
    o, lse = kv_attention(q, cache, table, lens)  # q: [B, heads * group, D]
    kv_accumulate(q, lse, weights, cache, table, lens)   # only where tokens are to be evicted

A prompt or drafted tokens take the same calls with several rows per sequence
(``cu``: int32 [B + 1] row offsets; without it every sequence has T / B rows).

With ``stream`` (a torch stream or a handle) a call runs on that stream.  Its
inputs have to be ready there, and whoever reads its results on another stream
waits for it, as with torch's own operations.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
from dataclasses import dataclass

import torch

from . import Fp4AttnError, lib

KV_PAGE = 64

# fp4attn_kv_cache_t and fp4attn_kv_batch_t, as bytes: packing one takes a fifth
# of the time of filling a ctypes structure, and small calls are bound by such.
_pack_cache = struct.Struct("@Piiiii").pack
_pack_batch = struct.Struct("@PPPiii").pack


def _Cache(pages, num_pages, heads, D, k_exp, v_exp):
    return _pack_cache(pages or 0, num_pages, heads, D, k_exp, v_exp)


def _Batch(table, lens, cu, B, max_pages, T):
    return _pack_batch(table or 0, lens or 0, cu or 0, B, max_pages, T)


@functools.lru_cache(maxsize=None)
def _L():
    L = lib()
    vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    c = b = ctypes.c_char_p
    L.fp4attn_kv_page_bytes.argtypes = [i, i, ctypes.POINTER(sz)]
    L.fp4attn_kv_append.argtypes = [c, b, vp, ll, ll, vp, ll, ll, vp]
    L.fp4attn_kv_read.argtypes = [c, b, vp, vp, vp]
    L.fp4attn_kv_attention_workspace_bytes.argtypes = [i, i, i, i, i, i, ctypes.POINTER(sz)]
    L.fp4attn_kv_attention.argtypes = [c, b, vp, ll, ll, i, i, f, f, i, vp, vp, vp, vp, sz, vp]
    L.fp4attn_kv_accumulate.argtypes = [c, b, vp, ll, ll, i, i, f, f, i, vp, vp, vp, i, f, vp]
    L.fp4attn_kv_evict.argtypes = [c, b, vp, i, vp, i, i, i, i, vp, vp, vp, vp]
    return L


def _check(status, name):
    if status:
        raise Fp4AttnError(status, name)


@dataclass
class KVCache:
    """Pages of K and V in 4 bits: u8 [num_pages, heads, 72 D] (64 tokens a page), and the exponents
    of the tensor scales 2^k_exp and 2^v_exp."""
    pages: torch.Tensor
    D: int
    k_exp: int = 0
    v_exp: int = 0

    @property
    def heads(self) -> int:
        return self.pages.shape[1]


def _in_32_bits(*numbers):
    """ctypes cuts a number to its low bits without a word."""
    if not all(-2 ** 31 <= x < 2 ** 31 for x in numbers):
        raise ValueError("%s: sizes must be numbers that 32 bits hold" % (numbers,))


def kv_page_bytes(heads: int, D: int) -> int:
    """Bytes of one page (64 tokens) of all KV heads."""
    _in_32_bits(heads, D)
    n = ctypes.c_size_t()
    _check(_L().fp4attn_kv_page_bytes(heads, D, ctypes.byref(n)), "fp4attn_kv_page_bytes")
    return n.value


def empty_kv_cache(num_pages: int, heads: int, D: int, device, k_exp: int = 0, v_exp: int = 0) -> KVCache:
    """A pool of pages.  Values up to 2688 * 2^exp in magnitude are held without clipping, and blocks
    whose largest value is 0.1 * 2^exp or more keep the full precision of their scale."""
    kv_page_bytes(heads, D)  # refuses what the library does not support
    return KVCache(torch.zeros((num_pages, heads, 72 * D), dtype=torch.uint8, device=device), D, k_exp, v_exp)


# The checks below run on every call, also on those whose kernel takes a few
# microseconds: each looks at an attribute once and builds no message before it
# is needed.  Devices are compared by index (-1: the CPU).

_MOST = 2 ** 31 - 1  # of a number for the library; more than it accepts of any
_Tensor, _i32, _f32, _bf16, _u8 = torch.Tensor, torch.int32, torch.float32, torch.bfloat16, torch.uint8
# (not there in a torch without CUDA, where every call stops at its checks)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _elsewhere(t, name, dev):
    return ValueError("%s is on %s, the cache on %s" % (name, t.device, torch.device("cuda", dev) if dev >= 0 else "cpu"))


def _index_shape(t, name, dev):
    if not isinstance(t, _Tensor) or t.dtype is not _i32 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor" % name)
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    return t.shape


def _geometry(cache, table, lens, cu, T, rows=True):
    """(cache, batch) as the library takes them, after the checks of everything they point to; and (device index,
    KV heads, D, B, table width)."""
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    pages, D = cache.pages, cache.D
    shape = pages.shape if isinstance(pages, _Tensor) else ()
    if len(shape) != 3 or (D != 64 and D != 128) or shape[2] != 72 * D or pages.dtype is not _u8 or \
            not pages.is_contiguous():
        raise ValueError("cache.pages must be a contiguous u8 tensor [num_pages, heads, 72 D], D in {64, 128}")
    dev = pages.get_device()
    ts = _index_shape(table, "table", dev)
    if len(ts) != 2:
        raise ValueError("table must be [B, max_pages]")
    B, M = ts
    ls = _index_shape(lens, "lens", dev)
    if len(ls) != 1 or ls[0] != B:
        raise ValueError("lens must have shape (%d,), not %s" % (B, tuple(ls)))
    at = 0
    if cu is not None:
        cs = _index_shape(cu, "cu", dev)
        if len(cs) != 1 or cs[0] != B + 1:
            raise ValueError("cu must have shape (%d,), not %s" % (B + 1, tuple(cs)))
        at = cu.data_ptr()
    elif rows and (B == 0 or T % B):
        raise ValueError("%d rows do not divide among %d sequences: cu is needed" % (T, B))
    num_pages, heads, _ = shape
    try:
        return (_pack_cache(pages.data_ptr(), num_pages, heads, D, cache.k_exp, cache.v_exp),
                _pack_batch(table.data_ptr(), lens.data_ptr(), at, B, M, T), dev, heads, D, B, M)
    except struct.error:
        raise ValueError("exponents %r, %r and sizes %s must be whole numbers that 32 bits hold"
                         % (cache.k_exp, cache.v_exp, (num_pages, heads, B, M, T))) from None


def _rows(t):
    """Number of packed rows, or 0 for what is refused later."""
    return t.shape[0] if isinstance(t, _Tensor) and t.dim() else 0


def _check_rows(t, name, heads, D, dev, T):
    """bf16 [T, heads, D] with contiguous channels and 16-byte aligned rows; (address, row stride, head stride)."""
    if not isinstance(t, _Tensor) or t.dtype is not _bf16 or t.dim() != 3:
        raise ValueError("%s must be a bf16 tensor [T, heads, D]" % name)
    n, h, d = t.shape
    if n != T or h != heads or d != D:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (T, heads, D)))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    r, s, e = t.stride()
    if n == 1:  # a stride that addresses nothing may be anything
        r = 0
    if h == 1:
        s = 0
    at = t.data_ptr()
    if (e != 1 or (r | s) & 7 or at & 15) and n:
        raise ValueError("%s needs contiguous channels, strides that are multiples of 8 and a 16-byte aligned start" % name)
    return at, r, s


def _check_out(t, name, dtype, shape, dev):
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s" % (name, dtype, tuple(shape)))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    return t


def _stream_of(stream, dev):
    """(handle, torch stream or None: the current one).  The last check of every call."""
    if dev < 0:
        raise ValueError("the cache must be on a CUDA device")
    if stream is None:
        return _raw_stream(dev), None
    if not isinstance(stream, torch.cuda.Stream):
        device = torch.device("cuda", dev)
        stream = torch.cuda.ExternalStream(int(stream), device=device) if stream else torch.cuda.default_stream(device)
    elif stream.device.index != dev:
        raise ValueError("stream belongs to %s, the cache to cuda:%d" % (stream.device, dev))
    handle = stream.cuda_stream
    return handle, None if handle == _raw_stream(dev) else stream


def _scratch(shape, dtype, dev, side):
    """Memory that the call alone uses.  What a side stream writes comes from that stream's memory: a block of the
    current stream may still be in use by kernels that the side stream does not wait for."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(side):
        return torch.empty(shape, dtype=dtype, device=dev)


def _new(shape, dtype, dev, side):
    """An output made by the call; one of a side stream is not reused there before the current stream, whose caller
    gets it, is past it."""
    t = _scratch(shape, dtype, dev, side)
    if side is not None:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _launch(dev, name, *args):
    """Calls the library, which launches on the current device: that of the tensors, made current where it is not."""
    if _current_device() == dev:
        status = getattr(_L(), name)(*args)
    else:
        with torch.cuda.device(dev):
            status = getattr(_L(), name)(*args)
    if status:
        raise Fp4AttnError(status, name)


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
              cu: torch.Tensor | None = None, stream=None) -> None:
    """fp4attn_kv_append: writes the new tokens' K and V rows (bf16 [T, heads, D], any row and head strides)
    at the last slots of their sequences.  lens counts the new tokens already."""
    T = _rows(k)
    c, b, dev, heads, D, _, _ = _geometry(cache, table, lens, cu, T)
    kp, kr, kh = _check_rows(k, "k", heads, D, dev, T)
    vp, vr, vh = _check_rows(v, "v", heads, D, dev, T)
    handle, _ = _stream_of(stream, dev)
    _launch(dev, "fp4attn_kv_append", c, b, kp, kr, kh, vp, vr, vh, handle)


def kv_read(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, total: int, cu: torch.Tensor | None = None,
            k: torch.Tensor | None = None, v: torch.Tensor | None = None, stream=None):
    """fp4attn_kv_read: the stored values of each sequence's last tokens, total rows in all (cu: which are whose;
    without it total / B each); (K, V) bf16 [total, heads, D]."""
    if total < 0:
        raise ValueError("total must not be negative")
    c, b, dev, heads, D, _, _ = _geometry(cache, table, lens, cu, total)
    shape = (total, heads, D)
    if k is not None:
        _check_out(k, "k", _bf16, shape, dev)
    if v is not None:
        _check_out(v, "v", _bf16, shape, dev)
    handle, side = _stream_of(stream, dev)
    if k is None:
        k = _new(shape, _bf16, dev, side)
    if v is None:
        v = _new(shape, _bf16, dev, side)
    _launch(dev, "fp4attn_kv_read", c, b, k.data_ptr(), v.data_ptr(), handle)
    return k, v


# What the library answers for these numbers on a device; no need to ask twice.
@functools.lru_cache(maxsize=1024)
def _workspace_of(dev, *sizes):
    with torch.cuda.device(dev):
        return kv_attention_workspace_bytes(*sizes)


def kv_attention_workspace_bytes(heads: int, D: int, B: int, max_pages: int, group: int, max_new: int) -> int:
    """Bytes of kv_attention's workspace for a table [B, max_pages] (0: none needed)."""
    _in_32_bits(heads, D, B, max_pages, group, max_new)
    n = ctypes.c_size_t()
    _check(_L().fp4attn_kv_attention_workspace_bytes(heads, D, B, max_pages, group, max_new, ctypes.byref(n)),
           "fp4attn_kv_attention_workspace_bytes")
    return n.value


def _queries(q, dev, heads, D, B, T, cu, max_new, softmax_scale, softcap, window, slopes):
    """Checks and defaults shared by attention and weights: (address, row stride, head stride, group, max_new, scale,
    slopes)."""
    Hq = q.shape[1] if isinstance(q, _Tensor) and q.dim() == 3 else 0
    if Hq == 0 or Hq % heads:
        raise ValueError("q must be [T, heads * group, D] over the cache's %d KV heads" % heads)
    at, r, s = _check_rows(q, "q", Hq, D, dev, T)
    each = T if cu is not None else T // B
    if max_new is None:
        max_new = each
    elif not 0 <= max_new <= each or (cu is None and max_new != each):
        raise ValueError("max_new = %s does not fit %d rows of %d sequences" % (max_new, T, B))
    scale = D ** -0.5 if softmax_scale is None else softmax_scale
    if not (0 < scale < math.inf and 0 <= softcap < math.inf and 0 <= window < 2 ** 31):
        raise ValueError("softmax_scale must be positive, softcap and window not negative, window below 2^31")
    slope_at = None if slopes is None else _check_out(slopes, "slopes", _f32, (Hq,), dev).data_ptr()
    return at, r, s, Hq // heads, max_new, scale, slope_at


def kv_attention(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                 cu: torch.Tensor | None = None, max_new: int | None = None, softmax_scale: float | None = None,
                 softcap: float = 0.0, window: int = 0, slopes: torch.Tensor | None = None,
                 o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None):
    """fp4attn_kv_attention: attention of the new tokens' queries (bf16 [T, heads * group, D]) over the cache, the
    new tokens included; (O bf16 like q, LSE fp32 [T, heads * group]).  max_new: the most new tokens of a sequence
    (with cu; T where it is not known, at the price of a kernel made for long prompts)."""
    T = _rows(q)
    c, b, dev, heads, D, B, M = _geometry(cache, table, lens, cu, T)
    at, r, s, group, max_new, scale, slope_at = _queries(q, dev, heads, D, B, T, cu, max_new, softmax_scale, softcap,
                                                         window, slopes)
    shape = q.shape
    if o is not None:
        _check_out(o, "o", _bf16, shape, dev)
    if lse is not None:
        _check_out(lse, "lse", _f32, shape[:2], dev)
    if workspace is not None and (not isinstance(workspace, _Tensor) or workspace.dtype is not _u8 or
                                  not workspace.is_contiguous() or workspace.get_device() != dev):
        raise ValueError("workspace must be a contiguous u8 tensor on the cache's device")
    handle, side = _stream_of(stream, dev)
    if o is None:
        o = _new(shape, _bf16, dev, side)
    if lse is None:
        lse = _new(shape[:2], _f32, dev, side)
    if workspace is None:
        need, ws_at = _workspace_of(dev, heads, D, B, M, group, max_new), None
        if need:
            workspace = _scratch((need,), _u8, dev, side)
            ws_at = workspace.data_ptr()
    else:
        need, ws_at = workspace.numel(), workspace.data_ptr()
    _launch(dev, "fp4attn_kv_attention", c, b, at, r, s, group, max_new, scale, softcap, window, slope_at, o.data_ptr(),
            lse.data_ptr(), ws_at, need, handle)
    return o, lse


def kv_accumulate(q: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor, cache: KVCache, table: torch.Tensor,
                  lens: torch.Tensor, cu: torch.Tensor | None = None, max_new: int | None = None,
                  softmax_scale: float | None = None, softcap: float = 0.0, window: int = 0,
                  slopes: torch.Tensor | None = None, decay: float = 1.0, stream=None) -> torch.Tensor:
    """fp4attn_kv_accumulate: adds to weights (fp32 [B, heads, W], W at least the longest length) the attention
    weight that the cached tokens get from the queries, whose lse is kv_attention's; what was there is multiplied
    by decay first.  In place; returns weights."""
    T = _rows(q)
    c, b, dev, heads, D, B, _ = _geometry(cache, table, lens, cu, T)
    at, r, s, group, max_new, scale, slope_at = _queries(q, dev, heads, D, B, T, cu, max_new, softmax_scale, softcap,
                                                         window, slopes)
    _check_out(lse, "lse", _f32, q.shape[:2], dev)
    W = weights.shape[-1] if isinstance(weights, _Tensor) and weights.dim() else 0
    _check_out(weights, "weights", _f32, (B, heads, W), dev)
    handle, _ = _stream_of(stream, dev)
    _launch(dev, "fp4attn_kv_accumulate", c, b, at, r, s, group, max_new, scale, softcap, window, slope_at,
            lse.data_ptr(), weights.data_ptr(), min(W, _MOST), decay, handle)
    return weights


def kv_evict(cache: KVCache, weights: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, new_table: torch.Tensor,
             keep: int, sinks: int = 0, recent: int = 0, kept: torch.Tensor | None = None,
             new_lens: torch.Tensor | None = None, new_weights: torch.Tensor | None = None, stream=None):
    """fp4attn_kv_evict: keeps, of every sequence and KV head, the first `sinks` tokens, the last `recent` and the
    heaviest others, `keep` in all, and copies them to the pages of new_table (pages that table does not list).
    (kept int32 [B, heads, keep], new_lens int32 [B], new_weights like weights): from here on these and new_table
    (with more pages behind, for what is to come) take the place of lens, weights and table.  The kept tokens have
    new slots, 0 .. new_lens - 1, and windows and slopes then count slots, not the tokens that were between; kept
    says which they were."""
    c, b, dev, heads, _, B, _ = _geometry(cache, table, lens, None, 0, rows=False)
    ns = _index_shape(new_table, "new_table", dev)
    if len(ns) != 2 or ns[0] != B:
        raise ValueError("new_table must be [%d, pages]" % B)
    W = weights.shape[-1] if isinstance(weights, _Tensor) and weights.dim() else 0
    _check_out(weights, "weights", _f32, (B, heads, W), dev)
    if not (0 < keep <= W and 0 <= sinks and 0 <= recent and sinks + recent <= keep):
        raise ValueError("keep = %s, sinks = %s, recent = %s do not fit weights of %d slots" % (keep, sinks, recent, W))
    if ns[1] * KV_PAGE < keep:
        raise ValueError("new_table lists %d pages, too few for %d tokens" % (ns[1], keep))
    if new_table.data_ptr() == table.data_ptr():
        raise ValueError("new_table must be another table than table, with pages of its own")
    shape = (B, heads, keep)
    if kept is not None:
        _check_out(kept, "kept", _i32, shape, dev)
    if new_lens is not None:
        _check_out(new_lens, "new_lens", _i32, (B,), dev)
    if new_weights is not None:
        _check_out(new_weights, "new_weights", _f32, weights.shape, dev)
    handle, side = _stream_of(stream, dev)
    if kept is None:
        kept = _new(shape, _i32, dev, side)
    if new_lens is None:
        new_lens = _new((B,), _i32, dev, side)
    if new_weights is None:
        new_weights = _new(weights.shape, _f32, dev, side)
    _launch(dev, "fp4attn_kv_evict", c, b, weights.data_ptr(), min(W, _MOST), new_table.data_ptr(), min(ns[1], _MOST),
            keep, sinks, recent, kept.data_ptr(), new_lens.data_ptr(), new_weights.data_ptr(), handle)
    return kept, new_lens, new_weights

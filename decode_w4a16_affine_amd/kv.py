"""Python binding of the paged 8-bit key/value cache (include/w4a16_kv.h).

Same conventions as the package's other functions: C-ABI names, tensors in,
dtype and shape checks before any pointer reaches the library, the current
stream of torch (of the tensors' GPU, which need not be the current one) unless
one is given, no fallback.

Tensor conventions (all on the same GPU; contiguous unless said otherwise):
  q, k, v, out            : torch.bfloat16; q, k, v may be parts of wider token
                            rows (only their last two dimensions are dense)
  k_cache, v_cache        : torch.int8 or torch.float8_e4m3fn, [pages, H, P, D] and [pages, H, D, P]
  k_scales, v_scales      : torch.bfloat16 [pages, H]
  lengths, tables, slots  : torch.int32
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _dtype, _shape
from . import lib as _base_lib

KV_INT8 = 0               # W4A16_KV_INT8
KV_FP8 = 1                # W4A16_KV_FP8
KV_DIMS = (64, 128, 256)
KV_PAGES = (16, 32, 64, 128, 256)
KV_MAX_REQUESTS = 1 << 20   # W4A16_KV_MAX_REQUESTS
KV_MAX_TOKENS = 1 << 20     # W4A16_KV_MAX_TOKENS
KV_MAX_HEADS = 1024         # W4A16_KV_MAX_HEADS
KV_MAX_GROUP = 64           # W4A16_KV_MAX_GROUP
KV_MAX_WIDTH = 1 << 22      # W4A16_KV_MAX_WIDTH
KV_MAX_DEQUANT = (1 << 24) - 1   # W4A16_KV_MAX_DEQUANT

KV_EXPORTS = ("w4a16_kv_plan", "w4a16_kv_append", "w4a16_kv_attention_workspace_bytes", "w4a16_kv_attention",
              "w4a16_kv_dequant")

_TYPES = {torch.int8: KV_INT8, torch.float8_e4m3fn: KV_FP8}
_vp = ctypes.c_void_p
_int = ctypes.c_int
_i64 = ctypes.c_int64


class KVCache(ctypes.Structure):
    """w4a16_kv_cache_t"""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp), ("type", _int), ("pages", _int),
                ("heads", _int), ("page", _int), ("dim", _int)]


_lib = None


def kv_lib() -> ctypes.CDLL:
    """libw4a16.so with the prototypes of the key/value cache."""
    global _lib
    if _lib is None:
        L = _base_lib()
        cache = ctypes.POINTER(KVCache)
        L.w4a16_kv_plan.restype = _int
        L.w4a16_kv_plan.argtypes = [_vp, _vp, _vp, _int, _vp, _int, _vp, _vp, _vp, _vp, _int, _int, _int, _vp]
        L.w4a16_kv_append.restype = _int
        L.w4a16_kv_append.argtypes = [_vp, _i64, _vp, _i64, _vp, cache, _int, _vp]
        L.w4a16_kv_attention_workspace_bytes.restype = ctypes.c_size_t
        L.w4a16_kv_attention_workspace_bytes.argtypes = [_int, _int, _int, _int, _int, _int, cache]
        L.w4a16_kv_attention.restype = _int
        L.w4a16_kv_attention.argtypes = [_vp, _i64, cache, _vp, _int, _vp, _vp, _vp, ctypes.c_float, _int, _int, _int,
                                         _int, _int, _int, _vp, ctypes.c_size_t, _vp]
        L.w4a16_kv_dequant.restype = _int
        L.w4a16_kv_dequant.argtypes = [cache, _vp, _int, _vp, _vp, _vp]
        _lib = L
    return _lib


# The checks below run on every call of a decode step, so each is one cheap
# test a tensor (get_device() is -1 for host tensors; pointers go to ctypes as
# plain numbers).

def _same_gpu(first, *ts) -> int:
    """The GPU that all tensors are on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    for t in ts:
        if t.get_device() != dev:
            raise ValueError("tensors must be on the GPU" if t.get_device() < 0 else
                             f"tensors must be on one device ({first.device} and {t.device})")
    return dev


def _dense(*ts) -> None:
    for t in ts:
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


# the current stream's handle without a Stream object around it (0.1 us a call instead of 1.1), where torch has it
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# A launch goes to the current GPU, and a null stream is that GPU's: a call whose tensors are on another one is made
# again with theirs current.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(dev: int, fn, *args):
    with torch.cuda.device(dev):
        return fn(*args)


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return _current_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _cache(k_cache, v_cache, k_scales, v_scales) -> KVCache:
    """The C struct of a cache's tensors, their types and shapes checked."""
    kind = _TYPES.get(k_cache.dtype)
    if kind is None:
        raise TypeError(f"k_cache must be torch.int8 or torch.float8_e4m3fn, got {k_cache.dtype}")
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be 4-D [pages, heads, page, D], got {list(k_cache.shape)}")
    _dtype(v_cache, k_cache.dtype, "v_cache")
    _dtype(k_scales, torch.bfloat16, "k_scales")
    _dtype(v_scales, torch.bfloat16, "v_scales")
    pages, heads, page, dim = k_cache.shape
    if v_cache.shape != (pages, heads, dim, page):
        _shape(v_cache, (pages, heads, dim, page), "v_cache")
    if k_scales.shape != (pages, heads):
        _shape(k_scales, (pages, heads), "k_scales")
    if v_scales.shape != (pages, heads):
        _shape(v_scales, (pages, heads), "v_scales")
    return KVCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), kind, pages,
                   heads, page, dim)


def _int32(names: str, *numbers) -> None:
    """Refuses numbers that the C ABI's 32-bit integers cannot hold (ctypes would pass their low bits)."""
    bits = 0
    for n in numbers:
        bits |= n
    if not -1 <= bits >> 31 <= 0:       # (beside a negative one, which the library refuses, others may pass)
        raise ValueError(f"{names} must fit 32 bits, got {numbers}")


def _vector(t, name, n=None):
    """The length of an int32 vector (checked against n where given)."""
    if t.dtype != torch.int32:
        _dtype(t, torch.int32, name)
    if n is not None:
        if t.shape != (n,):
            _shape(t, (n,), name)
    elif t.dim() != 1:
        raise ValueError(f"{name} must be 1-D, got {list(t.shape)}")
    return t.shape[0]


def _table(t, R):
    """The width of a block table [R, width]."""
    if t.dtype != torch.int32:
        _dtype(t, torch.int32, "block_table")
    if t.dim() != 2 or t.shape[0] != R:
        raise ValueError(f"block_table must have shape [{R}, width], got {list(t.shape)}")
    return t.shape[1]


def _rows(t, heads, dim, name):
    """Token count and token stride of a [T, heads, D] tensor whose token rows are dense."""
    if t.dtype != torch.bfloat16:
        _dtype(t, torch.bfloat16, name)
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must have shape [T, {'heads' if heads is None else heads}, {dim}], got {list(shape)}")
    tokens, row = shape[0], shape[1] * dim
    if t.numel() == 0:
        return tokens, row
    stride, head_stride, unit = t.stride()
    if tokens == 1:
        stride = row                    # no second row: any valid stride
    if unit != 1 or (head_stride != dim and shape[1] > 1) or stride < row:
        raise ValueError(f"{name} must be dense within a token (strides [>= {row}, {dim}, 1]), got {list(t.stride())}")
    return tokens, stride


# ---- C-ABI entry points ---------------------------------------------------------

def w4a16_kv_plan(ctx_lens, new_lens, free_pages, block_table, seq_lens, token_start, slot_map, pages_used, page: int,
                  stream=None) -> None:
    """Block tables and slot maps of a step from request lengths (block_table [R, width] is updated in place)."""
    R, num_free, width = _plan_inputs(ctx_lens, new_lens, free_pages, block_table)
    _int32("page", page)
    _vector(seq_lens, "seq_lens", R)
    _vector(token_start, "token_start", R + 1)
    tokens = _vector(slot_map, "slot_map")
    _vector(pages_used, "pages_used", 1)
    dev = _same_gpu(ctx_lens, new_lens, free_pages, block_table, seq_lens, token_start, slot_map, pages_used)
    _dense(ctx_lens, new_lens, free_pages, block_table, seq_lens, token_start, slot_map, pages_used)
    if _current_device() != dev:
        return _on(dev, w4a16_kv_plan, ctx_lens, new_lens, free_pages, block_table, seq_lens, token_start, slot_map,
                   pages_used, page, stream)
    _check(kv_lib().w4a16_kv_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), num_free,
                                  block_table.data_ptr(), width, seq_lens.data_ptr(), token_start.data_ptr(),
                                  slot_map.data_ptr(), pages_used.data_ptr(), R, tokens, page,
                                  _raw_stream(stream, dev)), "w4a16_kv_plan")


def _plan_inputs(ctx_lens, new_lens, free_pages, block_table):
    """Requests, free pages and table width of a plan's inputs, types and shapes checked."""
    R = _vector(ctx_lens, "ctx_lens")
    _vector(new_lens, "new_lens", R)
    num_free = _vector(free_pages, "free_pages")
    return R, num_free, _table(block_table, R)


def w4a16_kv_append(k, v, slot_map, k_cache, v_cache, k_scales, v_scales, stream=None) -> None:
    """Quantizes k, v [T, H, D] into the cache at slot_map [T] (slots outside the cache are skipped)."""
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    tokens, k_stride = _rows(k, c.heads, c.dim, "k")
    v_tokens, v_stride = _rows(v, c.heads, c.dim, "v")
    _vector(slot_map, "slot_map", tokens)
    if v_tokens != tokens:
        raise ValueError(f"k and v must have the same tokens, got {tokens} and {v_tokens}")
    dev = _same_gpu(k_cache, v_cache, k_scales, v_scales, slot_map, k, v)
    _dense(k_cache, v_cache, k_scales, v_scales, slot_map)
    if _current_device() != dev:
        return _on(dev, w4a16_kv_append, k, v, slot_map, k_cache, v_cache, k_scales, v_scales, stream)
    _check(kv_lib().w4a16_kv_append(k.data_ptr(), k_stride, v.data_ptr(), v_stride, slot_map.data_ptr(),
                                    ctypes.byref(c), tokens, _raw_stream(stream, dev)), "w4a16_kv_append")


def w4a16_kv_attention_workspace_bytes(tokens: int, requests: int, max_new: int, max_len: int, window: int,
                                       q_heads: int, k_cache, v_cache, k_scales, v_scales) -> int:
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    _int32("tokens, requests, max_new, max_len, window, q_heads", tokens, requests, max_new, max_len, window, q_heads)
    return int(kv_lib().w4a16_kv_attention_workspace_bytes(tokens, requests, max_new, max_len, window, q_heads,
                                                           ctypes.byref(c)))


def w4a16_kv_attention(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, out, workspace,
                       max_new: int, max_len: int = None, scale: float = None, window: int = 0, stream=None) -> None:
    """out [T, HQ, D] = causal attention of q [T, HQ, D] over the cache.

    token_start [R + 1] and seq_lens [R] as w4a16_kv_plan writes them; max_new
    and max_len bound the requests' new tokens and lengths (max_len None: what
    the block table's columns hold); scale None: 1 / sqrt(D); window 0: no
    window; workspace: a uint8 device tensor of at least
    w4a16_kv_attention_workspace_bytes bytes, or None where that is 0."""
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    inputs = _attention_inputs(c, q, block_table, seq_lens, token_start)
    if out.dtype != torch.bfloat16:
        _dtype(out, torch.bfloat16, "out")
    if out.shape != q.shape:
        _shape(out, q.shape, "out")
    if workspace is not None:
        _dtype(workspace, torch.uint8, "workspace")
        _same_gpu(out, workspace)
        _dense(workspace)
    dev = _same_gpu(k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, out, q)
    _dense(k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, out)
    if _current_device() != dev:
        return _on(dev, w4a16_kv_attention, q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start,
                   out, workspace, max_new, max_len, scale, window, stream)
    if max_len is None:
        max_len = inputs[3] * c.page
    _int32("max_new, max_len, window", max_new, max_len, window)
    _attention(ctypes.byref(c), inputs, q, block_table, seq_lens, token_start, out, workspace, max_new, max_len,
               1.0 / math.sqrt(c.dim) if scale is None else scale, window, _raw_stream(stream, dev))


def _attention_inputs(c, q, block_table, seq_lens, token_start):
    """Tokens, their stride, requests and table width of an attention's inputs, types and shapes checked."""
    tokens, q_stride = _rows(q, None, c.dim, "q")
    R = _vector(seq_lens, "seq_lens")
    _vector(token_start, "token_start", R + 1)
    return tokens, q_stride, R, _table(block_table, R)


def _attention(c, inputs, q, block_table, seq_lens, token_start, out, workspace, max_new, max_len, scale, window, stream):
    tokens, q_stride, R, width = inputs
    ws, ws_bytes = (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _check(kv_lib().w4a16_kv_attention(q.data_ptr(), q_stride, c, block_table.data_ptr(), width, seq_lens.data_ptr(),
                                       token_start.data_ptr(), out.data_ptr(), scale, window, tokens, R, max_new,
                                       max_len, q.shape[1], ws, ws_bytes, stream), "w4a16_kv_attention")


def w4a16_kv_dequant(k_cache, v_cache, k_scales, v_scales, pages, k_out, v_out, stream=None) -> None:
    """k_out, v_out [n, H, P, D] (fp32) = the values of pages [n]."""
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    n = _vector(pages, "pages")
    _dtype(k_out, torch.float32, "k_out")
    _dtype(v_out, torch.float32, "v_out")
    _shape(k_out, (n, c.heads, c.page, c.dim), "k_out")
    _shape(v_out, (n, c.heads, c.page, c.dim), "v_out")
    _same_gpu(k_cache, k_out, v_out)
    _dense(k_out, v_out)
    _dequant(c, (k_cache, v_cache, k_scales, v_scales, pages), n, k_out, v_out, stream)


def _dequant(c, inputs, n, k_out, v_out, stream):
    dev = _same_gpu(*inputs)
    _dense(*inputs)
    if _current_device() != dev:
        return _on(dev, _dequant, c, inputs, n, k_out, v_out, stream)
    _check(kv_lib().w4a16_kv_dequant(ctypes.byref(c), inputs[4].data_ptr(), n, k_out.data_ptr(), v_out.data_ptr(),
                                     _raw_stream(stream, dev)), "w4a16_kv_dequant")


# ---- allocating conveniences (torch allocates; the library computes) ------------
# On a stream of the caller's they run as its current stream, so that what they
# allocate is not given to others before the call has run.

def _current(stream, t):
    """A context with `stream` (a torch stream or a handle) current on t's GPU."""
    dev = _same_gpu(t)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), dev) if int(stream) else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def kv_cache(pages: int, heads: int, dim: int, page: int = 64, dtype=torch.int8, device="cuda"):
    """An empty cache: (k_cache, v_cache, k_scales, v_scales)."""
    return (torch.zeros((pages, heads, page, dim), dtype=dtype, device=device),
            torch.zeros((pages, heads, dim, page), dtype=dtype, device=device),
            torch.zeros((pages, heads), dtype=torch.bfloat16, device=device),
            torch.zeros((pages, heads), dtype=torch.bfloat16, device=device))


def kv_plan(ctx_lens, new_lens, free_pages, block_table, tokens: int, page: int, stream=None):
    """(seq_lens, token_start, slot_map [tokens], pages_used); block_table is updated in place."""
    if stream is not None:
        with _current(stream, ctx_lens):
            return kv_plan(ctx_lens, new_lens, free_pages, block_table, tokens, page)
    R, num_free, width = _plan_inputs(ctx_lens, new_lens, free_pages, block_table)
    _int32("tokens, page", tokens, page)
    dev = _same_gpu(ctx_lens, new_lens, free_pages, block_table)
    _dense(ctx_lens, new_lens, free_pages, block_table)
    if _current_device() != dev:
        return _on(dev, kv_plan, ctx_lens, new_lens, free_pages, block_table, tokens, page)
    out = ctx_lens.new_empty(2 * R + tokens + 2)      # (one allocation: its parts need no checks of their own)
    at = out.data_ptr()
    _check(kv_lib().w4a16_kv_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), num_free,
                                  block_table.data_ptr(), width, at, at + 4 * R, at + 4 * (2 * R + 1),
                                  at + 4 * (2 * R + 1 + tokens), R, tokens, page, _current_stream(dev)),
           "w4a16_kv_plan")
    return out.split((R, R + 1, tokens, 1))


def kv_attention(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, max_new: int,
                 max_len: int = None, scale: float = None, window: int = 0, stream=None):
    """Attention of the step's queries: a new out [T, HQ, D] (see w4a16_kv_attention)."""
    if stream is not None:
        with _current(stream, q):
            return kv_attention(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, max_new,
                                max_len, scale, window)
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    inputs = tokens, _, R, width = _attention_inputs(c, q, block_table, seq_lens, token_start)
    dev = _same_gpu(k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, q)
    _dense(k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start)
    if _current_device() != dev:
        return _on(dev, kv_attention, q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, max_new,
                   max_len, scale, window)
    if max_len is None:
        max_len = width * c.page
    _int32("max_new, max_len, window", max_new, max_len, window)
    ref = ctypes.byref(c)
    need = kv_lib().w4a16_kv_attention_workspace_bytes(tokens, R, max_new, max_len, window, q.shape[1], ref)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    ws = q.new_empty(need, dtype=torch.uint8) if need else None
    _attention(ref, inputs, q, block_table, seq_lens, token_start, out, ws, max_new, max_len,
               1.0 / math.sqrt(c.dim) if scale is None else scale, window, _current_stream(dev))
    return out


def kv_dequant(k_cache, v_cache, k_scales, v_scales, pages, stream=None):
    """(k_out, v_out) fp32 [n, H, P, D]: the values of pages [n]."""
    if stream is not None:
        with _current(stream, k_scales):
            return kv_dequant(k_cache, v_cache, k_scales, v_scales, pages)
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    n = _vector(pages, "pages")
    k_out = k_scales.new_empty((n, c.heads, c.page, c.dim), dtype=torch.float32)
    v_out = torch.empty_like(k_out)
    _dequant(c, (k_cache, v_cache, k_scales, v_scales, pages), n, k_out, v_out, None)
    return k_out, v_out

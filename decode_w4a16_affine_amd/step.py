"""Python binding of what a serving step runs beside the products and the cache (include/w4a16_step.h).

Same conventions as kv.py: C-ABI names, tensors in, dtype and shape checks before any pointer reaches the library, the
current stream of torch (of the tensors' GPU, which need not be the current one) unless one is given, no fallback.

Tensor conventions (all on the same GPU; contiguous unless said otherwise):
  q, k, outputs           : torch.bfloat16 [T, heads, D]; q, k may be parts of wider token rows (only their last two
                            dimensions are dense), and so may q_out, k_out
  norm weights            : torch.bfloat16 [D]
  inv_freq                : torch.float32 [rot / 2]
  positions               : torch.int32 [T], or [axes, T] with sections
  logits                  : torch.float32 or torch.bfloat16 [M, N], rows may be parts of wider ones
  uniforms, temperature, top_p, min_p, share : torch.float32 [M];  top_k, tokens : torch.int32 [M]
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import OUT_BF16, OUT_F32, _check, _dtype, _shape
from . import lib as _base_lib
from .kv import (KVCache, _attention_inputs, _cache, _current, _current_device, _dense, _int32, _on, _raw_stream, _rows,
                 _same_gpu, _vector)

ROPE_NORM = 1             # W4A16_ROPE_NORM
ROPE_INTERLEAVED = 2      # W4A16_ROPE_INTERLEAVED
ROPE_MAX_AXES = 4         # W4A16_ROPE_MAX_AXES

SAMPLE_MAX_ROWS = 65536   # W4A16_SAMPLE_MAX_ROWS
SAMPLE_MAX_N = 1 << 20    # W4A16_SAMPLE_MAX_N

STEP_EXPORTS = ("w4a16_qk_norm_rope", "w4a16_kv_attention_shared_workspace_bytes", "w4a16_kv_attention_shared",
                "w4a16_sample_workspace_bytes", "w4a16_sample")

_vp = ctypes.c_void_p
_int = ctypes.c_int
_i64 = ctypes.c_int64
_float = ctypes.c_float

_lib = None


def step_lib() -> ctypes.CDLL:
    """libw4a16.so with the prototypes of a serving step's operators."""
    global _lib
    if _lib is None:
        L = _base_lib()
        L.w4a16_qk_norm_rope.restype = _int
        L.w4a16_qk_norm_rope.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _float, _vp, _vp, ctypes.POINTER(_int), _int, _vp,
                                         _i64, _vp, _i64, _float, _int, _int, _int, _int, _int, _int, _vp]
        cache = ctypes.POINTER(KVCache)
        L.w4a16_kv_attention_shared_workspace_bytes.restype = ctypes.c_size_t
        L.w4a16_kv_attention_shared_workspace_bytes.argtypes = [_int] * 6 + [cache]
        L.w4a16_kv_attention_shared.restype = _int
        L.w4a16_kv_attention_shared.argtypes = [_vp, _i64, cache, _vp, _int, _vp, _vp, _vp, _vp, _float, _int, _int, _int,
                                                _int, _int, _int, _vp, ctypes.c_size_t, _vp]
        L.w4a16_sample_workspace_bytes.restype = ctypes.c_size_t
        L.w4a16_sample_workspace_bytes.argtypes = [_int, _int]
        L.w4a16_sample.restype = _int
        L.w4a16_sample.argtypes = [_vp, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _int, _int, _vp]
        _lib = L
    return _lib


# ---- norms of queries and keys, rotation ------------------------------------------

def _head(t, name):
    """Tokens, heads, D and token stride of a [T, heads, D] tensor whose token rows are dense."""
    if t.dtype is not torch.bfloat16:
        _dtype(t, torch.bfloat16, name)
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D [T, heads, D], got {list(shape)}")
    tokens, heads, dim = shape
    return tokens, heads, dim, heads * dim if t.is_contiguous() else _rows(t, heads, dim, name)[1]


_NO_HEAD = (0, 0, 0, 0)


def _head_rows(q, k):
    """(q's and k's tokens, heads, D and stride); q or k may be None."""
    a = _NO_HEAD if q is None else _head(q, "q")
    b = _NO_HEAD if k is None else _head(k, "k")
    if k is None:
        if q is None:
            raise ValueError("q and k are both None")
    elif q is not None and (a[0] != b[0] or a[2] != b[2]):
        raise ValueError(f"q and k must have the same tokens and D, got {list(q.shape)} and {list(k.shape)}")
    return a, b


def _rotation(inv_freq, positions, sections, tokens):
    """(rot, axes, sections as a C array or None)."""
    if inv_freq is None:
        if positions is not None or sections is not None:
            raise ValueError("positions and sections need inv_freq")
        return 0, 1, None
    if positions is None:
        raise ValueError("inv_freq needs positions")
    _dtype(inv_freq, torch.float32, "inv_freq")
    shape = inv_freq.shape
    if len(shape) != 1:
        raise ValueError(f"inv_freq must be 1-D [rot / 2], got {list(shape)}")
    _dtype(positions, torch.int32, "positions")
    half = shape[0]
    if sections is None:
        if positions.shape != (tokens,):
            _shape(positions, (tokens,), "positions")
        return 2 * half, 1, None
    axes = len(sections)
    if not 1 <= axes <= ROPE_MAX_AXES:
        raise ValueError(f"1 to {ROPE_MAX_AXES} sections, got {axes}")
    if min(sections) < 0 or sum(sections) != half:
        raise ValueError(f"sections must be pair counts that sum to {half}, got {list(sections)}")
    _shape(positions, (axes, tokens), "positions")
    return 2 * half, axes, (_int * axes)(*sections)


def _weight(w, dim, name):
    _dtype(w, torch.bfloat16, name)
    if w.shape != (dim,):
        _shape(w, (dim,), name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _given(*ts):
    return [t for t in ts if t is not None]


def w4a16_qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions, q_out, k_out, eps: float = 1e-6,
                       weight_offset: float = 0.0, norm: bool = True, interleaved: bool = False, sections=None,
                       stream=None) -> None:
    """q_out, k_out = q, k [T, heads, D], each head normed (norm) and its first 2 * len(inv_freq) elements rotated.

    A weight None is a factor of 1; q (with q_out) or k (with k_out) None is left out; inv_freq None rotates nothing;
    sections gives the pairs of each axis of positions [axes, T].  q_out may be q and k_out may be k."""
    rows = _head_rows(q, k)
    strides = []
    for x, out, name in ((q, q_out, "q_out"), (k, k_out, "k_out")):
        if (x is None) != (out is None):
            raise ValueError(f"{name} goes with its input")
        if out is not None and out.shape != x.shape:
            _shape(out, x.shape, name)
        strides.append(0 if out is None else _head(out, name)[3])
    _same_gpu(*_given(q, k, q_out, k_out))
    _rope(rows, q, k, q_weight, k_weight, inv_freq, positions, q_out, strides[0], k_out, strides[1], eps, weight_offset,
          norm, interleaved, sections, stream)


def _rope(rows, q, k, q_weight, k_weight, inv_freq, positions, q_out, qo_stride, k_out, ko_stride, eps, weight_offset,
          norm, interleaved, sections, stream):
    (tokens, q_heads, dim, q_stride), (k_tokens, k_heads, k_dim, k_stride) = rows
    if q is None:
        tokens, dim = k_tokens, k_dim
    if q_weight is not None:
        _weight(q_weight, dim, "q_weight")
    if k_weight is not None:
        _weight(k_weight, dim, "k_weight")
    rot, axes, sec = _rotation(inv_freq, positions, sections, tokens)
    small = _given(q_weight, k_weight, inv_freq, positions)
    dev = _same_gpu(k if q is None else q, *(small if q is None or k is None else (k, *small)))
    _dense(*small)
    if _current_device() != dev:
        return _on(dev, _rope, rows, q, k, q_weight, k_weight, inv_freq, positions, q_out, qo_stride, k_out, ko_stride,
                   eps, weight_offset, norm, interleaved, sections, stream)
    if q_out is None and k_out is None:      # the allocating form
        q_out, k_out = (None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k))
        qo_stride, ko_stride = q_heads * dim, k_heads * dim
    _check(step_lib().w4a16_qk_norm_rope(_ptr(q), q_stride, _ptr(k), k_stride, _ptr(q_weight), _ptr(k_weight),
                                         weight_offset, _ptr(inv_freq), _ptr(positions), sec, axes, _ptr(q_out),
                                         qo_stride, _ptr(k_out), ko_stride, eps,
                                         (ROPE_NORM if norm else 0) | (ROPE_INTERLEAVED if interleaved else 0), tokens,
                                         q_heads, k_heads, dim, rot, _raw_stream(stream, dev)), "w4a16_qk_norm_rope")
    return q_out, k_out


# ---- attention behind shared entries ------------------------------------------------

def w4a16_kv_attention_shared_workspace_bytes(tokens: int, requests: int, max_new: int, max_shared: int, max_own: int,
                                              q_heads: int, k_cache, v_cache, k_scales, v_scales) -> int:
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    _int32("tokens, requests, max_new, max_shared, max_own, q_heads", tokens, requests, max_new, max_shared, max_own,
           q_heads)
    return int(step_lib().w4a16_kv_attention_shared_workspace_bytes(tokens, requests, max_new, max_shared, max_own,
                                                                    q_heads, ctypes.byref(c)))


def w4a16_kv_attention_shared(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, shared_len, out,
                              workspace, max_new: int, max_shared: int, max_own: int, scale: float = None,
                              stream=None) -> None:
    """out [T, HQ, D] = causal attention of q [T, HQ, D] for requests that begin with the same shared_len [1] entries.

    Those lie in the pages of block_table's row 0, a request's others in those of its own row; max_new, max_shared
    and max_own bound the requests' new tokens, shared_len and the entries behind it; the rest as
    w4a16_kv_attention has it.  workspace: a uint8 device tensor of at least
    w4a16_kv_attention_shared_workspace_bytes bytes, or None where that is 0."""
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
    _same_gpu(q, out)
    _dense(out)
    _shared(c, inputs, q, (k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, shared_len), out,
            workspace, max_new, max_shared, max_own, scale, stream)


def _shared(c, inputs, q, ts, out, workspace, max_new, max_shared, max_own, scale, stream):
    _vector(ts[7], "shared_len", 1)
    _int32("max_new, max_shared, max_own", max_new, max_shared, max_own)
    dev = _same_gpu(*ts, q)
    _dense(*ts)
    if _current_device() != dev:
        return _on(dev, _shared, c, inputs, q, ts, out, workspace, max_new, max_shared, max_own, scale, stream)
    tokens, q_stride, R, width = inputs
    ref = ctypes.byref(c)
    if out is None:      # the allocating form
        need = step_lib().w4a16_kv_attention_shared_workspace_bytes(tokens, R, max_new, max_shared, max_own, q.shape[1], ref)
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        workspace = q.new_empty(need, dtype=torch.uint8) if need else None
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _check(step_lib().w4a16_kv_attention_shared(q.data_ptr(), q_stride, ref, ts[4].data_ptr(), width, ts[5].data_ptr(),
                                                ts[6].data_ptr(), ts[7].data_ptr(), out.data_ptr(),
                                                1.0 / math.sqrt(c.dim) if scale is None else scale, tokens, R, max_new,
                                                max_shared, max_own, q.shape[1], ws, ws_bytes, _raw_stream(stream, dev)),
           "w4a16_kv_attention_shared")
    return out


# ---- sampling -----------------------------------------------------------------------

def w4a16_sample_workspace_bytes(M: int, N: int) -> int:
    _int32("M, N", M, N)
    return int(step_lib().w4a16_sample_workspace_bytes(M, N))


def w4a16_sample(logits, uniforms, temperature, top_k, top_p, min_p, tokens, share, workspace, stream=None) -> None:
    """tokens [M], share [M] or None: a token drawn from each row of logits [M, N] (see include/w4a16_step.h).

    uniforms None draws the largest logits; temperature, top_k, top_p and min_p None are 1, 0 (off), 1 (off) and 0
    (off); workspace: a uint8 device tensor of at least w4a16_sample_workspace_bytes bytes, or None where that is 0."""
    rows = _logits(logits)
    for t, name in ((tokens, "tokens"), (share, "share")):
        if t is not None:
            _row_values(t, rows[0], name)
    if tokens is None:
        raise ValueError("tokens is None")
    if workspace is not None:
        _dtype(workspace, torch.uint8, "workspace")
    given = _given(tokens, share, workspace)
    _same_gpu(logits, *given)
    _dense(*given)
    _sample(rows, logits, uniforms, temperature, top_k, top_p, min_p, tokens, share, workspace, stream)


def _logits(logits):
    """(M, N, row stride, dtype code)"""
    if logits.dtype == torch.float32:
        code = OUT_F32
    elif logits.dtype == torch.bfloat16:
        code = OUT_BF16
    else:
        raise TypeError(f"logits must be torch.float32 or torch.bfloat16, got {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError(f"logits must be 2-D [M, N], got {list(logits.shape)}")
    M, N = logits.shape
    _int32("M, N", M, N)
    stride, unit = logits.stride()
    if M <= 1:
        stride = N                      # no second row: any valid stride
    if N > 1 and unit != 1 or stride < N:
        raise ValueError(f"rows of logits must be dense and apart, got strides {list(logits.stride())}")
    return M, N, stride, code


def _row_values(t, M, name):
    want = torch.int32 if name in ("top_k", "tokens") else torch.float32
    if t.dtype != want:
        _dtype(t, want, name)
    if t.shape != (M,):
        _shape(t, (M,), name)


def _sample(rows, logits, uniforms, temperature, top_k, top_p, min_p, tokens, share, workspace, stream):
    M, N, stride, code = rows
    given = []
    for t, name in ((uniforms, "uniforms"), (temperature, "temperature"), (top_k, "top_k"), (top_p, "top_p"),
                    (min_p, "min_p")):
        if t is not None:
            _row_values(t, M, name)
            given.append(t)
    dev = _same_gpu(logits, *given)
    _dense(*given)
    if _current_device() != dev:
        return _on(dev, _sample, rows, logits, uniforms, temperature, top_k, top_p, min_p, tokens, share, workspace, stream)
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    _check(step_lib().w4a16_sample(logits.data_ptr(), code, stride, _ptr(uniforms), _ptr(temperature), _ptr(top_k),
                                   _ptr(top_p), _ptr(min_p), tokens.data_ptr(), _ptr(share), ws, ws_bytes, M, N,
                                   _raw_stream(stream, dev)), "w4a16_sample")


# ---- allocating conveniences (torch allocates; the library computes) ------------

def qk_norm_rope(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, eps: float = 1e-6,
                 weight_offset: float = 0.0, norm: bool = True, interleaved: bool = False, sections=None, stream=None):
    """(q_out, k_out), dense and new (see w4a16_qk_norm_rope)."""
    if stream is not None and not (q is None and k is None):
        with _current(stream, k if q is None else q):
            return qk_norm_rope(q, k, q_weight, k_weight, inv_freq, positions, eps, weight_offset, norm, interleaved,
                                sections)
    return _rope(_head_rows(q, k), q, k, q_weight, k_weight, inv_freq, positions, None, 0, None, 0, eps, weight_offset, norm,
                 interleaved, sections, None)


def kv_attention_shared(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, shared_len,
                        max_new: int, max_shared: int, max_own: int, scale: float = None, stream=None):
    """Attention of a step behind shared entries: a new out [T, HQ, D] (see w4a16_kv_attention_shared)."""
    if stream is not None:
        with _current(stream, q):
            return kv_attention_shared(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start,
                                       shared_len, max_new, max_shared, max_own, scale)
    c = _cache(k_cache, v_cache, k_scales, v_scales)
    inputs = _attention_inputs(c, q, block_table, seq_lens, token_start)
    return _shared(c, inputs, q, (k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, token_start, shared_len),
                   None, None, max_new, max_shared, max_own, scale, None)


def sample(logits, uniforms=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """(tokens int32 [M], share fp32 [M]): a token drawn from each row of logits (see w4a16_sample)."""
    if stream is not None:
        with _current(stream, logits):
            return sample(logits, uniforms, temperature, top_k, top_p, min_p)
    rows = _logits(logits)
    M, N = rows[:2]
    need = step_lib().w4a16_sample_workspace_bytes(M, N)
    tokens = logits.new_empty((M,), dtype=torch.int32)
    share = logits.new_empty((M,), dtype=torch.float32)
    ws = logits.new_empty((need,), dtype=torch.uint8) if need else None
    _sample(rows, logits, uniforms, temperature, top_k, top_p, min_p, tokens, share, ws, None)
    return tokens, share

"""ctypes binding of libspecforward.so (argument marshalling only).

The operators that a verify forward needs on either side of its model: the paged
KV cache's write (``spec_kv_append``) and attention (``spec_attention``), and the
penalties, biases and grammar masks on its logits (``spec_adjust``). As in
``binding.py`` every step of the computation runs in the HIP library; this module
checks dtypes, shapes, devices and layouts (ValueError on a mismatch), allocates
outputs, keeps one workspace per (device, stream), and passes raw device pointers
plus the current stream to the C ABI declared in ``include/spec_forward.h``.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

from .binding import BF16, F32, SpecVerifyError, _user_workspace

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecforward.so")

F16 = 2
E4M3 = 3

_QKV = {torch.bfloat16: BF16, torch.float16: F16}
_CACHE = {torch.bfloat16: BF16, torch.float16: F16, torch.float8_e4m3fn: E4M3}
_LOGITS = {torch.float32: F32, torch.bfloat16: BF16}

_lib = None
_lock = threading.Lock()


def forward_lib():
    """The loaded HIP library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise SpecVerifyError(
                        -8, f"{LIB_PATH} is missing: build it with `python -m token_verification_amd.build`")
                L = ctypes.CDLL(LIB_PATH)
                P, I, F, S, N = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
                C = ctypes.c_int
                L.spec_kv_append.argtypes = [P, P, P, P, C, I, I, I, I, P, P, P, P, C, N, I, P, I, P, P, P, P, P]
                L.spec_kv_append.restype = C
                L.spec_attention.argtypes = [P, P, C, I, I, I, I, I, P, P, P, P, C, N, I, P, I, P, P, F, F, I, P, P,
                                             P, P, P, S, P]
                L.spec_attention.restype = C
                L.spec_attention_workspace_size.argtypes = [I, I, I, I, I, C, I, I]
                L.spec_attention_workspace_size.restype = S
                L.spec_adjust.argtypes = [P, I, I, I, C, P, I, P, P, I, P, P, P, P, P, P, P, I, P, I, P, P, C, P]
                L.spec_adjust.restype = C
                L.spec_forward_last_error.restype = ctypes.c_char_p
                _lib = L
    return _lib


def _raise(rc: int):
    raise SpecVerifyError(rc, forward_lib().spec_forward_last_error().decode())


# The small calls' time is the host's, so these go straight to what torch.cuda's functions of
# similar names call.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing


def _call(fn, dev: torch.device, *args) -> None:
    """fn(*args, stream) on dev's current stream, with dev the current device."""
    index = dev.index
    if index == _current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        _raise(rc)


_pack_stride = struct.Struct("3q").pack


def _stride(t: torch.Tensor) -> bytes:
    s = t.stride()
    return _pack_stride(s[0], s[1], s[2])


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check_sizes(bits: int) -> None:
    """bits: the sizes that the library takes as int32, or-ed (ctypes would cut them)."""
    if bits >> 31:
        raise ValueError("a size is beyond 2^31 - 1")


def _check(t, name: str, shape, dtype, dev: torch.device) -> None:
    """A dense tensor of this shape and dtype on dev."""
    try:
        fine = t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous()
    except AttributeError:
        fine = False
    if not fine:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {dev}")


def _check_strided(t, name: str, es: int, dev: torch.device) -> None:
    """A [.., .., .., D] tensor whose rows the library can load in 16-byte pieces."""
    s = t.stride()
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if s[3] != 1 or t.data_ptr() % 16 or (s[0] | s[1] | s[2]) * es % 16:
        raise ValueError(f"{name} must be contiguous in its last dimension, with a 16-byte aligned start and "
                         f"strides that are multiples of 16 bytes (got strides {list(s)} of {es}-byte elements)")


def _span(t: torch.Tensor) -> tuple:
    """The bytes from t's first element to behind its last."""
    at = t.data_ptr()
    return at, at + (sum(s * (n - 1) for s, n in zip(t.stride(), t.shape)) + 1) * t.element_size()


def _check_apart(out: torch.Tensor, name: str, **inputs) -> None:
    a, b = _span(out)
    for other, t in inputs.items():
        c, d = _span(t)
        if a < d and c < b:
            raise ValueError(f"{name} overlaps {other}")


def _overlaps_itself(t: torch.Tensor) -> bool:
    """Whether two indices of t may share a place (an expanded cache, say)."""
    if t.is_contiguous():
        return False
    extent = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size > 1:
            if stride < extent:
                return True
            extent = stride * (size - 1) + extent
    return False


def _check_cache(k_cache, v_cache, page_table, kv_len, draft_len, k_scale, v_scale, B: int, D: int, dtype,
                 dev: torch.device):
    """(Hkv, pages, page_size, max_pages, cache dtype code) of a paged cache."""
    try:
        shape, kind, es = k_cache.shape, k_cache.dtype, k_cache.element_size()
        fine = len(shape) == 4 and shape[3] == D and v_cache.shape == shape and v_cache.dtype is kind
    except AttributeError:
        fine = False
    if not fine:
        raise ValueError(f"k_cache and v_cache must be [pages, Hkv, page_size, D] tensors of one shape and dtype, "
                         f"with D = {D}")
    e4m3 = kind is torch.float8_e4m3fn
    if not e4m3 and kind is not dtype:
        raise ValueError(f"k_cache and v_cache must be {dtype} or float8_e4m3fn (got {kind})")
    _check_strided(k_cache, "k_cache", es, dev)
    _check_strided(v_cache, "v_cache", es, dev)
    pages, Hkv, page_size, _ = shape
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 [B, max_pages] tensor")
    max_pages = page_table.shape[1]
    _check_sizes(B | max_pages)
    _check(page_table, "page_table", (B, max_pages), torch.int32, dev)
    _check(kv_len, "kv_len", (B,), torch.int32, dev)
    if draft_len is not None:
        _check(draft_len, "draft_len", (B,), torch.int32, dev)
    if e4m3:
        _check(k_scale, "k_scale (of a float8_e4m3fn cache)", (Hkv,), torch.float32, dev)
        _check(v_scale, "v_scale (of a float8_e4m3fn cache)", (Hkv,), torch.float32, dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale go with a float8_e4m3fn cache only")
    return Hkv, pages, page_size, max_pages, _CACHE[kind]


def spec_kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   page_table: torch.Tensor, kv_len: torch.Tensor, *, draft_len: Optional[torch.Tensor] = None,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> None:
    """Write the keys and values of a step's new tokens into a paged cache, in place
    (see include/spec_forward.h).

    k, v [B, R, Hkv, D] bfloat16 or float16, any strides with whole 16-byte rows
    (e.g. slices of a fused projection's output); k_cache, v_cache [pages, Hkv,
    page_size, D] of the same dtype or float8_e4m3fn (then with k_scale, v_scale
    float32 [Hkv]), again of any such strides: a cache stored as [pages,
    page_size, Hkv, D] is passed as its transpose(1, 2). Token i of batch row b
    goes to position kv_len[b] + i (int32 [B]) of the sequence, which
    page_table (int32 [B, max_pages]) maps to a page. With draft_len (int32
    [B]) only tokens 0..draft_len[b] are written.
    """
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or not k.is_cuda or k.dtype not in _QKV:
        raise ValueError("k must be a bfloat16 or float16 [B, R, Hkv, D] device tensor")
    shape, dtype, dev = k.shape, k.dtype, k.device
    if not isinstance(v, torch.Tensor) or v.shape != shape or v.dtype is not dtype:
        raise ValueError("v must match k's shape and dtype")
    B, R, H, D = shape
    _check_strided(k, "k", 2, dev)
    _check_strided(v, "v", 2, dev)
    Hkv, pages, page_size, max_pages, code = _check_cache(k_cache, v_cache, page_table, kv_len, draft_len, k_scale,
                                                          v_scale, B, D, dtype, dev)
    if H != Hkv:
        raise ValueError(f"k holds {H} heads, the cache {Hkv}")
    _check_sizes(R)
    if _overlaps_itself(k_cache) or _overlaps_itself(v_cache):
        raise ValueError("k_cache and v_cache must hold every element at a place of its own")
    _call(forward_lib().spec_kv_append, dev, k.data_ptr(), _stride(k), v.data_ptr(), _stride(v), _QKV[dtype],
          B, R, H, D, k_cache.data_ptr(), _stride(k_cache), v_cache.data_ptr(), _stride(v_cache), code, pages,
          page_size, page_table.data_ptr(), max_pages, kv_len.data_ptr(), _ptr(draft_len), _ptr(k_scale),
          _ptr(v_scale))


_ws_cache: dict = {}
_need_cache: dict = {}


def _workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    """One workspace per (device, stream). A call that is captured into a graph gets
    one of its own, from the graph's memory: graphs captured on one stream may be
    replayed on different ones at the same time."""
    if _capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    key = (dev.index, _raw_stream(dev.index))
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _ws_cache[key] = ws
    return ws


def spec_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                   kv_len: torch.Tensor, *, draft_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                   softcap: float = 0.0, window: int = 0, slopes: Optional[torch.Tensor] = None,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of a step's new tokens over a paged cache that already holds their keys
    and values (spec_kv_append; see include/spec_forward.h).

    q [B, R, Hq, D] bfloat16 or float16 (strides as spec_kv_append's k), R = 1 for
    single tokens or k + 1 for a verify step; query head h reads cache head
    h // (Hq // Hkv). Token i of batch row b sees positions up to kv_len[b] + i,
    with window > 0 the last `window` of them. scale (default 1 / sqrt(D))
    multiplies q . k, softcap > 0 caps the scores by softcap * tanh(s / softcap),
    and slopes (float32 [Hq]) adds slopes[h] * (t - position) to them. The cache,
    page_table, draft_len and scales are spec_kv_append's. Returns [B, R, Hq, D]
    of q's dtype (zeros for tokens behind draft_len's, NaN for batch rows with a
    length or page out of range).
    """
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or not q.is_cuda or q.dtype not in _QKV:
        raise ValueError("q must be a bfloat16 or float16 [B, R, Hq, D] device tensor")
    shape, dtype, dev = q.shape, q.dtype, q.device
    B, R, Hq, D = shape
    _check_strided(q, "q", 2, dev)
    Hkv, pages, page_size, max_pages, code = _check_cache(k_cache, v_cache, page_table, kv_len, draft_len, k_scale,
                                                          v_scale, B, D, dtype, dev)
    if not 0 <= window <= 0x7fffffff:
        raise ValueError(f"window must be in [0, 2^31 - 1] (got {window})")
    if slopes is not None:
        _check(slopes, "slopes", (Hq,), torch.float32, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _check(out, "out", shape, dtype, dev)
        if out.data_ptr() % 16:
            raise ValueError("out must be 16-byte aligned")
        _check_apart(out, "out", q=q, k_cache=k_cache, v_cache=v_cache)
    key = (B, R, Hq, Hkv, D, code, page_size, max_pages)
    need = _need_cache.get(key)
    if need is None:
        need = int(forward_lib().spec_attention_workspace_size(*key))
        if need == 0:
            raise SpecVerifyError(-2, f"unsupported sizes B={B} R={R} Hq={Hq} Hkv={Hkv} D={D} "
                                      f"page_size={page_size} max_pages={max_pages}")
        _need_cache[key] = need
    ws = _workspace(dev, need) if workspace is None else _user_workspace(workspace, dev, need)
    _call(forward_lib().spec_attention, dev, q.data_ptr(), _stride(q), _QKV[dtype], B, R, Hq, Hkv, D,
          k_cache.data_ptr(), _stride(k_cache), v_cache.data_ptr(), _stride(v_cache), code, pages, page_size,
          page_table.data_ptr(), max_pages, kv_len.data_ptr(), _ptr(draft_len),
          1.0 / math.sqrt(D) if scale is None else float(scale), float(softcap), int(window), _ptr(slopes),
          _ptr(k_scale), _ptr(v_scale), out.data_ptr(), ws.data_ptr(), ws.nbytes)
    return out


def spec_adjust(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *,
                history: Optional[torch.Tensor] = None, hist_len: Optional[torch.Tensor] = None,
                prompt_len: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                frequency: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                bias_tokens: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                admit: Optional[torch.Tensor] = None, admit_row: Optional[torch.Tensor] = None,
                draft_len: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and grammar masks on the logits of a verify
    step, for spec_verify (see include/spec_forward.h).

    logits [B, R, V] float32 or bfloat16: target rows (R = k + 1) or draft rows
    (R = k) of the drafts tokens (int32 [B, k]; may be None when R is 1), row i
    following the history and drafts 0..i-1. history int32 [B, H] with hist_len
    (int32 [B]) committed tokens, the first prompt_len (int32 [B], default 0) of
    them the prompt; repetition (over history and drafts), frequency and presence
    (over what was generated) float32 [B]. bias_tokens int32 / bias_values float32
    [B, n]: entries outside [0, V) are padding. admit: 32-bit masks [n, (V + 31) //
    32] as spec_gate's, admit_row int32 [B, R] the mask of each row (-1: none;
    default: row b * R + i). With draft_len (int32 [B]) the rows behind those in
    use are left as they are. Returns out (default: a new tensor; logits itself
    adjusts in place) of out_dtype (default: the logits' dtype; float32 also for
    bfloat16 logits).
    """
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3 or not logits.is_cuda or logits.dtype not in _LOGITS:
        raise ValueError("logits must be a float32 or bfloat16 [B, R, V] device tensor")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    shape, kind, dev = logits.shape, logits.dtype, logits.device
    B, R, V = shape
    k = 0
    if tokens is not None:
        if not isinstance(tokens, torch.Tensor) or tokens.dim() != 2:
            raise ValueError("tokens must be an int32 [B, k] tensor")
        k = tokens.shape[1]
        _check(tokens, "tokens", (B, k), torch.int32, dev)
        if R != k + 1 and R != k:
            raise ValueError(f"logits hold {R} rows per batch row, {k} drafts need {k} or {k + 1}")
    elif R != 1:
        raise ValueError("tokens is required when logits hold more than one row per batch row")
    H = 0
    if (history is None) != (hist_len is None) or (prompt_len is not None and history is None):
        raise ValueError("history and hist_len go together, and prompt_len needs them")
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 2:
            raise ValueError("history must be an int32 [B, H] tensor")
        H = history.shape[1]
        _check(history, "history", (B, H), torch.int32, dev)
        _check(hist_len, "hist_len", (B,), torch.int32, dev)
        if prompt_len is not None:
            _check(prompt_len, "prompt_len", (B,), torch.int32, dev)
    for t, name in ((repetition, "repetition"), (frequency, "frequency"), (presence, "presence")):
        if t is not None:
            _check(t, name, (B,), torch.float32, dev)
    nb = 0
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    if bias_tokens is not None:
        if not isinstance(bias_tokens, torch.Tensor) or bias_tokens.dim() != 2:
            raise ValueError("bias_tokens must be an int32 [B, n] tensor")
        nb = bias_tokens.shape[1]
        _check(bias_tokens, "bias_tokens", (B, nb), torch.int32, dev)
        _check(bias_values, "bias_values", (B, nb), torch.float32, dev)
    n_admit = 0
    if admit is not None:
        if not isinstance(admit, torch.Tensor) or admit.dim() != 2 or admit.shape[1] != (V + 31) // 32 \
                or admit.shape[0] < 1 or admit.element_size() != 4 or admit.device != dev or not admit.is_contiguous():
            raise ValueError(f"admit must be a contiguous 32-bit [n, {(V + 31) // 32}] mask on {dev}")
        n_admit = admit.shape[0]
        if admit_row is None and n_admit != B * R:
            raise ValueError(f"admit without admit_row must hold B * R = {B * R} rows (got {n_admit})")
    if admit_row is not None:
        if admit is None:
            raise ValueError("admit_row needs admit")
        _check(admit_row, "admit_row", (B, R), torch.int32, dev)
    if draft_len is not None:
        _check(draft_len, "draft_len", (B,), torch.int32, dev)
    _check_sizes(B | R | V | H | nb | n_admit)
    if out is None:
        dtype = kind if out_dtype is None else out_dtype
        if dtype != kind and dtype != torch.float32:
            raise ValueError(f"out_dtype must be float32 or the logits' dtype (got {dtype})")
        out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _check(out, "out", (B, R, V), getattr(out, "dtype", None) if out_dtype is None else out_dtype, dev)
        if out.dtype != logits.dtype and out.dtype != torch.float32:
            raise ValueError(f"out must be float32 or of the logits' dtype (got {out.dtype})")
        a, b = logits.data_ptr(), out.data_ptr()
        if (a != b or out.dtype != logits.dtype) and a < b + out.numel() * out.element_size() \
                and b < a + logits.numel() * logits.element_size():
            raise ValueError("out overlaps logits without being the same tensor")
    _call(forward_lib().spec_adjust, dev, logits.data_ptr(), B, R, V, _LOGITS[logits.dtype], _ptr(tokens), k,
          _ptr(draft_len), _ptr(history), H, _ptr(hist_len), _ptr(prompt_len), _ptr(repetition), _ptr(frequency),
          _ptr(presence), _ptr(bias_tokens), _ptr(bias_values), nb, _ptr(admit), n_admit, _ptr(admit_row),
          out.data_ptr(), _LOGITS[out.dtype])
    return out

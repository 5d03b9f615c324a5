"""PagedAttention over a flattened, variable-length token batch on one GB300.

Thin Python binding of libpkv.so: every function marshals arguments into the
C ABI declared in include/pkv.h and calls it; all computation runs in the
library (CUDA kernels for sm_103a, C++ host code).  PyTorch is used only to
hand over device pointers and the current CUDA stream.  If the library is not
built, importing the binding's entry points raises ImportError.
"""

from __future__ import annotations

import contextlib
import ctypes as C

import numpy as np

from . import _ffi
from ._ffi import (ERR_BLOCK_ID, ERR_METADATA, ERR_NO_BLOCKS, ERR_POSITION,  # noqa: F401
                   ERR_SLOT, ERR_TIMEOUT, PKV_BF16, PKV_F32)

__all__ = [
    "PkvError", "lib", "reshape_and_cache", "rope_reshape_and_cache", "copy_blocks",
    "attention_workspace_bytes", "new_workspace",
    "paged_attention_varlen", "reshape_and_cache_paged_attention", "read_error_word",
    "PreparedCall", "prepare_reshape_and_cache_paged_attention",
    "mxfp4_block_bytes", "new_cache_mxfp4", "reshape_and_cache_mxfp4", "gather_cache_mxfp4",
    "mxfp4_attention_workspace_bytes", "new_workspace_mxfp4", "paged_attention_varlen_mxfp4",
    "fp8_block_bytes", "new_cache_fp8", "reshape_and_cache_fp8", "rope_reshape_and_cache_fp8",
    "gather_cache_fp8", "fp8_attention_workspace_bytes", "new_workspace_fp8",
    "paged_attention_varlen_fp8", "build_cos_sin_cache",
    "build_step_metadata",
    "build_slot_mapping", "Allocator", "Scheduler",
]

_lib = None


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        _lib = _ffi.load()
    return _lib


class PkvError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = lib().pkv_last_error().decode(errors="replace")
        super().__init__(f"{where}: {_ffi.ERRORS.get(code, code)}: {msg}")
        self.code = code


def _check(code: int, where: str) -> int:
    if code < 0:
        raise PkvError(code, where)
    return code


# ---------------------------------------------------------------------------
# device entry points (torch tensors in, no computation here)
# ---------------------------------------------------------------------------
def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return PKV_F32
    if t.dtype == torch.bfloat16:
        return PKV_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream_ptr(stream) -> int | None:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _token_stride(t) -> int:
    # [tokens, heads, dim] with heads and dim contiguous (one stride() call:
    # per-dimension stride(i) calls cost several times more host time)
    st = t.stride()
    if len(st) != 3 or st[2] != 1 or st[1] != t.shape[2]:
        raise ValueError("expected [tokens, heads, head_dim] with contiguous heads and dims")
    return st[0]


def _row_stride(block_table) -> int:
    st = block_table.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError("block_table must be [R, max_blocks] with unit inner stride")
    return st[0]


def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, error_word=None,
                      stream=None) -> None:
    """Scatter key/value [T, Hkv, D] into the caches [NB, B, Hkv, D] at slot_mapping[T] (int64)."""
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    nb, bs, hkv, d = key_cache.shape
    code = lib().pkv_reshape_and_cache(
        key.data_ptr(), value.data_ptr(), _token_stride(key), _token_stride(value),
        key_cache.data_ptr(), value_cache.data_ptr(), slot_mapping.data_ptr(),
        int(slot_mapping.shape[0]), nb, bs, hkv, d, _dtype_code(key_cache),
        error_word.data_ptr() if error_word is not None else None, _stream_ptr(stream))
    _check(code, "reshape_and_cache")


def rope_reshape_and_cache(positions, query, key, value, key_cache, value_cache, slot_mapping,
                           cos_sin_cache, rotary_dim: int | None = None, is_neox: bool = True,
                           key_out=None, error_word=None, stream=None) -> None:
    """Rotate query [T, H, D] in place and key [T, Hkv, D] by cos_sin_cache[positions]
    (float32 [max_position, rotary_dim]), and scatter the rotated key and value
    into the caches [NB, B, Hkv, D] at slot_mapping (int64 [T]).  key_out, if
    given, receives the rotated key too (it may be `key`)."""
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()
            and cos_sin_cache.is_contiguous()):
        raise ValueError("caches and cos_sin_cache must be contiguous")
    import torch
    if cos_sin_cache.dtype != torch.float32 or cos_sin_cache.dim() != 2:
        raise TypeError("cos_sin_cache must be float32 [max_position, rotary_dim]")
    if positions.dtype != torch.int64 or slot_mapping.dtype != torch.int64:
        raise TypeError("positions and slot_mapping must be int64")
    nb, bs, hkv, d = key_cache.shape
    rd = int(cos_sin_cache.shape[1]) if rotary_dim is None else int(rotary_dim)
    if rd != cos_sin_cache.shape[1]:
        raise ValueError("rotary_dim must equal cos_sin_cache.shape[1]")
    ks = _token_stride(key)
    if key_out is not None and _token_stride(key_out) != ks:
        raise ValueError("key_out must have key's token stride")
    code = lib().pkv_rope_reshape_and_cache(
        positions.data_ptr(), query.data_ptr(), _token_stride(query), int(query.shape[1]),
        key.data_ptr(), ks, key_out.data_ptr() if key_out is not None else None,
        value.data_ptr(), _token_stride(value), key_cache.data_ptr(), value_cache.data_ptr(),
        slot_mapping.data_ptr(), cos_sin_cache.data_ptr(), int(cos_sin_cache.shape[0]), rd,
        int(bool(is_neox)), int(positions.shape[0]), nb, bs, hkv, d, _dtype_code(key_cache),
        error_word.data_ptr() if error_word is not None else None, _stream_ptr(stream))
    _check(code, "rope_reshape_and_cache")


def copy_blocks(src_key_cache, src_value_cache, dst_key_cache, dst_value_cache, block_pairs,
                error_word=None, stream=None) -> None:
    """Copy whole blocks: dst[pairs[i, 1]] = src[pairs[i, 0]] for K and V.  Pools are
    [num_blocks, block_size, Hkv, D] tensors (device, or pinned host memory the
    device can map); block_pairs is int32 [n, 2] (device or pinned host)."""
    for t in (src_key_cache, src_value_cache, dst_key_cache, dst_value_cache, block_pairs):
        if not t.is_contiguous():
            raise ValueError("pools and block_pairs must be contiguous")
    if src_key_cache.shape[1:] != dst_key_cache.shape[1:] or \
            src_key_cache.dtype != dst_key_cache.dtype:
        raise ValueError("source and destination pools must have the same block shape and dtype")
    block_bytes = src_key_cache[0].numel() * src_key_cache.element_size()
    code = lib().pkv_copy_blocks(
        src_key_cache.data_ptr(), src_value_cache.data_ptr(), dst_key_cache.data_ptr(),
        dst_value_cache.data_ptr(), block_pairs.data_ptr(), int(block_pairs.shape[0]),
        int(src_key_cache.shape[0]), int(dst_key_cache.shape[0]), block_bytes,
        error_word.data_ptr() if error_word is not None else None, _stream_ptr(stream))
    _check(code, "copy_blocks")


def attention_workspace_bytes(num_reqs: int, num_heads: int, head_dim: int) -> int:
    return int(lib().pkv_attention_workspace_bytes(num_reqs, num_heads, head_dim))


def new_workspace(num_reqs: int, num_heads: int, head_dim: int, device="cuda"):
    """A zero-filled workspace large enough for batches of up to num_reqs requests."""
    import torch
    n = attention_workspace_bytes(num_reqs, num_heads, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def read_error_word(workspace) -> int:
    """The PKV_ERR_* bits the kernels recorded in this workspace (synchronises)."""
    return int(workspace[:4].view(dtype=__import__("torch").int32).item()) & 0xFFFFFFFF


def paged_attention_varlen(q, key_cache, value_cache, block_table, query_start_loc, seq_lens,
                           num_computed_tokens, scale: float, out=None, workspace=None,
                           max_query_len: int = 0, stream=None):
    """Causal GQA attention of the flattened batch q [T, H, D] over the paged caches.

    block_table int32 [R, max_blocks]; query_start_loc int32 [R + 1]; seq_lens,
    num_computed_tokens int32 [R].  Returns out [T, H, D]: a CUDA tensor, or
    a pinned CPU tensor that the kernels store into directly.
    """
    import torch
    T, H, D = q.shape
    nb, bs, hkv, d2 = key_cache.shape
    R = int(seq_lens.shape[0])
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(R, H, D, q.device)
    code = lib().pkv_paged_attention_varlen(
        q.data_ptr(), _token_stride(q), key_cache.data_ptr(), value_cache.data_ptr(),
        block_table.data_ptr(), _row_stride(block_table), query_start_loc.data_ptr(),
        seq_lens.data_ptr(), num_computed_tokens.data_ptr(), float(scale), out.data_ptr(),
        _token_stride(out), T, R, nb, bs, H, hkv, D, _dtype_code(q), int(max_query_len),
        workspace.data_ptr(), workspace.nbytes, _stream_ptr(stream))
    _check(code, "paged_attention_varlen")
    return out


def reshape_and_cache_paged_attention(key, value, slot_mapping, q, key_cache, value_cache,
                                      block_table, query_start_loc, seq_lens, num_computed_tokens,
                                      scale: float, out=None, workspace=None,
                                      max_query_len: int = 0, stream=None):
    """reshape_and_cache of key/value [T, Hkv, D] at slot_mapping (int64 [T]),
    then paged_attention_varlen of q [T, H, D]; one kernel for any bf16
    step.  Returns out [T, H, D]: a CUDA tensor, or a pinned CPU tensor that
    the kernels store into directly."""
    import torch
    T, H, D = q.shape
    nb, bs, hkv, _ = key_cache.shape
    R = int(seq_lens.shape[0])
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(R, H, D, q.device)
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    code = lib().pkv_reshape_and_cache_paged_attention(
        key.data_ptr(), _token_stride(key), value.data_ptr(), _token_stride(value),
        slot_mapping.data_ptr(), q.data_ptr(), _token_stride(q), key_cache.data_ptr(),
        value_cache.data_ptr(), block_table.data_ptr(), _row_stride(block_table),
        query_start_loc.data_ptr(), seq_lens.data_ptr(), num_computed_tokens.data_ptr(),
        float(scale), out.data_ptr(), _token_stride(out), T, R, nb, bs, H, hkv, D, _dtype_code(q),
        int(max_query_len), workspace.data_ptr(), workspace.nbytes, _stream_ptr(stream))
    _check(code, "reshape_and_cache_paged_attention")
    return out


class PreparedCall:
    """A C-ABI call whose arguments were marshalled once.  Calling it makes the
    same library call again, on the stream resolved at preparation: for a
    serving loop whose buffers stay in place from step to step, this leaves
    out the per-call Python work (pointer, stride and stream lookups).  The
    library still validates every call.  The tensors it was prepared from are
    kept alive; their storage and shapes must not change."""

    __slots__ = ("_fn", "_args", "_keep", "_where")

    def __init__(self, fn, args, keep, where):
        self._fn, self._args, self._keep, self._where = fn, args, keep, where

    def __call__(self):
        code = self._fn(*self._args)
        if code < 0:
            raise PkvError(code, self._where)
        return self._keep[0]


def prepare_reshape_and_cache_paged_attention(key, value, slot_mapping, q, key_cache,
                                              value_cache, block_table, query_start_loc,
                                              seq_lens, num_computed_tokens, scale: float, out,
                                              workspace, max_query_len: int = 0, stream=None):
    """reshape_and_cache_paged_attention with its arguments marshalled once;
    returns a PreparedCall that issues the call (and returns out) each time it
    is called.  out and workspace are required: they are part of the state the
    calls reuse."""
    import torch
    T, H, D = q.shape
    nb, bs, hkv, _ = key_cache.shape
    R = int(seq_lens.shape[0])
    if not (key_cache.is_contiguous() and value_cache.is_contiguous()):
        raise ValueError("caches must be contiguous")
    if slot_mapping.dtype != torch.int64:
        raise TypeError("slot_mapping must be int64")
    args = (key.data_ptr(), _token_stride(key), value.data_ptr(), _token_stride(value),
            slot_mapping.data_ptr(), q.data_ptr(), _token_stride(q), key_cache.data_ptr(),
            value_cache.data_ptr(), block_table.data_ptr(), _row_stride(block_table),
            query_start_loc.data_ptr(), seq_lens.data_ptr(), num_computed_tokens.data_ptr(),
            float(scale), out.data_ptr(), _token_stride(out), T, R, nb, bs, H, hkv, D,
            _dtype_code(q), int(max_query_len), workspace.data_ptr(), workspace.nbytes,
            _stream_ptr(stream))
    keep = (out, key, value, slot_mapping, q, key_cache, value_cache, block_table,
            query_start_loc, seq_lens, num_computed_tokens, workspace)
    return PreparedCall(lib().pkv_reshape_and_cache_paged_attention, args, keep,
                        "reshape_and_cache_paged_attention")


# ---------------------------------------------------------------------------
# the 4-bit paged cache and the device-built step metadata
# ---------------------------------------------------------------------------
# These calls launch kernels of a few microseconds, so the checks of each are one
# expression of cheap comparisons (dtype objects, device indices), and what is
# wrong is worked out by name only when something is.
def _check_device(where: str, index: int, *tensors) -> None:
    """The tensors (None allowed) are on CUDA device `index`."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            index = -1
    if index < 0:
        raise ValueError(f"{where}: all tensors must be on one CUDA device")


def _error_ptr(where: str, t):
    """Address of an error word (None: none), a 32-bit integer."""
    if t is None:
        return None
    if t.element_size() != 4 or t.is_floating_point() or t.numel() < 1:
        raise TypeError(f"{where}: error_word must be int32 with at least one entry")
    return t.data_ptr()


def _expect(where: str, name: str, t, dtype, shape) -> None:
    """t is a contiguous tensor of this dtype and shape."""
    if t.dtype is not dtype:
        raise TypeError(f"{where}: {name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be contiguous")


_raw_stream = _current_device = None


def _device_call(where: str, name: str, index: int, stream, *args) -> None:
    """The library's function `name`(*args, stream) with the tensors' device
    current, on its current stream if none is given."""
    global _raw_stream, _current_device
    if _raw_stream is None:
        import torch
        # (the one that is asked for above last: another thread may be here too)
        _current_device = torch._C._cuda_getDevice
        _raw_stream = torch._C._cuda_getCurrentRawStream
    if stream is None:
        ptr = _raw_stream(index)
    else:
        device = getattr(stream, "device", None)
        if device is not None and device.index != index:
            raise ValueError(f"{where}: the stream is on another device than the tensors")
        ptr = stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if index == _current_device():
        code = fn(*args, ptr)
    else:
        import torch
        with torch.cuda.device(index):
            code = fn(*args, ptr)
    if code < 0:
        raise PkvError(code, where)


def _allocating_on(index: int, stream):
    """Context in which a call's own buffers are made: on its stream, so that
    their memory is neither filled nor reused ahead of it.  (Host tensors, which
    the call refuses by name, have index -1.)"""
    import torch
    if index < 0:
        return contextlib.nullcontext()
    if stream is not None:
        return torch.cuda.stream(stream)
    return torch.cuda.device(index)


def mxfp4_block_bytes(num_kv_heads: int, head_dim: int, block_size: int = 16) -> int:
    """Bytes of one block of one 4-bit cache."""
    n = int(lib().pkv_mxfp4_block_bytes(block_size, num_kv_heads, head_dim))
    if n == 0:
        raise ValueError(f"no 4-bit cache of {num_kv_heads} KV heads of {head_dim} in blocks of "
                         f"{block_size}: head_dim is 64 or 128, block_size 16")
    return n


def new_cache_mxfp4(num_blocks: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """(key_cache, value_cache): zeroed 4-bit caches, uint8 [num_blocks, block bytes]."""
    import torch
    shape = (num_blocks, mxfp4_block_bytes(num_kv_heads, head_dim))
    return (torch.zeros(shape, dtype=torch.uint8, device=device),
            torch.zeros(shape, dtype=torch.uint8, device=device))


def _check_pools(where: str, key_cache, value_cache, num_kv_heads: int, head_dim: int,
                 block_bytes=mxfp4_block_bytes) -> None:
    import torch
    if head_dim != 64 and head_dim != 128:
        raise ValueError(f"{where}: head_dim must be 64 or 128, not {head_dim}")
    shape = (key_cache.shape[0], block_bytes(num_kv_heads, head_dim))
    _expect(where, "key_cache", key_cache, torch.uint8, shape)
    _expect(where, "value_cache", value_cache, torch.uint8, shape)


def _rows_and_pools(where: str, key, value, key_cache, value_cache, slot_mapping, error_word,
                    block_bytes=mxfp4_block_bytes):
    """(device index, T, num_blocks, Hkv, D, dtype code) of K and V rows [T, Hkv, D]
    with their caches and slots."""
    import torch
    T, hkv, d = key.shape
    nb = key_cache.shape[0]
    # 16 tokens of head_dim / 2 code bytes and head_dim / 32 scale bytes per KV head, or of
    # head_dim code bytes and 16 for the scale
    pool = (nb, hkv * d * 17 // 2 if block_bytes is mxfp4_block_bytes else hkv * (d + 1) * 16)
    dev = key.get_device()
    u8, dtype = torch.uint8, key.dtype
    if not (dev >= 0 and value.shape == key.shape and value.dtype is dtype
            and key_cache.dtype is u8 and value_cache.dtype is u8
            and key_cache.shape == pool and value_cache.shape == pool and (d == 64 or d == 128)
            and key_cache.is_contiguous() and value_cache.is_contiguous()
            and slot_mapping.dtype is torch.int64 and slot_mapping.shape == (T,)
            and slot_mapping.is_contiguous()
            and value.get_device() == dev == key_cache.get_device()
            and value_cache.get_device() == dev == slot_mapping.get_device()
            and (error_word is None or error_word.get_device() == dev)):
        if value.shape != key.shape or value.dtype is not dtype:
            raise ValueError(f"{where}: the K and the V rows must have one shape and dtype")
        _check_pools(where, key_cache, value_cache, hkv, d, block_bytes)
        _expect(where, "slot_mapping", slot_mapping, torch.int64, (T,))
        _check_device(where, dev, value, key_cache, value_cache, slot_mapping, error_word)
    return dev, T, nb, hkv, d, PKV_BF16 if dtype is torch.bfloat16 else _dtype_code(key)


def reshape_and_cache_mxfp4(key, value, key_cache, value_cache, slot_mapping, error_word=None,
                            stream=None) -> None:
    """Quantise key/value [T, Hkv, D] (bfloat16 or float32) into the 4-bit caches
    (new_cache_mxfp4) at slot_mapping[T] (int64; negative: padding)."""
    where = "reshape_and_cache_mxfp4"
    err = _error_ptr(where, error_word)
    dev, T, nb, hkv, d, dtype = _rows_and_pools(where, key, value, key_cache, value_cache,
                                                slot_mapping, error_word)
    _device_call(where, "pkv_reshape_and_cache_mxfp4", dev, stream, key.data_ptr(),
                 value.data_ptr(), _token_stride(key), _token_stride(value), key_cache.data_ptr(),
                 value_cache.data_ptr(), slot_mapping.data_ptr(), T, nb, 16, hkv, d, dtype, err)


def gather_cache_mxfp4(key_cache, value_cache, slot_mapping, key_out, value_out, error_word=None,
                       stream=None):
    """Read the rows at slot_mapping[T] (int64; negative: the row of the outputs
    is left alone) back from the 4-bit caches into key_out and value_out
    [T, Hkv, D], bfloat16 or float32; exact.  Returns (key_out, value_out)."""
    where = "gather_cache_mxfp4"
    err = _error_ptr(where, error_word)
    dev, T, nb, hkv, d, dtype = _rows_and_pools(where, key_out, value_out, key_cache, value_cache,
                                                slot_mapping, error_word)
    _device_call(where, "pkv_gather_cache_mxfp4", dev, stream, key_cache.data_ptr(),
                 value_cache.data_ptr(), slot_mapping.data_ptr(), key_out.data_ptr(),
                 value_out.data_ptr(), _token_stride(key_out), _token_stride(value_out), T, nb, 16,
                 hkv, d, dtype, err)
    return key_out, value_out


def mxfp4_attention_workspace_bytes(num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    n = int(lib().pkv_mxfp4_attention_workspace_bytes(num_heads, num_kv_heads, head_dim))
    if n == 0:
        raise ValueError(f"no attention over 4-bit caches of {num_heads}/{num_kv_heads} heads of "
                         f"{head_dim}: up to 16 whole query heads per KV head, head_dim 64 or 128")
    return n


def new_workspace_mxfp4(num_heads: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """A workspace of paged_attention_varlen_mxfp4, for any batch.  All but its
    last 256 MiB are needed: a shorter slice serves, with less room for what long
    prompts convert ahead."""
    import torch
    ws = torch.empty(mxfp4_attention_workspace_bytes(num_heads, num_kv_heads, head_dim),
                     dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the error word
    return ws


def paged_attention_varlen_mxfp4(q, key_cache, value_cache, block_table, query_start_loc, seq_lens,
                                 num_computed_tokens, scale: float, out=None, workspace=None,
                                 max_query_len: int = 0, stream=None):
    """paged_attention_varlen over the 4-bit caches: causal GQA attention of the
    flattened batch q [T, H, D] (bfloat16), up to 16 query heads per KV head.
    The number of KV heads is the one the caches' block size gives.  Returns
    out [T, H, D]; rows that belong to no request are left as they were."""
    return _attend_quantised("paged_attention_varlen_mxfp4", "pkv_paged_attention_varlen_mxfp4",
                             mxfp4_block_bytes, new_workspace_mxfp4, lambda D: 17 * D // 2, q, key_cache,
                             value_cache, block_table, query_start_loc, seq_lens, num_computed_tokens,
                             scale, out, workspace, max_query_len, stream)


def _attend_quantised(where: str, name: str, block_bytes, new_workspace_of, head_bytes, q, key_cache,
                      value_cache, block_table, query_start_loc, seq_lens, num_computed_tokens, scale,
                      out, workspace, max_query_len, stream):
    """The attention call over 4-bit or 8-bit caches whose blocks hold head_bytes(D) a KV head."""
    import torch
    T, H, D = q.shape
    chunk = head_bytes(max(2, D))
    hkv = max(1, key_cache.shape[1] // chunk)
    nb, R = key_cache.shape[0], seq_lens.shape[0]
    pool = (nb, hkv * chunk)
    dev = q.get_device()
    u8, i32 = torch.uint8, torch.int32
    if not (dev >= 0 and q.dtype is torch.bfloat16
            and key_cache.dtype is u8 and value_cache.dtype is u8
            and key_cache.shape == pool and value_cache.shape == pool and (D == 64 or D == 128)
            and key_cache.is_contiguous() and value_cache.is_contiguous()
            and block_table.dtype is i32 and block_table.dim() == 2 and block_table.shape[0] == R
            and query_start_loc.dtype is i32 and query_start_loc.shape == (R + 1,)
            and seq_lens.dtype is i32 and seq_lens.dim() == 1
            and num_computed_tokens.dtype is i32 and num_computed_tokens.shape == (R,)
            and query_start_loc.is_contiguous() and seq_lens.is_contiguous()
            and num_computed_tokens.is_contiguous()
            and key_cache.get_device() == dev == value_cache.get_device()
            and block_table.get_device() == dev == query_start_loc.get_device()
            and seq_lens.get_device() == dev == num_computed_tokens.get_device()):
        _check_pools(where, key_cache, value_cache, hkv, D, block_bytes)
        if q.dtype is not torch.bfloat16:
            raise TypeError(f"{where}: q must be bfloat16")
        if block_table.dtype is not i32 or block_table.dim() != 2 or block_table.shape[0] != R:
            raise ValueError(f"{where}: block_table must be int32 [{R}, max_blocks]")
        _expect(where, "query_start_loc", query_start_loc, i32, (R + 1,))
        _expect(where, "seq_lens", seq_lens, i32, (R,))
        _expect(where, "num_computed_tokens", num_computed_tokens, i32, (R,))
        _check_device(where, dev, key_cache, value_cache, block_table, query_start_loc, seq_lens,
                      num_computed_tokens)
    if out is None or workspace is None:
        with _allocating_on(dev, stream):
            if out is None:
                out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
            if workspace is None:
                workspace = new_workspace_of(H, hkv, D, q.device)
    if out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError(f"{where}: out must have q's shape and dtype")
    if out.get_device() != dev or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"{where}: out and a contiguous workspace must be on q's CUDA device")
    _device_call(where, name, dev, stream, q.data_ptr(),
                 _token_stride(q), key_cache.data_ptr(), value_cache.data_ptr(),
                 block_table.data_ptr(), _row_stride(block_table), block_table.shape[1],
                 query_start_loc.data_ptr(), seq_lens.data_ptr(), num_computed_tokens.data_ptr(),
                 float(scale), out.data_ptr(), _token_stride(out), T, R, nb, 16, H, hkv, D, int(max_query_len),
                 workspace.data_ptr(), workspace.nbytes)
    return out


# ---------------------------------------------------------------------------
# the 8-bit paged cache and the table of rotary angles
# ---------------------------------------------------------------------------
def fp8_block_bytes(num_kv_heads: int, head_dim: int, block_size: int = 16) -> int:
    """Bytes of one block of one 8-bit cache."""
    n = int(lib().pkv_fp8_block_bytes(block_size, num_kv_heads, head_dim))
    if n == 0:
        raise ValueError(f"no 8-bit cache of {num_kv_heads} KV heads of {head_dim} in blocks of "
                         f"{block_size}: head_dim is 64 or 128, block_size 16")
    return n


def new_cache_fp8(num_blocks: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """(key_cache, value_cache): zeroed 8-bit caches, uint8 [num_blocks, block bytes]."""
    import torch
    shape = (num_blocks, fp8_block_bytes(num_kv_heads, head_dim))
    return (torch.zeros(shape, dtype=torch.uint8, device=device),
            torch.zeros(shape, dtype=torch.uint8, device=device))


def reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, error_word=None,
                          stream=None) -> None:
    """Quantise key/value [T, Hkv, D] (bfloat16 or float32) into the 8-bit caches
    (new_cache_fp8) at slot_mapping[T] (int64; negative: padding).  The rows of a block and
    KV head share a scale, which grows with them; writing row 0 begins the block anew.  At most
    2^20 tokens: part of the cost grows with their square (131072 in order take 0.5 ms, in no
    order 2.9)."""
    where = "reshape_and_cache_fp8"
    err = _error_ptr(where, error_word)
    dev, T, nb, hkv, d, dtype = _rows_and_pools(where, key, value, key_cache, value_cache,
                                                slot_mapping, error_word, fp8_block_bytes)
    _device_call(where, "pkv_reshape_and_cache_fp8", dev, stream, key.data_ptr(),
                 value.data_ptr(), _token_stride(key), _token_stride(value), key_cache.data_ptr(),
                 value_cache.data_ptr(), slot_mapping.data_ptr(), T, nb, 16, hkv, d, dtype, err)


def rope_reshape_and_cache_fp8(positions, query, key, value, key_cache, value_cache, slot_mapping,
                               cos_sin_cache, is_neox: bool = True, query_out=None,
                               error_word=None, stream=None) -> None:
    """Rotate query [T, H, D] (in place, or to query_out) and key [T, Hkv, D] by
    cos_sin_cache[positions] (float32 [max_position, rotary_dim], as build_cos_sin_cache
    makes it), and quantise the rotated key and the value into the 8-bit caches at
    slot_mapping (int64 [T]) as reshape_and_cache_fp8 does."""
    import torch
    where = "rope_reshape_and_cache_fp8"
    err = _error_ptr(where, error_word)
    if query_out is None:
        query_out = query
    T, d, dev = key.shape[0], key.shape[2], key.get_device()
    if not (query.dim() == 3 and query.shape[0] == T and query.shape[2] == d
            and query.dtype is key.dtype and query_out.shape == query.shape
            and query_out.dtype is query.dtype and positions.dtype is torch.int64
            and positions.shape == (T,) and positions.is_contiguous()
            and cos_sin_cache.dtype is torch.float32 and cos_sin_cache.dim() == 2
            and cos_sin_cache.is_contiguous() and query.get_device() == dev == positions.get_device()
            and query_out.get_device() == dev == cos_sin_cache.get_device()):
        if query.dim() != 3 or query.shape[0] != T or query.shape[2] != d or query.dtype is not key.dtype:
            raise ValueError(f"{where}: query must be [{T}, H, {d}] of key's dtype")
        if query_out.shape != query.shape or query_out.dtype is not query.dtype:
            raise ValueError(f"{where}: query_out must have query's shape and dtype")
        _expect(where, "positions", positions, torch.int64, (T,))
        if cos_sin_cache.dtype is not torch.float32:
            raise TypeError(f"{where}: cos_sin_cache must be float32, not {cos_sin_cache.dtype}")
        if cos_sin_cache.dim() != 2 or not cos_sin_cache.is_contiguous():
            raise ValueError(f"{where}: cos_sin_cache must be a contiguous [max_position, rotary_dim]")
        _check_device(where, dev, query, query_out, positions, cos_sin_cache)
    dev, T, nb, hkv, d, dtype = _rows_and_pools(where, key, value, key_cache, value_cache,
                                                slot_mapping, error_word, fp8_block_bytes)
    _device_call(where, "pkv_rope_reshape_and_cache_fp8", dev, stream, positions.data_ptr(),
                 query.data_ptr(), _token_stride(query), query_out.data_ptr(), _token_stride(query_out),
                 query.shape[1], key.data_ptr(), _token_stride(key), value.data_ptr(),
                 _token_stride(value), key_cache.data_ptr(), value_cache.data_ptr(),
                 slot_mapping.data_ptr(), cos_sin_cache.data_ptr(), cos_sin_cache.shape[0],
                 cos_sin_cache.shape[1], int(bool(is_neox)), T, nb, 16, hkv, d, dtype, err)


def gather_cache_fp8(key_cache, value_cache, slot_mapping, key_out, value_out, error_word=None,
                     stream=None):
    """Read the rows at slot_mapping[T] (int64; negative: the row of the outputs is left
    alone) back from the 8-bit caches into key_out and value_out [T, Hkv, D], bfloat16 or
    float32; exact.  Returns (key_out, value_out)."""
    where = "gather_cache_fp8"
    err = _error_ptr(where, error_word)
    dev, T, nb, hkv, d, dtype = _rows_and_pools(where, key_out, value_out, key_cache, value_cache,
                                                slot_mapping, error_word, fp8_block_bytes)
    _device_call(where, "pkv_gather_cache_fp8", dev, stream, key_cache.data_ptr(),
                 value_cache.data_ptr(), slot_mapping.data_ptr(), key_out.data_ptr(),
                 value_out.data_ptr(), _token_stride(key_out), _token_stride(value_out), T, nb, 16,
                 hkv, d, dtype, err)
    return key_out, value_out


def fp8_attention_workspace_bytes(num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    n = int(lib().pkv_fp8_attention_workspace_bytes(num_heads, num_kv_heads, head_dim))
    if n == 0:
        raise ValueError(f"no attention over 8-bit caches of {num_heads}/{num_kv_heads} heads of "
                         f"{head_dim}: up to 16 whole query heads per KV head, head_dim 64 or 128")
    return n


def new_workspace_fp8(num_heads: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """A workspace of paged_attention_varlen_fp8, for any batch.  All but its last 256 MiB are
    needed: a shorter slice serves, with less room for what long prompts convert ahead."""
    import torch
    ws = torch.empty(fp8_attention_workspace_bytes(num_heads, num_kv_heads, head_dim),
                     dtype=torch.uint8, device=device)
    ws[:256].zero_()  # the error word
    return ws


def paged_attention_varlen_fp8(q, key_cache, value_cache, block_table, query_start_loc, seq_lens,
                               num_computed_tokens, scale: float, out=None, workspace=None,
                               max_query_len: int = 0, stream=None):
    """paged_attention_varlen over the 8-bit caches: causal GQA attention of the flattened
    batch q [T, H, D] (bfloat16), up to 16 query heads per KV head.  The number of KV heads
    is the one the caches' block size gives.  Returns out [T, H, D]; rows that belong to no
    request are left as they were."""
    return _attend_quantised("paged_attention_varlen_fp8", "pkv_paged_attention_varlen_fp8",
                             fp8_block_bytes, new_workspace_fp8, lambda D: 16 * (D + 1), q, key_cache,
                             value_cache, block_table, query_start_loc, seq_lens, num_computed_tokens,
                             scale, out, workspace, max_query_len, stream)


def build_cos_sin_cache(max_position: int, rotary_dim: int, base: float = 10000.0,
                        scaling: str = "none", factor: float = 1.0, original_max_position: int = 0,
                        low: float = 1.0, high: float = 32.0, attention_factor: float | None = None,
                        start: int = 0, out=None, device="cuda", stream=None):
    """The table that the RoPE calls read, float32 [max_position, rotary_dim]: row p has the
    cosines, then the sines, of position start + p (start: to extend a table), times
    attention_factor.  scaling for contexts `factor` times as long: "none"; "linear"
    (positions interpolated); "ntk" (a larger base); "parts" (pairs that turn less than `low`
    times within original_max_position interpolated, those that turn more than `high` times
    kept, mixed in between); "yarn" (mixed over the pairs' indices instead;
    attention_factor is 0.1 ln(factor) + 1 unless given, else 1)."""
    import math

    import torch
    where = "build_cos_sin_cache"
    if scaling not in _ffi.ROPE_SCALINGS:
        raise ValueError(f"{where}: scaling must be one of {', '.join(_ffi.ROPE_SCALINGS)}, not {scaling!r}")
    n, rd = int(max_position), int(rotary_dim)
    if n < 0 or rd <= 0:
        raise ValueError(f"{where}: a table of {n} positions of {rd}")
    if attention_factor is None:
        attention_factor = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor >= 1.0 else 1.0
    if out is None:
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"{where}: the table is made on a CUDA device, not on {device}")
        index = torch.cuda.current_device() if device.index is None else device.index
        with _allocating_on(index, stream):
            out = torch.empty((n, rd), dtype=torch.float32, device=torch.device("cuda", index))
    _expect(where, "out", out, torch.float32, (n, rd))
    _check_device(where, out.get_device())
    _device_call(where, "pkv_build_cos_sin_cache", out.get_device(), stream, out.data_ptr(), n, int(start),
                 rd, float(base), _ffi.ROPE_SCALINGS[scaling], float(factor), int(original_max_position),
                 float(low), float(high), float(attention_factor))
    return out


def build_step_metadata(query_lens, num_computed_tokens, block_table, free_ring, free_state,
                        num_tokens: int, free_state_out=None, query_start_loc=None, seq_lens=None,
                        slot_mapping=None, positions=None, error_word=None, block_size: int = 16,
                        stream=None):
    """The step's metadata built on the device from request lengths (int32 [R]
    tensors): takes each request's new blocks from free_ring (int32) in request
    order, appends them to its row of block_table (int32 [R, max_blocks], in
    place), and returns (query_start_loc int32 [R + 1], seq_lens int32 [R],
    slot_mapping int64 [num_tokens], positions int64 [num_tokens]), padded with
    slot -1 and position 0 behind the last new token.  free_state is int64 [4]
    = {blocks ever taken, blocks ever returned, 0, 0}; the new counts go to
    free_state_out (default: free_state, in place).  A step that does not fit is
    refused whole: an empty step, with the reason's bit in error_word."""
    import torch
    where = "build_step_metadata"
    err = _error_ptr(where, error_word)
    R, T = query_lens.shape[0], int(num_tokens)
    i32, i64 = torch.int32, torch.int64
    dev = query_lens.get_device()
    if free_state_out is None:
        free_state_out = free_state
    if query_start_loc is None or seq_lens is None or slot_mapping is None or positions is None:
        with _allocating_on(dev, stream):
            new = dict(device=query_lens.device)
            if query_start_loc is None:
                query_start_loc = torch.empty(R + 1, dtype=i32, **new)
            if seq_lens is None:
                seq_lens = torch.empty(R, dtype=i32, **new)
            if slot_mapping is None:
                slot_mapping = torch.empty(T, dtype=i64, **new)
            if positions is None:
                positions = torch.empty(T, dtype=i64, **new)
    if not (dev >= 0 and query_lens.dtype is i32 and num_computed_tokens.dtype is i32
            and block_table.dtype is i32 and free_ring.dtype is i32 and free_state.dtype is i64
            and free_state_out.dtype is i64 and query_start_loc.dtype is i32
            and seq_lens.dtype is i32 and slot_mapping.dtype is i64 and positions.dtype is i64
            and query_lens.shape == (R,) == num_computed_tokens.shape == seq_lens.shape
            and block_table.dim() == 2 and block_table.shape[0] == R and free_ring.dim() == 1
            and free_state.shape == (4,) and free_state_out.numel() >= 2
            and query_start_loc.shape == (R + 1,) and slot_mapping.shape == (T,) == positions.shape
            and query_lens.is_contiguous() and num_computed_tokens.is_contiguous()
            and free_ring.is_contiguous() and free_state.is_contiguous()
            and free_state_out.is_contiguous() and query_start_loc.is_contiguous()
            and seq_lens.is_contiguous() and slot_mapping.is_contiguous()
            and positions.is_contiguous()
            and num_computed_tokens.get_device() == dev == block_table.get_device()
            and free_ring.get_device() == dev == free_state.get_device()
            and free_state_out.get_device() == dev == query_start_loc.get_device()
            and seq_lens.get_device() == dev == slot_mapping.get_device()
            and positions.get_device() == dev
            and (error_word is None or error_word.get_device() == dev)):
        _expect(where, "query_lens", query_lens, i32, (R,))
        _expect(where, "num_computed_tokens", num_computed_tokens, i32, (R,))
        if block_table.dtype is not i32 or block_table.dim() != 2 or block_table.shape[0] != R:
            raise ValueError(f"{where}: block_table must be int32 [{R}, max_blocks]")
        if free_ring.dtype is not i32 or free_ring.dim() != 1 or not free_ring.is_contiguous():
            raise ValueError(f"{where}: free_ring must be a contiguous int32 [ring size]")
        _expect(where, "free_state", free_state, i64, (4,))
        if free_state_out.dtype is not i64 or free_state_out.numel() < 2 or \
                not free_state_out.is_contiguous():
            raise ValueError(f"{where}: free_state_out must be int64 with at least 2 entries")
        _expect(where, "query_start_loc", query_start_loc, i32, (R + 1,))
        _expect(where, "seq_lens", seq_lens, i32, (R,))
        _expect(where, "slot_mapping", slot_mapping, i64, (T,))
        _expect(where, "positions", positions, i64, (T,))
        _check_device(where, dev, num_computed_tokens, block_table, free_ring, free_state,
                      free_state_out, query_start_loc, seq_lens, slot_mapping, positions, error_word)
    _device_call(where, "pkv_build_step_metadata", dev, stream, query_lens.data_ptr(),
                 num_computed_tokens.data_ptr(), R, block_table.data_ptr(),
                 _row_stride(block_table), block_table.shape[1], free_ring.data_ptr(),
                 free_ring.numel(),
                 free_state.data_ptr(), free_state_out.data_ptr(), block_size, T,
                 query_start_loc.data_ptr(), seq_lens.data_ptr(), slot_mapping.data_ptr(),
                 positions.data_ptr(), err)
    return query_start_loc, seq_lens, slot_mapping, positions


# ---------------------------------------------------------------------------
# host entry points (numpy arrays)
# ---------------------------------------------------------------------------
def _ptr(a: np.ndarray) -> int:
    # the address as an int (ctypes passes it as void*); cheaper than data_as
    return a.ctypes.data


def build_slot_mapping(block_table: np.ndarray, query_start_loc, num_computed_tokens,
                       block_size: int, out: np.ndarray | None = None) -> np.ndarray:
    """slot_mapping (int64 [num_tokens]) of the step, built on the host; `out`,
    if given, is a C-contiguous int64 array of num_tokens entries (for instance
    a view of a pinned staging buffer) written in place."""
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    qsl = np.ascontiguousarray(query_start_loc, dtype=np.int32)
    nc = np.ascontiguousarray(num_computed_tokens, dtype=np.int32)
    n = int(qsl[-1]) if len(qsl) else 0
    if out is None:
        out = np.empty(n, dtype=np.int64)
    elif out.dtype != np.int64 or out.shape != (n,) or not out.flags.c_contiguous:
        raise ValueError(f"out must be a contiguous int64 array of {n} entries")
    _check(lib().pkv_build_slot_mapping(_ptr(bt), bt.shape[1], _ptr(qsl), _ptr(nc), len(nc),
                                        block_size, _ptr(out), n), "build_slot_mapping")
    return out


class Allocator:
    """Reserve / commit / rollback block allocator (host)."""

    def __init__(self, num_blocks: int, block_size: int, max_blocks_per_req: int | None = None,
                 _handle=None, num_cpu_blocks: int = 0):
        self._own = _handle is None
        self.num_blocks = num_blocks
        self.num_cpu_blocks = num_cpu_blocks
        self._h = _handle or lib().pkv_alloc_create_with_cpu_pool(
            num_blocks, block_size, max_blocks_per_req or num_blocks, num_cpu_blocks)
        if not self._h:
            raise PkvError(-1, "pkv_alloc_create")

    def __del__(self):
        if getattr(self, "_own", False) and self._h:
            lib().pkv_alloc_destroy(self._h)
            self._h = None

    def reserve(self, plan) -> bool:
        """plan: [(req_id, new_tokens)].  False if the blocks are not there."""
        ids = np.array([r for r, _ in plan], dtype=np.int32)
        toks = np.array([s for _, s in plan], dtype=np.int32)
        code = lib().pkv_alloc_reserve(self._h, len(ids), _ptr(ids), _ptr(toks))
        if code == -4:
            return False
        _check(code, "reserve")
        return True

    def commit(self):
        _check(lib().pkv_alloc_commit(self._h), "commit")

    def rollback(self):
        _check(lib().pkv_alloc_rollback(self._h), "rollback")

    def free_request(self, req: int) -> int:
        return _check(lib().pkv_alloc_free_request(self._h, req), "free_request")

    def stats(self) -> dict:
        s = _ffi.AllocStats()
        _check(lib().pkv_alloc_get_stats(self._h, C.byref(s)), "stats")
        return {n: getattr(s, n) for n, _ in s._fields_}

    def table(self, req: int) -> list[int]:
        buf = np.empty(self.num_blocks, dtype=np.int32)
        n = _check(lib().pkv_alloc_table(self._h, req, _ptr(buf), len(buf)), "table")
        return buf[:n].tolist()

    def held_tokens(self, req: int) -> int:
        return int(lib().pkv_alloc_held_tokens(self._h, req))

    def free_list(self) -> list[int]:
        buf = np.empty(self.num_blocks, dtype=np.int32)
        n = _check(lib().pkv_alloc_free_list(self._h, _ptr(buf), len(buf)), "free_list")
        return buf[:n].tolist()

    def check(self):
        _check(lib().pkv_alloc_check(self._h), "check")

    # -- prefix sharing --------------------------------------------------------
    def match_prefix(self, req: int, namespace: int, tokens) -> int:
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        return _check(lib().pkv_alloc_match_prefix(self._h, req, namespace, _ptr(t), len(t)),
                      "match_prefix")

    def peek_prefix(self, namespace: int, tokens) -> tuple[int, int]:
        """(matched tokens, how many matched blocks are cached now)."""
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        cached = C.c_int32(0)
        n = _check(lib().pkv_alloc_peek_prefix(self._h, namespace, _ptr(t), len(t),
                                               C.byref(cached)), "peek_prefix")
        return n, cached.value

    def fork(self, parent: int, child: int) -> None:
        _check(lib().pkv_alloc_fork(self._h, parent, child), "fork")

    def pending_copies(self) -> list[tuple[int, int]]:
        buf = np.empty(2 * max(1, self.num_blocks), dtype=np.int32)
        n = _check(lib().pkv_alloc_pending_copies(self._h, _ptr(buf), len(buf) // 2),
                   "pending_copies")
        return [(int(buf[2 * i]), int(buf[2 * i + 1])) for i in range(n)]

    def prefix_stats(self) -> dict:
        s = _ffi.PrefixStats()
        _check(lib().pkv_alloc_get_prefix_stats(self._h, C.byref(s)), "prefix_stats")
        return {n: getattr(s, n) for n, _ in s._fields_}

    def ref_count(self, block: int) -> int:
        return _check(lib().pkv_alloc_ref_count(self._h, block), "ref_count")

    def cached_list(self) -> list[int]:
        buf = np.empty(self.num_blocks, dtype=np.int32)
        n = _check(lib().pkv_alloc_cached_list(self._h, _ptr(buf), len(buf)), "cached_list")
        return buf[:n].tolist()

    def available(self) -> int:
        return int(lib().pkv_alloc_available(self._h))

    # -- swapping ----------------------------------------------------------------
    def swap_out(self, req: int):
        """([(gpu, cpu)], released) or None if the CPU pool is too small."""
        buf = np.empty(2 * max(1, self.num_blocks), dtype=np.int32)
        rel = C.c_int32(0)
        n = lib().pkv_alloc_swap_out(self._h, req, _ptr(buf), len(buf) // 2, C.byref(rel))
        if n == -4:
            return None
        _check(n, "swap_out")
        return [(int(buf[2 * i]), int(buf[2 * i + 1])) for i in range(n)], rel.value

    def swap_in_status(self, req: int) -> str:
        st = _check(lib().pkv_alloc_swap_in_status(self._h, req), "swap_in_status")
        return ("ok", "later", "never")[st]

    def swap_in(self, req: int) -> list[tuple[int, int]]:
        buf = np.empty(2 * max(1, self.num_blocks), dtype=np.int32)
        n = _check(lib().pkv_alloc_swap_in(self._h, req, _ptr(buf), len(buf) // 2), "swap_in")
        return [(int(buf[2 * i]), int(buf[2 * i + 1])) for i in range(n)]

    def swapped_blocks(self, req: int):
        """(CPU blocks, T_i) of a swapped request, or ([], 0)."""
        buf = np.empty(max(1, self.num_cpu_blocks), dtype=np.int32)
        tok = C.c_int64(0)
        n = _check(lib().pkv_alloc_swapped_blocks(self._h, req, _ptr(buf), len(buf),
                                                  C.byref(tok)), "swapped_blocks")
        return buf[:n].tolist(), tok.value

    def cpu_free_list(self) -> list[int]:
        buf = np.empty(max(1, self.num_cpu_blocks), dtype=np.int32)
        n = _check(lib().pkv_alloc_cpu_free_list(self._h, _ptr(buf), len(buf)), "cpu_free_list")
        return buf[:n].tolist()


class Scheduler:
    """Continuous-batching scheduler with recompute preemption (host)."""

    def __init__(self, max_num_seqs, max_num_batched_tokens, chunk_size, max_model_len,
                 block_size, num_blocks, max_blocks_per_req, artificial_preempt_prob=0.0,
                 artificial_preempt_max=0, artificial_seed=0, preemption_mode="recompute",
                 num_cpu_blocks=0):
        if preemption_mode not in ("recompute", "swap"):
            raise ValueError("preemption_mode must be 'recompute' or 'swap'")
        swap = preemption_mode == "swap"
        cfg = _ffi.SchedConfig(max_num_seqs, max_num_batched_tokens, chunk_size, max_model_len,
                               block_size, num_blocks, max_blocks_per_req, artificial_preempt_max,
                               artificial_preempt_prob, artificial_seed, 1 if swap else 0,
                               num_cpu_blocks)
        self._h = lib().pkv_sched_create(C.byref(cfg))
        if not self._h:
            raise PkvError(-1, "pkv_sched_create")
        self.num_blocks = num_blocks
        self.max_blocks_per_req = max_blocks_per_req
        self.allocator = Allocator(num_blocks, block_size, _handle=lib().pkv_sched_allocator(self._h),
                                   num_cpu_blocks=num_cpu_blocks if swap else 0)
        self.info = _ffi.StepInfo()

    def __del__(self):
        if getattr(self, "_h", None):
            lib().pkv_sched_destroy(self._h)
            self._h = None

    def add_request(self, req_id: int, prompt_len: int, max_output: int, namespace: int = 0,
                    tokens=None) -> bool:
        """Queue a request; with `tokens` (its prompt's token ids) it takes part in
        prefix sharing within `namespace`."""
        if tokens is None:
            code = lib().pkv_sched_add_request(self._h, req_id, prompt_len, max_output)
        else:
            t = np.ascontiguousarray(tokens, dtype=np.int32)
            if len(t) != prompt_len:
                return False
            code = lib().pkv_sched_add_request_tokens(self._h, req_id, prompt_len, max_output,
                                                      namespace, _ptr(t))
        return bool(_check(code, "add_request"))

    def step(self) -> dict:
        _check(lib().pkv_sched_step(self._h, C.byref(self.info)), "step")
        i = self.info
        n = i.num_reqs
        ids = np.empty(n, np.int32)
        toks = np.empty(n, np.int32)
        before = np.empty(n, np.int32)
        lib().pkv_sched_plan(self._h, _ptr(ids), _ptr(toks), _ptr(before), n)
        pre = np.empty(max(i.num_preempted, 1), np.int32)
        adm = np.empty(max(i.num_admitted, 1), np.int32)
        lib().pkv_sched_preempted(self._h, _ptr(pre), len(pre))
        lib().pkv_sched_admitted(self._h, _ptr(adm), len(adm))
        no, ni = C.c_int32(0), C.c_int32(0)
        _check(lib().pkv_sched_swaps(self._h, None, 0, C.byref(no), None, 0, C.byref(ni)), "swaps")
        outp = np.empty(2 * max(1, no.value), np.int32)
        inp = np.empty(2 * max(1, ni.value), np.int32)
        _check(lib().pkv_sched_swaps(self._h, _ptr(outp), no.value, C.byref(no), _ptr(inp),
                                     ni.value, C.byref(ni)), "swaps")
        cap = 1 << 12
        so, si, ig = (np.empty(cap, np.int32) for _ in range(3))
        nso, nsi, nig = C.c_int32(0), C.c_int32(0), C.c_int32(0)
        _check(lib().pkv_sched_swap_events(self._h, _ptr(so), C.byref(nso), _ptr(si),
                                           C.byref(nsi), _ptr(ig), C.byref(nig), cap), "swap_events")
        return {"entries": list(zip(ids.tolist(), toks.tolist(), before.tolist())),
                "preempted": pre[:i.num_preempted].tolist(), "admitted": adm[:i.num_admitted].tolist(),
                "swap_out_pairs": [tuple(x) for x in outp[:2 * no.value].reshape(-1, 2).tolist()],
                "swap_in_pairs": [tuple(x) for x in inp[:2 * ni.value].reshape(-1, 2).tolist()],
                "swapped_out": so[:nso.value].tolist(), "swapped_in": si[:nsi.value].tolist(),
                "ignored": ig[:nig.value].tolist(),
                "num_tokens": int(i.num_tokens), "max_blocks": int(i.max_blocks),
                "max_query_len": int(i.max_query_len)}

    def build_metadata(self, block_table, query_start_loc, seq_lens, num_computed, slot_mapping):
        """Fill caller-owned numpy buffers (e.g. views of pinned host tensors)."""
        _check(lib().pkv_sched_build_metadata(
            self._h, _ptr(block_table), block_table.shape[1], _ptr(query_start_loc),
            _ptr(seq_lens), _ptr(num_computed), _ptr(slot_mapping)), "build_metadata")

    def metadata(self, stride: int | None = None):
        i = self.info
        stride = stride or max(int(i.max_blocks), 1)
        bt = np.empty((i.num_reqs, stride), np.int32)
        qsl = np.empty(i.num_reqs + 1, np.int32)
        seq = np.empty(i.num_reqs, np.int32)
        nc = np.empty(i.num_reqs, np.int32)
        slots = np.empty(int(i.num_tokens), np.int64)
        self.build_metadata(bt, qsl, seq, nc, slots)
        return bt, qsl, seq, nc, slots

    def finish_step(self, executed_ok: bool) -> list[int]:
        buf = np.empty(1024, np.int32)
        n = _check(lib().pkv_sched_finish_step(self._h, 1 if executed_ok else 0, _ptr(buf),
                                               len(buf)), "finish_step")
        return buf[:min(n, len(buf))].tolist()

    def request(self, req_id: int) -> dict | None:
        st = _ffi.RequestState()
        code = lib().pkv_sched_request(self._h, req_id, C.byref(st))
        if code == -6:
            return None
        _check(code, "request")
        return {n: getattr(st, n) for n, _ in st._fields_ if n != "pad_"}

    def queues(self):
        cap = 1 << 16
        run = np.empty(cap, np.int32)
        wait = np.empty(cap, np.int32)
        nr, nw = C.c_int32(0), C.c_int32(0)
        _check(lib().pkv_sched_queues(self._h, _ptr(run), C.byref(nr), _ptr(wait), C.byref(nw),
                                      cap), "queues")
        return run[:nr.value].tolist(), wait[:nw.value].tolist()

    def swapped_queue(self) -> list[int]:
        cap = 1 << 16
        buf = np.empty(cap, np.int32)
        n = C.c_int32(0)
        _check(lib().pkv_sched_swapped_queue(self._h, _ptr(buf), C.byref(n), cap), "swapped_queue")
        return buf[:n.value].tolist()

    def counters(self) -> dict:
        out = (C.c_int64 * 4)()
        _check(lib().pkv_sched_counters(self._h, out), "counters")
        return {"preemptions": out[0], "recomputed_tokens": out[1], "finished": out[2],
                "inject_left": out[3]}

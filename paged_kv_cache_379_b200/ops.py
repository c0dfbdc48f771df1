"""Python binding of the C ABI: the same names, argument marshalling only.

Each function checks dtypes / devices / contiguity of the torch tensors it is
given, passes their device pointers and the current CUDA stream to the
library, and raises :class:`PagedKVError` on a negative status.  Every step of
the computation runs in the library's CUDA kernels; nothing here computes.

Tensor conventions (see include/pagedkv.h):
  key_cache, value_cache : bf16 [num_blocks, block_size, num_kv_heads, head_dim]
  query, out             : bf16 [num_seqs, num_heads, head_dim]
  block_tables           : int32 [num_seqs, max_blocks_per_seq]
  seq_lens               : int32 [num_seqs]
  slot_mapping           : int64 [num_tokens]
  src_dst_pairs          : int64 [num_pairs, 2]
  FP8 caches             : uint8 E4M3 codes [num_blocks, block_size, num_kv_heads, head_dim]
                           with one fp32 scale per cache (k_scale, v_scale)
  4-bit caches             : uint8 [num_blocks, num_kv_heads, block_size * (head_dim / 2 + 4)]
                           (codes, then a bf16 (scale, zero) pair per row; new_int4_cache);
                           copy_blocks and swap_blocks take cache.view(torch.bfloat16).unsqueeze(1)
"""

from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._lib import PagedKVError, check, load  # noqa: F401

# First bytes of every decode workspace: the dynamic scheduler's counters.
WORKSPACE_HEADER_BYTES = 256

__all__ = [
    "slot_mapping", "reshape_and_cache", "copy_blocks", "decode", "decode_one_pass",
    "decode_split", "decode_partitions", "lse_reduce", "decode_workspace_size", "decode_plan",
    "validate_tables", "device_status", "PagedKVError", "new_workspace", "workspace_views",
    "decode_split_noalloc", "swap_blocks", "reshape_and_cache_fp8", "decode_fp8", "decode_fp8_split",
    "prefill", "append_decode_kv", "append_decode_kv_fp8", "selftest_bounded_wait", "append_decode_kv_cow",
    "cow_sources", "prefix_groups", "decode_shared",
    "int4_record_bytes", "new_int4_cache", "reshape_and_cache_int4", "append_decode_kv_int4",
    "dequantize_blocks_int4", "decode_int4", "decode_int4_workspace_size", "new_int4_workspace",
    "qk_norm_rope", "qk_norm_rope_cache", "qk_norm_rope_cache_fp8", "qk_norm_rope_cache_int4",
    "prepare_batch", "release_blocks",
]


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor | None, dtype, name: str, ndim: int | None = None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t.data_ptr()


def _cache_dims(key_cache, value_cache, dtype=torch.bfloat16):
    _dev(key_cache, dtype, "key_cache", 4)
    _dev(value_cache, dtype, "value_cache", 4)
    if key_cache.shape != value_cache.shape:
        raise ValueError("key_cache and value_cache shapes differ")
    nb, bs, hkv, d = key_cache.shape
    return nb, bs, hkv, d


def slot_mapping(block_tables, block_size: int, *, seq_lens=None, positions=None, seq_ids=None,
                 out=None, stream=None):
    """Device address translation; decode form (positions=None) uses pos = seq_len - 1."""
    lib = load()
    bt = _dev(block_tables, torch.int32, "block_tables", 2)
    n = positions.shape[0] if positions is not None else (
        seq_ids.shape[0] if seq_ids is not None else seq_lens.shape[0])
    if out is None:
        out = torch.empty(n, dtype=torch.int64, device=block_tables.device)
    check("pa_slot_mapping", lib.pa_slot_mapping(
        _dev(out, torch.int64, "out", 1), bt, block_tables.shape[0], block_tables.shape[1],
        _dev(seq_ids, torch.int32, "seq_ids", 1),
        _dev(positions, torch.int64, "positions", 1), _dev(seq_lens, torch.int32, "seq_lens", 1),
        n, int(block_size), _stream(stream)))
    return out


def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, stream=None) -> None:
    lib = load()
    nb, bs, hkv, d = _cache_dims(key_cache, value_cache)
    k = _dev(key, torch.bfloat16, "key", 3)
    v = _dev(value, torch.bfloat16, "value", 3)
    if tuple(key.shape[1:]) != (hkv, d) or key.shape != value.shape:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_dim] matching the cache")
    sm = _dev(slot_mapping, torch.int64, "slot_mapping", 1)
    if slot_mapping.shape[0] != key.shape[0]:
        raise ValueError("slot_mapping length != num_tokens")
    check("pa_reshape_and_cache", lib.pa_reshape_and_cache(
        k, v, key_cache.data_ptr(), value_cache.data_ptr(), sm, key.shape[0], hkv, d, bs, nb,
        _stream(stream)))


def reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale: float, v_scale: float,
                          stream=None) -> None:
    """pa_reshape_and_cache_fp8: bf16 rows quantised to E4M3 codes in uint8 caches."""
    lib = load()
    nb, bs, hkv, d = _cache_dims(key_cache, value_cache, torch.uint8)
    k = _dev(key, torch.bfloat16, "key", 3)
    v = _dev(value, torch.bfloat16, "value", 3)
    if tuple(key.shape[1:]) != (hkv, d) or key.shape != value.shape:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_dim] matching the cache")
    sm = _dev(slot_mapping, torch.int64, "slot_mapping", 1)
    if slot_mapping.shape[0] != key.shape[0]:
        raise ValueError("slot_mapping length != num_tokens")
    check("pa_reshape_and_cache_fp8", lib.pa_reshape_and_cache_fp8(
        k, v, key_cache.data_ptr(), value_cache.data_ptr(), sm, key.shape[0], hkv, d, bs, nb, float(k_scale),
        float(v_scale), _stream(stream)))


def _append_args(key, value, key_cache, value_cache, block_tables, seq_lens, slot_mapping, cache_dtype):
    nb, bs, hkv, d = _cache_dims(key_cache, value_cache, cache_dtype)
    k = _dev(key, torch.bfloat16, "key", 3)
    v = _dev(value, torch.bfloat16, "value", 3)
    B = seq_lens.shape[0]
    if tuple(key.shape) != (B, hkv, d) or key.shape != value.shape:
        raise ValueError("key/value must be [num_seqs, num_kv_heads, head_dim] matching the cache")
    bt = _dev(block_tables, torch.int32, "block_tables", 2)
    if block_tables.shape[0] != B:
        raise ValueError("block_tables rows != num_seqs")
    sm = _dev(slot_mapping, torch.int64, "slot_mapping", 1)
    return (k, v, key_cache.data_ptr(), value_cache.data_ptr(), bt, _dev(seq_lens, torch.int32, "seq_lens", 1), sm,
            B, block_tables.shape[1], hkv, d, bs, nb)


def append_decode_kv(key, value, key_cache, value_cache, block_tables, seq_lens, slot_mapping=None,
                     stream=None) -> None:
    """pa_append_decode_kv: slot of each sequence's newest position + cache write, one launch."""
    a = _append_args(key, value, key_cache, value_cache, block_tables, seq_lens, slot_mapping, torch.bfloat16)
    check("pa_append_decode_kv", load().pa_append_decode_kv(*a, _stream(stream)))


def append_decode_kv_cow(key, value, key_cache, value_cache, block_tables, seq_lens, cow_src, slot_mapping=None,
                         stream=None) -> None:
    """pa_append_decode_kv_cow: the step's copy-on-write copies and cache write,
    one launch; cow_src int32 [num_seqs] (device): the block each sequence's
    write block is a copy of, or -1 (see cow_sources)."""
    a = _append_args(key, value, key_cache, value_cache, block_tables, seq_lens, slot_mapping, torch.bfloat16)
    cs = _dev(cow_src, torch.int32, "cow_src", 1)
    if cow_src is not None and cow_src.shape[0] != seq_lens.shape[0]:
        raise ValueError("cow_src length != num_seqs")
    check("pa_append_decode_kv_cow", load().pa_append_decode_kv_cow(*a[:6], cs, *a[6:], _stream(stream)))


def cow_sources(slot_mapping, block_size: int, src_dst_pairs) -> np.ndarray:
    """pa_cow_sources (host): per-sequence copy source of the block each slot
    lies in, from the pool's (src, dst) pairs; -1 where none."""
    slots = np.ascontiguousarray(slot_mapping, dtype=np.int64)
    pairs = np.ascontiguousarray(src_dst_pairs, dtype=np.int64).reshape(-1, 2)
    out = np.empty(slots.shape[0], dtype=np.int32)
    check("pa_cow_sources", load().pa_cow_sources(
        slots.ctypes.data_as(ctypes.c_void_p), int(slots.shape[0]), int(block_size),
        pairs.ctypes.data_as(ctypes.c_void_p), int(pairs.shape[0]), out.ctypes.data_as(ctypes.c_void_p)))
    return out


def prefix_groups(block_tables, seq_lens, block_size: int, partition_size: int):
    """pa_prefix_groups (host): runs of consecutive sequences sharing leading
    partitions.  Returns (group_start int32 [G+1], group_parts int32 [G])."""
    bt = np.ascontiguousarray(block_tables, dtype=np.int32)
    sl = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B = int(sl.shape[0])
    start = np.empty(B + 1, dtype=np.int32)
    parts = np.empty(max(B, 1), dtype=np.int32)
    n = ctypes.c_int(0)
    check("pa_prefix_groups", load().pa_prefix_groups(
        bt.ctypes.data_as(ctypes.c_void_p), B, int(bt.shape[1]) if bt.ndim == 2 else 1,
        sl.ctypes.data_as(ctypes.c_void_p), int(block_size), int(partition_size),
        start.ctypes.data_as(ctypes.c_void_p), parts.ctypes.data_as(ctypes.c_void_p), ctypes.byref(n)))
    return start[:n.value + 1].copy(), parts[:n.value].copy()


def append_decode_kv_fp8(key, value, key_cache, value_cache, block_tables, seq_lens, k_scale: float,
                         v_scale: float, slot_mapping=None, stream=None) -> None:
    """pa_append_decode_kv_fp8: as append_decode_kv into E4M3 code caches."""
    a = _append_args(key, value, key_cache, value_cache, block_tables, seq_lens, slot_mapping, torch.uint8)
    check("pa_append_decode_kv_fp8", load().pa_append_decode_kv_fp8(*a, float(k_scale), float(v_scale),
                                                                    _stream(stream)))


def copy_blocks(key_cache, value_cache, src_dst_pairs, stream=None) -> None:
    lib = load()
    nb, bs, hkv, d = _cache_dims(key_cache, value_cache)
    pr = _dev(src_dst_pairs, torch.int64, "src_dst_pairs", 2)
    if src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be [num_pairs, 2]")
    check("pa_copy_blocks", lib.pa_copy_blocks(
        key_cache.data_ptr(), value_cache.data_ptr(), pr, src_dst_pairs.shape[0], hkv, d, bs, nb,
        _stream(stream)))


def swap_blocks(dst_key_cache, dst_value_cache, src_key_cache, src_value_cache, src_dst_pairs, stream=None) -> None:
    """pa_swap_blocks: block copies between a device cache and a pinned host cache (either way).

    Host-side tensors must be pinned (``tensor.pin_memory()``); ``src_dst_pairs``
    is an int64 [P, 2] tensor in device or pinned host memory."""
    lib = load()
    for name, t in (("dst_key_cache", dst_key_cache), ("dst_value_cache", dst_value_cache),
                    ("src_key_cache", src_key_cache), ("src_value_cache", src_value_cache)):
        if t.dtype != torch.bfloat16 or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous bf16 [num_blocks, block_size, heads, head_dim] tensor")
        if not t.is_cuda and not t.is_pinned():
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
    if src_key_cache.shape[1:] != dst_key_cache.shape[1:] or src_key_cache.shape != src_value_cache.shape or \
            dst_key_cache.shape != dst_value_cache.shape:
        raise ValueError("cache shapes do not match")
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2 or \
            not src_dst_pairs.is_contiguous():
        raise ValueError("src_dst_pairs must be a contiguous int64 [P, 2] tensor")
    _, bs, hkv, d = src_key_cache.shape
    check("pa_swap_blocks", lib.pa_swap_blocks(
        dst_key_cache.data_ptr(), dst_value_cache.data_ptr(), src_key_cache.data_ptr(), src_value_cache.data_ptr(),
        src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], hkv, d, bs, src_key_cache.shape[0],
        dst_key_cache.shape[0], _stream(stream)))


def _decode_common(query, key_cache, value_cache, block_tables, seq_lens, cache_dtype=torch.bfloat16):
    nb, bs, hkv, d = _cache_dims(key_cache, value_cache, cache_dtype)
    q = _dev(query, torch.bfloat16, "query", 3)
    B, hq, dq = query.shape
    if dq != d:
        raise ValueError("query head_dim != cache head_dim")
    bt = _dev(block_tables, torch.int32, "block_tables", 2)
    sl = _dev(seq_lens, torch.int32, "seq_lens", 1)
    if block_tables.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_tables / seq_lens batch size != query batch size")
    return q, bt, sl, B, hq, hkv, d, bs, nb, block_tables.shape[1]


def decode_workspace_size(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
                          partition_size: int = 0) -> int:
    """Bytes of decode workspace; partition_size 0 = what pa_decode would choose."""
    return int(load().pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len,
                                               partition_size))


def decode_plan(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
                workspace_bytes: int) -> int:
    """0 if pa_decode runs one pass for these sizes, else the split partition size."""
    return int(load().pa_decode_plan(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len,
                                     int(workspace_bytes)))


def _out(out, query):
    if out is None:
        out = torch.empty_like(query)
    return _dev(out, torch.bfloat16, "out", 3), out


def _ws(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def decode(query, key_cache, value_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
           *, out=None, workspace=None, stream=None):
    """pa_decode: one pass or split, chosen by the library."""
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens)
    o, out = _out(out, query)
    wp, wb = _ws(workspace)
    check("pa_decode", lib.pa_decode(o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale),
                                     bs, hkv, B, hq, d, mb, nb, int(max_seq_len), wp, wb, _stream(stream)))
    return out


def decode_fp8(query, key_cache, value_cache, block_tables, seq_lens, scale: float, k_scale: float,
               v_scale: float, max_seq_len: int, *, out=None, workspace=None, stream=None):
    """pa_decode_fp8: pa_decode over uint8 E4M3 caches with per-tensor scales."""
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens,
                                                          torch.uint8)
    o, out = _out(out, query)
    wp, wb = _ws(workspace)
    check("pa_decode_fp8", lib.pa_decode_fp8(
        o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), float(k_scale), float(v_scale),
        bs, hkv, B, hq, d, mb, nb, int(max_seq_len), wp, wb, _stream(stream)))
    return out


def decode_fp8_split(query, key_cache, value_cache, block_tables, seq_lens, scale: float, k_scale: float,
                     v_scale: float, max_seq_len: int, partition_size: int, workspace=None, *, out=None,
                     stream=None):
    """pa_decode_fp8_split: partition_size 0 = one pass, else the split form."""
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens,
                                                          torch.uint8)
    o, out = _out(out, query)
    wp, wb = _ws(workspace)
    check("pa_decode_fp8_split", lib.pa_decode_fp8_split(
        o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), float(k_scale), float(v_scale),
        bs, hkv, B, hq, d, mb, nb, int(max_seq_len), int(partition_size), wp, wb, _stream(stream)))
    return out


def prefill(query, key_cache, value_cache, block_tables, seq_lens, q_start, scale: float, *, out=None,
            stream=None):
    """pa_prefill: causal multi-query attention of each sequence's chunk (query rows
    q_start[s] .. q_start[s+1]-1, the last positions of the sequence) over its paged cache."""
    if not (float(scale) > 0.0 and float(scale) < float("inf")):
        raise ValueError("scale must be positive and finite")
    lib = load()
    nb, bs, hkv, d = _cache_dims(key_cache, value_cache)
    q = _dev(query, torch.bfloat16, "query", 3)
    T, hq, dq = query.shape
    if dq != d:
        raise ValueError("query head_dim != cache head_dim")
    bt = _dev(block_tables, torch.int32, "block_tables", 2)
    sl = _dev(seq_lens, torch.int32, "seq_lens", 1)
    qs = _dev(q_start, torch.int32, "q_start", 1)
    B = seq_lens.shape[0]
    if block_tables.shape[0] != B or q_start.shape[0] != B + 1:
        raise ValueError("block_tables rows / q_start length do not match seq_lens")
    o, out = _out(out, query)
    check("pa_prefill", lib.pa_prefill(o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, qs,
                                       float(scale), bs, hkv, B, hq, d, block_tables.shape[1], nb, T,
                                       _stream(stream)))
    return out


def decode_one_pass(query, key_cache, value_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                    *, out=None, stream=None):
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens)
    o, out = _out(out, query)
    check("pa_decode_one_pass", lib.pa_decode_one_pass(
        o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), bs, hkv, B, hq, d, mb, nb,
        int(max_seq_len), _stream(stream)))
    return out


def decode_split(query, key_cache, value_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                 partition_size: int, workspace, *, out=None, stream=None):
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens)
    o, out = _out(out, query)
    wp, wb = _ws(workspace)
    check("pa_decode_split", lib.pa_decode_split(
        o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), bs, hkv, B, hq, d, mb, nb,
        int(max_seq_len), int(partition_size), wp, wb, _stream(stream)))
    return out


def decode_shared(query, key_cache, value_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                  partition_size: int, group_start, group_parts, workspace, *, out=None, stream=None):
    """pa_decode_shared: the split decode with shared-prefix groups (int32 device
    tensors group_start [G+1], group_parts [G]; see prefix_groups)."""
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens)
    o, out = _out(out, query)
    wp, wb = _ws(workspace)
    gs = _dev(group_start, torch.int32, "group_start", 1)
    gp = _dev(group_parts, torch.int32, "group_parts", 1)
    ng = int(group_parts.shape[0])
    if group_start.shape[0] != ng + 1:
        raise ValueError("group_start must have num_groups + 1 entries")
    check("pa_decode_shared", lib.pa_decode_shared(
        o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), bs, hkv, B, hq, d, mb, nb,
        int(max_seq_len), int(partition_size), gs, gp, ng, wp, wb, _stream(stream)))
    return out


# ---- 4-bit cache ----------------------------------------------------------------------

# The calls below are made once per layer and step, where the time of the marshalling itself counts: they ask
# each tensor for as little as the checks need (get_device, dim and size answer without building objects).

# torch.cuda.current_device() without its check for a first use, and current_stream(dev).cuda_stream without the
# objects; a torch built without CUDA has neither name
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _device(t, name: str) -> int:
    """The device of a call's first tensor: the library launches on the current one, so it has to be that."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{_current_device()}")
    return dev


def _on(dev: int, t, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    d = t.get_device()
    if d != dev:
        raise ValueError(f"{name} must be a CUDA tensor" if d < 0 else f"{name} is on cuda:{d}, not on cuda:{dev}")


def _arr(dev: int, t, dtype, name: str, ndim: int, n: int = -1):
    """Pointer of a contiguous tensor of a type and rank (and length, where n >= 0) on the call's device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        shape = t.shape
        if len(shape) == ndim and (n < 0 or shape[0] == n):
            return t.data_ptr()
    _on(dev, t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    raise ValueError(f"{name} must have {n} entries, got {t.size(0)}")


def _opt(dev: int, t, dtype, name: str, n: int):
    return None if t is None else _arr(dev, t, dtype, name, 1, n)


def _rows(dev: int, t, name: str, tokens: int, heads: int, head_dim: int):
    """(pointer, token stride) of a bf16 [tokens, heads, head_dim] view whose rows are contiguous."""
    _on(dev, t, name)
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != (tokens, heads, head_dim):
        raise ValueError(f"{name} must be {[tokens, heads, head_dim]}, got {list(t.shape)}")
    st = t.stride()
    if tokens and (st[2] != 1 or (heads > 1 and st[1] != head_dim)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (st[0] if tokens > 1 else heads * head_dim)


def _dims3(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must have 3 dims, got {tuple(shape)}")
    return shape


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return _current_raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _output(make, shape, device, stream):
    """A call's default output (bf16), allocated and filled in the order of the stream that the call runs on: on
    another one, its fill, or what the allocator's last user of that memory still has in flight, could land on top
    of the result."""
    if stream is None:
        return make(shape, dtype=torch.bfloat16, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_raw_stream(stream, device.index), device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=torch.bfloat16, device=device)


def int4_record_bytes(block_size: int, head_dim: int) -> int:
    """Bytes of one (block, KV head) record of a 4-bit cache."""
    return int(block_size) * (int(head_dim) // 2 + 4)


def new_int4_cache(num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """A zero-filled 4-bit cache tensor (one of the two: keys or values)."""
    return torch.zeros(num_blocks, num_kv_heads, int4_record_bytes(block_size, head_dim), dtype=torch.uint8,
                       device=device)


def _int4_caches(dev: int, key_cache, value_cache, head_dim: int):
    """(key pointer, value pointer, num_blocks, block_size, num_kv_heads) of two 4-bit caches."""
    kc = _arr(dev, key_cache, torch.uint8, "key_cache", 3)
    vc = _arr(dev, value_cache, torch.uint8, "value_cache", 3)
    shape = key_cache.shape
    if value_cache.shape != shape:
        raise ValueError("key_cache and value_cache shapes differ")
    nb, hkv, rec = shape
    row = head_dim // 2 + 4
    if head_dim <= 0 or rec % row != 0:
        raise ValueError(f"cache records of {rec} bytes do not hold rows of head_dim {head_dim}")
    return kc, vc, nb, rec // row, hkv


def reshape_and_cache_int4(key, value, key_cache, value_cache, slot_mapping, stream=None) -> None:
    """pa_reshape_and_cache_int4: bf16 rows (strided by token) quantised into 4-bit caches."""
    dev = _device(key, "key")
    T, _, d = _dims3(key, "key")
    kc, vc, nb, bs, hkv = _int4_caches(dev, key_cache, value_cache, d)
    k, ks = _rows(dev, key, "key", T, hkv, d)
    v, vs = _rows(dev, value, "value", T, hkv, d)
    sm = _arr(dev, slot_mapping, torch.int64, "slot_mapping", 1, T)
    check("pa_reshape_and_cache_int4", load().pa_reshape_and_cache_int4(
        k, v, ks, vs, kc, vc, sm, T, hkv, d, bs, nb, _raw_stream(stream, dev)))


def append_decode_kv_int4(key, value, key_cache, value_cache, block_tables, seq_lens, slot_mapping=None,
                          stream=None) -> None:
    """pa_append_decode_kv_int4: as append_decode_kv into 4-bit caches."""
    dev = _device(key, "key")
    B, _, d = _dims3(key, "key")
    kc, vc, nb, bs, hkv = _int4_caches(dev, key_cache, value_cache, d)
    k, ks = _rows(dev, key, "key", B, hkv, d)
    v, vs = _rows(dev, value, "value", B, hkv, d)
    bt = _arr(dev, block_tables, torch.int32, "block_tables", 2, B)
    sl = _arr(dev, seq_lens, torch.int32, "seq_lens", 1, B)
    sm = _opt(dev, slot_mapping, torch.int64, "slot_mapping", B)
    check("pa_append_decode_kv_int4", load().pa_append_decode_kv_int4(
        k, v, ks, vs, kc, vc, bt, sl, sm, B, block_tables.size(1), hkv, d, bs, nb, _raw_stream(stream, dev)))


def dequantize_blocks_int4(key_cache, value_cache, block_ids, head_dim: int, *, key_out=None, value_out=None,
                           stream=None):
    """pa_dequantize_blocks_int4: the listed blocks as bf16 blocks [n, block_size, num_kv_heads, head_dim]."""
    dev, d = _device(key_cache, "key_cache"), int(head_dim)
    kc, vc, nb, bs, hkv = _int4_caches(dev, key_cache, value_cache, d)
    ids = _arr(dev, block_ids, torch.int32, "block_ids", 1)
    n = block_ids.size(0)
    if key_out is None:
        key_out = _output(torch.zeros, (n, bs, hkv, d), key_cache.device, stream)
    if value_out is None:
        value_out = _output(torch.zeros, (n, bs, hkv, d), key_cache.device, stream)
    ko = _arr(dev, key_out, torch.bfloat16, "key_out", 4, n)
    vo = _arr(dev, value_out, torch.bfloat16, "value_out", 4, n)
    shape = (n, bs, hkv, d)
    if key_out.shape != shape or value_out.shape != shape:
        raise ValueError(f"key_out / value_out must be {list(shape)}")
    check("pa_dequantize_blocks_int4", load().pa_dequantize_blocks_int4(
        ko, vo, kc, vc, ids, n, hkv, d, bs, nb, _raw_stream(stream, dev)))
    return key_out, value_out


def decode_int4_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of decode_int4 workspace; the same for every batch."""
    return int(load().pa_decode_int4_workspace_size(num_heads, num_kv_heads, head_dim))


def new_int4_workspace(num_heads: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """A zero-filled decode_int4 workspace (its counters must start at zero)."""
    return torch.zeros(decode_int4_workspace_size(num_heads, num_kv_heads, head_dim), dtype=torch.uint8,
                       device=device)


def decode_int4(query, key_cache, value_cache, block_tables, seq_lens, scale: float, workspace, *, out=None,
                stream=None):
    """pa_decode_int4: single-query paged decode over 4-bit caches."""
    dev = _device(query, "query")
    q = _arr(dev, query, torch.bfloat16, "query", 3)
    shape = query.shape
    B, hq, d = shape
    kc, vc, nb, bs, hkv = _int4_caches(dev, key_cache, value_cache, d)
    bt = _arr(dev, block_tables, torch.int32, "block_tables", 2, B)
    sl = _arr(dev, seq_lens, torch.int32, "seq_lens", 1, B)
    if out is None:
        out = _output(torch.empty, shape, query.device, stream)
    o = _arr(dev, out, torch.bfloat16, "out", 3, B)
    if out.shape != shape:
        raise ValueError("out must have the query's shape")
    if workspace is None:
        wp, wb = None, 0
    else:
        _on(dev, workspace, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        wp, wb = workspace.data_ptr(), workspace.nbytes
    check("pa_decode_int4", load().pa_decode_int4(
        o, q, kc, vc, bt, sl, float(scale), bs, hkv, B, hq, d, block_tables.size(1), nb, wp, wb,
        _raw_stream(stream, dev)))
    return out


# ---- head norm + rotation -------------------------------------------------------------

def _rope_args(query, key, q_weight, k_weight, cos_sin, positions, query_out, stream):
    """What the rotation calls share: the device, the sizes, and the leading pointers."""
    dev = _device(query, "query")
    T, hq, d = _dims3(query, "query")
    hkv = _dims3(key, "key")[1]
    q, qs = _rows(dev, query, "query", T, hq, d)
    k, ks = _rows(dev, key, "key", T, hkv, d)
    qw = _opt(dev, q_weight, torch.bfloat16, "q_weight", d)
    kw = _opt(dev, k_weight, torch.bfloat16, "k_weight", d)
    cs = _arr(dev, cos_sin, torch.float32, "cos_sin", 2)
    ps = _arr(dev, positions, torch.int64, "positions", 1, T)
    if query_out is None:
        query_out = _output(torch.empty, (T, hq, d), query.device, stream)
    qo, qos = _rows(dev, query_out, "query_out", T, hq, d)
    return dev, T, hq, hkv, d, query_out, qo, qos, q, qs, k, ks, (qw, kw, cs, ps)


def qk_norm_rope(query, key, q_weight, k_weight, cos_sin, positions, *, eps: float = 1e-6, interleaved: bool = False,
                 query_out=None, key_out=None, stream=None):
    """pa_qk_norm_rope: RMS norm of every query and key head and position rotation.  Returns (query_out, key_out)."""
    dev, T, hq, hkv, d, query_out, qo, qos, q, qs, k, ks, rest = _rope_args(query, key, q_weight, k_weight, cos_sin,
                                                                            positions, query_out, stream)
    if key_out is None:
        key_out = _output(torch.empty, (T, hkv, d), key.device, stream)
    ko, kos = _rows(dev, key_out, "key_out", T, hkv, d)
    check("pa_qk_norm_rope", load().pa_qk_norm_rope(
        qo, ko, q, k, *rest, float(eps), qos, kos, qs, ks, cos_sin.size(1), 1 if interleaved else 0, cos_sin.size(0),
        T, hq, hkv, d, _raw_stream(stream, dev)))
    return query_out, key_out


def _rope_cache(name, extra, query, key, value, q_weight, k_weight, cos_sin, positions, slot_mapping, key_cache,
                value_cache, eps, interleaved, query_out, stream):
    dev, T, hq, hkv, d, query_out, qo, qos, q, qs, k, ks, rest = _rope_args(query, key, q_weight, k_weight, cos_sin,
                                                                            positions, query_out, stream)
    v, vs = _rows(dev, value, "value", T, hkv, d)
    if name == "pa_qk_norm_rope_cache_int4":
        kc, vc, nb, bs, heads = _int4_caches(dev, key_cache, value_cache, d)
        dim = d
    else:
        dtype = torch.uint8 if extra else torch.bfloat16
        kc, vc = _arr(dev, key_cache, dtype, "key_cache", 4), _arr(dev, value_cache, dtype, "value_cache", 4)
        nb, bs, heads, dim = key_cache.shape
        if value_cache.shape != key_cache.shape:
            raise ValueError("key_cache and value_cache shapes differ")
    if heads != hkv or dim != d:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_dim] matching the cache")
    sm = _arr(dev, slot_mapping, torch.int64, "slot_mapping", 1, T)
    check(name, getattr(load(), name)(
        qo, q, k, v, *rest, sm, kc, vc, float(eps), qos, qs, ks, vs, cos_sin.size(1), 1 if interleaved else 0,
        cos_sin.size(0), T, hq, hkv, d, bs, nb, *extra, _raw_stream(stream, dev)))
    return query_out


def qk_norm_rope_cache(query, key, value, q_weight, k_weight, cos_sin, positions, slot_mapping, key_cache,
                       value_cache, *, eps: float = 1e-6, interleaved: bool = False, query_out=None, stream=None):
    """pa_qk_norm_rope_cache: qk_norm_rope with the keys and values written to bf16 caches.  Returns query_out."""
    return _rope_cache("pa_qk_norm_rope_cache", (), query, key, value, q_weight, k_weight, cos_sin, positions,
                       slot_mapping, key_cache, value_cache, eps, interleaved, query_out, stream)


def qk_norm_rope_cache_fp8(query, key, value, q_weight, k_weight, cos_sin, positions, slot_mapping, key_cache,
                           value_cache, k_scale: float, v_scale: float, *, eps: float = 1e-6,
                           interleaved: bool = False, query_out=None, stream=None):
    """pa_qk_norm_rope_cache_fp8: as qk_norm_rope_cache into E4M3 code caches."""
    return _rope_cache("pa_qk_norm_rope_cache_fp8", (float(k_scale), float(v_scale)), query, key, value, q_weight,
                       k_weight, cos_sin, positions, slot_mapping, key_cache, value_cache, eps, interleaved,
                       query_out, stream)


def qk_norm_rope_cache_int4(query, key, value, q_weight, k_weight, cos_sin, positions, slot_mapping, key_cache,
                            value_cache, *, eps: float = 1e-6, interleaved: bool = False, query_out=None,
                            stream=None):
    """pa_qk_norm_rope_cache_int4: as qk_norm_rope_cache into 4-bit caches."""
    return _rope_cache("pa_qk_norm_rope_cache_int4", (), query, key, value, q_weight, k_weight, cos_sin, positions,
                       slot_mapping, key_cache, value_cache, eps, interleaved, query_out, stream)


# ---- a step's tables and slots --------------------------------------------------------

def prepare_batch(block_tables, context_lens, query_lens, free_blocks, num_free, block_size: int, num_blocks: int, *,
                  seq_lens, q_start, num_free_out, status, seq_ids=None, positions=None, slot_mapping=None,
                  num_tokens: int | None = None, stream=None) -> None:
    """pa_prepare_batch: new blocks, lengths, row starts, positions and slots of a ragged batch, on the device.

    The outputs are the caller's tensors.  The per-token arrays (seq_ids int32, positions and slot_mapping int64)
    are optional and of one length, the step's row capacity; num_tokens gives that capacity where none is passed."""
    dev = _device(block_tables, "block_tables")
    i32, i64 = torch.int32, torch.int64
    bt = _arr(dev, block_tables, i32, "block_tables", 2)
    B, n = block_tables.size(0), num_tokens
    if n is None:
        first = seq_ids if seq_ids is not None else positions if positions is not None else slot_mapping
        if first is None:
            raise ValueError("num_tokens is needed where no per-token array is passed")
        n = first.size(0)
    check("pa_prepare_batch", load().pa_prepare_batch(
        bt, _arr(dev, context_lens, i32, "context_lens", 1, B), _arr(dev, query_lens, i32, "query_lens", 1, B),
        _arr(dev, free_blocks, i32, "free_blocks", 1), _arr(dev, num_free, i32, "num_free", 1, 1),
        _arr(dev, seq_lens, i32, "seq_lens", 1, B), _arr(dev, q_start, i32, "q_start", 1, B + 1),
        _opt(dev, seq_ids, i32, "seq_ids", n), _opt(dev, positions, i64, "positions", n),
        _opt(dev, slot_mapping, i64, "slot_mapping", n), _arr(dev, num_free_out, i32, "num_free_out", 1, 1),
        _arr(dev, status, i32, "status", 1, 1), B, block_tables.size(1), int(n), free_blocks.size(0),
        int(block_size), int(num_blocks), _raw_stream(stream, dev)))


def release_blocks(block_tables, seq_lens, release, free_blocks, num_free, block_size: int, num_blocks: int, *,
                   status, stream=None) -> None:
    """pa_release_blocks: the blocks of the requests marked in `release` (int32) back on the free stack."""
    dev = _device(block_tables, "block_tables")
    i32 = torch.int32
    bt = _arr(dev, block_tables, i32, "block_tables", 2)
    B = block_tables.size(0)
    check("pa_release_blocks", load().pa_release_blocks(
        bt, _arr(dev, seq_lens, i32, "seq_lens", 1, B), _arr(dev, release, i32, "release", 1, B),
        _arr(dev, free_blocks, i32, "free_blocks", 1), _arr(dev, num_free, i32, "num_free", 1, 1),
        _arr(dev, status, i32, "status", 1, 1), B, block_tables.size(1), free_blocks.size(0), int(block_size), int(num_blocks),
        _raw_stream(stream, dev)))


# Bytes of the fixed scratch array inside the library (PA_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 16 << 20


def decode_split_noalloc(query, key_cache, value_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                         partition_size: int, *, out=None, stream=None):
    """pa_decode_split_noalloc: the split form with the library's own fixed scratch.

    For callers that cannot provide a workspace (see include/pagedkv.h).  Raises
    PagedKVError(PA_ERR_SCRATCH_TOO_SMALL) if the problem needs more than
    NOALLOC_SCRATCH_BYTES of split workspace.  Calls must not overlap on the GPU.
    """
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens)
    o, out = _out(out, query)
    check("pa_decode_split_noalloc", lib.pa_decode_split_noalloc(
        o, q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), bs, hkv, B, hq, d, mb, nb,
        int(max_seq_len), int(partition_size), _stream(stream)))
    return out


def decode_partitions(query, key_cache, value_cache, block_tables, seq_lens, scale: float, max_seq_len: int,
                      partition_size: int, workspace, stream=None):
    """pa_decode_partitions; returns views (o, m, l) into the workspace."""
    lib = load()
    q, bt, sl, B, hq, hkv, d, bs, nb, mb = _decode_common(query, key_cache, value_cache, block_tables, seq_lens)
    wp, wb = _ws(workspace)
    check("pa_decode_partitions", lib.pa_decode_partitions(
        q, key_cache.data_ptr(), value_cache.data_ptr(), bt, sl, float(scale), bs, hkv, B, hq, d, mb, nb,
        int(max_seq_len), int(partition_size), wp, wb, _stream(stream)))
    return workspace_views(workspace, B, hq, d, max_seq_len, partition_size)


def workspace_views(workspace, num_seqs, num_heads, head_dim, max_seq_len, partition_size):
    """(o, m, l) float32 views of a split-form workspace (layout of include/pagedkv.h)."""
    parts = max(1, -(-int(max_seq_len) // int(partition_size)))
    rows = num_seqs * num_heads * parts
    a256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
    raw = workspace.view(torch.uint8)[WORKSPACE_HEADER_BYTES:]
    ob = rows * head_dim * 4
    o = raw[:ob].view(torch.float32).view(num_seqs, num_heads, parts, head_dim)
    m = raw[a256(ob):a256(ob) + rows * 4].view(torch.float32).view(num_seqs, num_heads, parts)
    lo = a256(ob) + a256(rows * 4)
    l = raw[lo:lo + rows * 4].view(torch.float32).view(num_seqs, num_heads, parts)
    return o, m, l


def new_workspace(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, max_seq_len: int,
                  partition_size: int = 0, device="cuda"):
    """A zero-filled decode workspace (the scheduler counters must start at zero)."""
    nbytes = decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, max_seq_len, partition_size)
    return torch.zeros(max(nbytes, WORKSPACE_HEADER_BYTES), dtype=torch.uint8, device=device)


def lse_reduce(out, workspace, seq_lens, max_seq_len: int, partition_size: int, stream=None):
    lib = load()
    o = _dev(out, torch.bfloat16, "out", 3)
    B, hq, d = out.shape
    wp, _ = _ws(workspace)
    check("pa_lse_reduce", lib.pa_lse_reduce(o, wp, _dev(seq_lens, torch.int32, "seq_lens", 1), B, hq, d,
                                             int(max_seq_len), int(partition_size), _stream(stream)))
    return out


def validate_tables(block_tables, seq_lens, block_size: int, num_blocks: int, max_seq_len: int,
                    stream=None) -> int:
    """Number of sequences breaking a decode precondition (synchronises)."""
    lib = load()
    bad = torch.zeros(1, dtype=torch.int32, device=block_tables.device)
    check("pa_validate_tables", lib.pa_validate_tables(
        _dev(block_tables, torch.int32, "block_tables", 2), _dev(seq_lens, torch.int32, "seq_lens", 1),
        block_tables.shape[0], block_tables.shape[1], int(block_size), int(num_blocks), int(max_seq_len),
        bad.data_ptr(), _stream(stream)))
    return int(bad.item())


def selftest_bounded_wait(stream=None) -> None:
    """Launch one device wait that nothing satisfies; it gives up after about a
    second and leaves PA_ERR_DEVICE_TIMEOUT for device_status() to report."""
    check("pa_selftest_bounded_wait", load().pa_selftest_bounded_wait(_stream(stream)))


def device_status() -> int:
    """0, or a negative status: PA_ERR_DEVICE_TIMEOUT (-9) if a bounded device wait
    gave up, PA_ERR_VALUE_RANGE (-12) if the prefill read a value entry beyond the
    fp16 range of its P.V operand, PA_ERR_BAD_BLOCK (-7) if decode_int4 met a table
    entry outside the cache.  Reading clears it."""
    return int(load().pa_device_status())

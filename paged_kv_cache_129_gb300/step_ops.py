"""A serving step over a paged cache: block tables and slot maps built on the GPU, rotary positions fused with
the paged write, and causal attention of ragged runs of new tokens over an FP8 cache.

Argument marshalling for the calls of that name in ``include/pa.h``; like the rest of the binding it computes
nothing itself.  Tensors of one call live on one device, which need not be the current one; ``stream`` defaults to
that device's current stream.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch

from .binding import _check, _cuda, _dtype_code, _fp8_cache, _need, _stream_ptr, _TORCH_DTYPES, library

LAYOUTS = {"half": 0, "interleaved": 1}


class TableStep(NamedTuple):
    """What ``advance_tables`` leaves for the calls of its step."""

    context_lens: torch.Tensor  # int32 [B], new tokens included
    num_free: torch.Tensor  # int32 [1]
    q_offsets: torch.Tensor  # int32 [B + 1]
    positions: torch.Tensor  # int32 [num_tokens]
    slot_mapping: torch.Tensor  # int64 [num_tokens]


def _one_device(device: torch.device, *tensors) -> None:
    index = device.index
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors of a call must be on one device")


def _int32(t: torch.Tensor, name: str) -> None:
    _cuda(t, name)
    if t.dtype is not torch.int32:
        raise ValueError(f"{name} must be int32")


def _fresh(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """A new tensor for a call on ``stream``: the allocator must not hand its memory to another stream's
    tensor while the call is in flight."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        t.record_stream(stream)
    return t


def _launch(fn, device: torch.device, stream, *args) -> None:
    """One library call on ``device``, on ``stream`` or the device's current stream."""
    index = device.index
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_ptr(stream, device)
    if index == torch._C._cuda_getDevice():
        _check(fn(*args, raw))
    else:
        with torch.cuda.device(device):
            _check(fn(*args, raw))


def advance_tables(block_tables: torch.Tensor, context_lens: torch.Tensor, new_lens: torch.Tensor,
                   free_blocks: torch.Tensor, num_free: torch.Tensor, block_size: int, num_tokens: int,
                   out: Optional[TableStep] = None, stream=None) -> TableStep:
    """``pa_advance_tables``: a step's block tables, lengths, positions and slots from the requests' lengths.

    ``block_tables`` int32 [B, max_blocks] (updated), ``context_lens`` and ``new_lens`` int32 [B] (a negative
    ``new_lens[b]`` ends request b and gives its blocks back), ``free_blocks`` int32 [num_blocks], a stack of
    ``num_free[0]`` ids (updated above its count by blocks given back).  ``num_tokens`` is a bound of the new tokens:
    rows past the last one get slot -1.  ``out``: five tensors as ``TableStep`` to write to; its ``context_lens`` and
    ``num_free`` may be the inputs.
    """
    for name, t in (("block_tables", block_tables), ("context_lens", context_lens), ("new_lens", new_lens),
                    ("free_blocks", free_blocks), ("num_free", num_free)):
        _int32(t, name)
    _need(block_tables.dim() == 2, "block_tables: int32 [B, max_blocks]")
    b, width = block_tables.shape
    dev = block_tables.device
    _need(context_lens.shape == (b,) and new_lens.shape == (b,), "context_lens / new_lens: int32 [B]")
    _need(free_blocks.dim() == 1 and num_free.numel() == 1, "free_blocks: int32 [num_blocks], num_free: int32 [1]")
    num_tokens = int(num_tokens)
    _need(num_tokens >= 0, "num_tokens must not be negative")
    if out is None:
        out = TableStep(_fresh(b, torch.int32, dev, stream), _fresh(1, torch.int32, dev, stream),
                        _fresh(b + 1, torch.int32, dev, stream), _fresh(num_tokens, torch.int32, dev, stream),
                        _fresh(num_tokens, torch.int64, dev, stream))
    else:
        out = TableStep(*out)
        for t, n, dt in zip(out, (b, 1, b + 1, num_tokens, num_tokens), (torch.int32,) * 4 + (torch.int64,)):
            _cuda(t, "out")
            if t.dtype is not dt or t.numel() != n:
                raise ValueError(f"out: {n} elements of {dt}")
    _one_device(dev, context_lens, new_lens, free_blocks, num_free, *out)
    _launch(library().pa_advance_tables, dev, stream, block_tables.data_ptr(), context_lens.data_ptr(), new_lens.data_ptr(),
            free_blocks.data_ptr(), num_free.data_ptr(), *[t.data_ptr() for t in out], b, width, free_blocks.numel(),
            int(block_size), num_tokens)
    return out


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     context: int = 0, low: float = 1.0, high: float = 32.0, device=None) -> torch.Tensor:
    """Angles per position of the ``rotary_dim / 2`` pairs, float64: ``base ** (-2i / rotary_dim)``, for contexts
    ``factor`` times longer by

    * ``"linear"``: every angle divided by ``factor``;
    * ``"base"``: the base multiplied by ``factor ** (r / (r - 2))``, so that the slowest pair is divided by ``factor``
      and the fastest not at all;
    * ``"ramp"``: pairs that turn less than ``low`` times over the trained ``context`` divided by ``factor``, those that
      turn more than ``high`` times kept, and a blend, linear in the number of turns, between.
    """
    _need(rotary_dim >= 2 and rotary_dim % 2 == 0, "rotary_dim must be even and positive")
    _need(base > 0 and factor > 0, "base and factor must be positive")
    r = rotary_dim
    if scaling == "base":
        _need(r > 2, "scaling the base needs rotary_dim > 2")
        base = base * factor ** (r / (r - 2))
    inv = torch.pow(torch.tensor(float(base), dtype=torch.float64), -torch.arange(0, r, 2, dtype=torch.float64) / r)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "ramp":
        _need(context > 0 and high > low, "ramp scaling needs the trained context and low < high")
        keep = ((context * inv / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        inv = inv * keep + inv / factor * (1.0 - keep)
    else:
        _need(scaling in ("none", "base"), f"unknown scaling {scaling!r}")
    return inv.to(device) if device is not None else inv


def _rows(t: torch.Tensor, name: str, d: int) -> int:
    """Checks [T, heads, d] rows with contiguous heads; returns the stride between tokens."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"{name} must be [T, heads, {d}]")
    tokens, heads, _ = shape
    if stride[2] != 1 or (heads != 1 and stride[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if tokens <= 1:
        return heads * d
    if stride[0] < heads * d:
        raise ValueError(f"{name}: tokens must not overlap")
    return stride[0]


def _rope_inputs(query, key, value, inv_freq, layout, query_out, hkv, d, stream):
    """Shared checks of the rotary calls; returns (query_out, token strides, rotary_dim, layout code)."""
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    strides = _rows(query, "query", d), _rows(key, "key", d), _rows(value, "value", d)
    t = query.shape[0]
    _need(key.shape == (t, hkv, d) and value.shape == key.shape, "key/value must be [T, H_kv, d]")
    _need(query.dtype == key.dtype == value.dtype, "query, key and value must share a dtype")
    rotary_dim = 0
    if inv_freq is not None:
        _cuda(inv_freq, "inv_freq")
        _need(inv_freq.dtype == torch.float64 and inv_freq.dim() == 1, "inv_freq: float64 [rotary_dim / 2]")
        rotary_dim = 2 * inv_freq.shape[0]
    if query_out is None:
        query_out = _fresh(tuple(query.shape), query.dtype, query.device, stream)
    _cuda(query_out, "query_out")
    _need(query_out.shape == query.shape and query_out.dtype == query.dtype, "query_out must match query")
    return query_out, strides, rotary_dim, LAYOUTS[layout]


def rope_write_kv(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                  value_cache: torch.Tensor, inv_freq: torch.Tensor, positions: torch.Tensor, slot_mapping: torch.Tensor,
                  layout: str = "half", factor: float = 1.0, query_out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """``pa_rope_write_kv``: turns query ``[T, H_q, d]`` and key ``[T, H_kv, d]`` by their positions and writes keys and
    values to ``slot_mapping`` (as ``write_kv``), in one launch; returns the turned queries.

    ``inv_freq`` (float64, ``rope_frequencies``) gives the angle per position of the first ``2 * len(inv_freq)`` elements
    of a head, paired ``"half"`` (i with i + r / 2) or ``"interleaved"`` (2i with 2i + 1); ``factor`` multiplies the turned
    elements.  query, key and value may be views with a stride between tokens.
    """
    for name, t in (("key_cache", key_cache), ("value_cache", value_cache), ("positions", positions),
                    ("slot_mapping", slot_mapping)):
        _cuda(t, name)
    _need(key_cache.dim() == 4 and value_cache.shape == key_cache.shape, "caches must be [N, H_kv, bs, d]")
    num_blocks, hkv, bs, d = key_cache.shape
    _need(inv_freq is not None, "inv_freq: float64 [rotary_dim / 2]")
    query_out, strides, rot, code = _rope_inputs(query, key, value, inv_freq, layout, query_out, hkv, d, stream)
    t = query.shape[0]
    _need(query.dtype == key_cache.dtype == value_cache.dtype, "query, key, value and caches must share a dtype")
    _need(positions.dtype == torch.int32 and positions.shape == (t,), "positions: int32 [T]")
    _need(slot_mapping.dtype == torch.int64 and slot_mapping.shape == (t,), "slot_mapping: int64 [T]")
    dev = key_cache.device
    _one_device(dev, query, key, value, value_cache, inv_freq, positions, slot_mapping, query_out)
    _launch(library().pa_rope_write_kv, dev, stream, query_out.data_ptr(), query.data_ptr(), key.data_ptr(), value.data_ptr(),
            key_cache.data_ptr(), value_cache.data_ptr(), inv_freq.data_ptr(), positions.data_ptr(), slot_mapping.data_ptr(),
            *strides, t, query.shape[1], hkv, d, rot, code, float(factor), bs, num_blocks, _dtype_code(query))
    return query_out


def _runs(block_tables, context_lens, q_offsets) -> None:
    for name, t in (("block_tables", block_tables), ("context_lens", context_lens), ("q_offsets", q_offsets)):
        _int32(t, name)
    _need(block_tables.dim() == 2, "block_tables: int32 [B, max_blocks]")
    b = block_tables.shape[0]
    _need(context_lens.numel() == b, "context_lens: int32 [B]")
    _need(q_offsets.numel() == b + 1, "q_offsets: int32 [B + 1]")


def rope_append_fp8(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                    value_cache: Optional[torch.Tensor], k_scale: torch.Tensor, v_scale: torch.Tensor,
                    inv_freq: Optional[torch.Tensor], block_tables: torch.Tensor, context_lens: torch.Tensor,
                    q_offsets: torch.Tensor, layout: str = "half", factor: float = 1.0,
                    query_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``pa_rope_append_fp8``: turns queries and keys as ``rope_write_kv`` and appends keys and values to an FP8 cache whose
    block scales follow the data (a block's scale grows with its largest magnitude, and the codes it holds with it).

    Request b's new tokens are rows ``q_offsets[b]`` to ``q_offsets[b + 1]``, the last positions of its ``context_lens[b]``
    tokens.  ``inv_freq`` None: no rotation.  ``value_cache`` None: K and V records.  Returns the turned queries.
    """
    num_blocks, hkv, bs, d = _fp8_cache(key_cache, value_cache, k_scale, v_scale)
    query_out, strides, rot, code = _rope_inputs(query, key, value, inv_freq, layout, query_out, hkv, d, stream)
    _runs(block_tables, context_lens, q_offsets)
    dev = key_cache.device
    _one_device(dev, query, key, value, value_cache, k_scale, v_scale, inv_freq, block_tables, context_lens, q_offsets,
                query_out)
    _launch(library().pa_rope_append_fp8, dev, stream, query_out.data_ptr(), query.data_ptr(), key.data_ptr(),
            value.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr() if value_cache is not None else None,
            k_scale.data_ptr(), v_scale.data_ptr(), inv_freq.data_ptr() if rot else None, block_tables.data_ptr(),
            context_lens.data_ptr(), q_offsets.data_ptr(), *strides, block_tables.shape[0], query.shape[0], query.shape[1],
            hkv, d, rot, code, float(factor), bs, block_tables.shape[1], num_blocks, _dtype_code(query))
    return query_out


def attend_fp8_workspace_size(num_tokens: int, num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              block_size: int, max_blocks_per_seq: int, dtype: torch.dtype) -> int:
    """Bytes of scratch that ``attend_fp8`` wants for these sizes, on the current device."""
    return int(library().pa_attend_fp8_workspace_size(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                      max_blocks_per_seq, _TORCH_DTYPES[dtype]))


def attend_fp8(query: torch.Tensor, key_cache: torch.Tensor, value_cache: Optional[torch.Tensor], k_scale: torch.Tensor,
               v_scale: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, q_offsets: torch.Tensor,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``pa_attend_fp8``: query ``[T, H_q, d]`` (f16/bf16) holds each request's last ``q_offsets[b + 1] - q_offsets[b]``
    positions; each row attends its request's positions up to its own over the E4M3 cache (``value_cache`` None: K and V
    records).  Rows behind ``q_offsets[B]`` of ``out`` are left as they were.  ``workspace`` defaults to a fresh one.
    For one token of every request and no longer run, ``decode_fp8`` takes less than half the time.
    """
    num_blocks, hkv, bs, d = _fp8_cache(key_cache, value_cache, k_scale, v_scale)
    _cuda(query, "query")
    _need(query.dim() == 3 and query.shape[2] == d, "query must be [T, H_q, d]")
    _runs(block_tables, context_lens, q_offsets)
    dev = key_cache.device
    t, hq, _ = query.shape
    if out is None:
        out = _fresh(tuple(query.shape), query.dtype, dev, stream)
    _cuda(out, "out")
    _need(out.shape == query.shape and out.dtype == query.dtype, "out must match query")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    b, width = block_tables.shape
    code = _dtype_code(query)
    if workspace is None:
        size_of = library().pa_attend_fp8_workspace_size
        if dev.index == torch._C._cuda_getDevice():
            need = size_of(t, b, hq, hkv, d, bs, width, code)
        else:
            with torch.cuda.device(dev):
                need = size_of(t, b, hq, hkv, d, bs, width, code)
        workspace = _fresh(max(int(need), 256), torch.uint8, dev, stream)
    _cuda(workspace, "workspace")
    _one_device(dev, query, value_cache, k_scale, v_scale, block_tables, context_lens, q_offsets, out, workspace)
    _launch(library().pa_attend_fp8, dev, stream, out.data_ptr(), query.data_ptr(), key_cache.data_ptr(),
            value_cache.data_ptr() if value_cache is not None else None, k_scale.data_ptr(), v_scale.data_ptr(),
            block_tables.data_ptr(), context_lens.data_ptr(), q_offsets.data_ptr(), b, t, hq, hkv, d, bs, width, num_blocks,
            float(scale), code, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out

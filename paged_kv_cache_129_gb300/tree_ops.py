"""A speculative step with a drafted tree over a paged cache: masks and positions from parent indices, norms fused with
the rotary write, attention of the nodes, greedy acceptance, and the accepted branch compacted in every layer.

Argument marshalling for the calls of that name in ``include/pa.h``; like the rest of the binding it computes
nothing itself.  Tensors of one call live on one device, which need not be the current one; ``stream`` defaults to
that device's current stream.
"""
from __future__ import annotations

import math
from array import array
from typing import NamedTuple, Optional

import torch

from .binding import _cuda, _dtype_code, _need, _TORCH_DTYPES, library
from .step_ops import _fresh, _int32, _launch, _one_device, _rope_inputs, _runs

MAX_TREE_NODES = 1024  # of one request


class TreeMasks(NamedTuple):
    """What ``tree_masks`` leaves for the calls of its step."""

    positions: torch.Tensor  # int32 [T]
    tree_mask: torch.Tensor  # int64 [T, words]


class TreePath(NamedTuple):
    """The branch that ``accept_tree`` found."""

    accepted: torch.Tensor  # int32 [B, max_accepted], -1 behind the last node
    num_accepted: torch.Tensor  # int32 [B]
    next_tokens: torch.Tensor  # [B], of the tokens' dtype


class TreeState(NamedTuple):
    """What ``compact_tree`` leaves for the next step."""

    context_lens: torch.Tensor  # int32 [B]
    num_free: torch.Tensor  # int32 [1]


def _int32s(names: str, *tensors) -> None:
    """``_int32`` of several tensors, named only where one is none: these checks are much of a small call's time."""
    for t in tensors:
        if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
            for name, x in zip(names.split(), tensors):
                _int32(x, name)


def _outputs(out, kind, wanted, device, stream):
    """The outputs of a call: fresh ones, or the given ones if they have these shapes and dtypes."""
    if out is None:
        return kind(*[_fresh(shape, dtype, device, stream) for shape, dtype in wanted])
    if type(out) is not kind:
        out = kind(*out)
    for t, (shape, dtype) in zip(out, wanted):
        if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
            _cuda(t, "out")
            raise ValueError(f"out: {list(shape)} of {dtype}")
    return out


def _nodes(parents: torch.Tensor, q_offsets: torch.Tensor) -> tuple:
    _int32s("parents q_offsets", parents, q_offsets)
    if parents.dim() != 1 or q_offsets.dim() != 1 or q_offsets.shape[0] < 1:
        raise ValueError("parents: int32 [T], q_offsets: int32 [B + 1]")
    return parents.shape[0], q_offsets.shape[0] - 1


def tree_masks(parents: torch.Tensor, context_lens: torch.Tensor, q_offsets: torch.Tensor, mask_words: int,
               out: Optional[TreeMasks] = None, stream=None) -> TreeMasks:
    """``pa_tree_masks``: for the nodes of each request's tree (rows ``q_offsets[b]`` to ``q_offsets[b + 1]``; ``parents``
    int32 [T], a node's parent among its request's nodes, before it, or -1), the nodes that each sees, itself and its
    ancestors, as bits of ``mask_words`` int64 words, and its position.  ``context_lens`` counts the nodes.
    """
    t, b = _nodes(parents, q_offsets)
    _int32(context_lens, "context_lens")
    _need(context_lens.shape == (b,), "context_lens: int32 [B]")
    dev, words = parents.device, int(mask_words)
    _need(1 <= words <= MAX_TREE_NODES // 64, "mask_words must be 1 to 16")
    out = _outputs(out, TreeMasks, (((t,), torch.int32), ((t, words), torch.int64)), dev, stream)
    _one_device(dev, context_lens, q_offsets, *out)
    _launch(library().pa_tree_masks, dev, stream, out.positions.data_ptr(), out.tree_mask.data_ptr(), parents.data_ptr(),
            context_lens.data_ptr(), q_offsets.data_ptr(), b, t, words)
    return out


def norm_rope_write_kv(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor, key_cache: torch.Tensor,
                       value_cache: torch.Tensor, q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                       inv_freq: Optional[torch.Tensor], positions: torch.Tensor, slot_mapping: torch.Tensor, eps: float = 1e-6,
                       weight_offset: float = 0.0, layout: str = "half", factor: float = 1.0,
                       query_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``pa_norm_rope_write_kv``: ``rope_write_kv`` with every query and key head divided by its root mean square and
    multiplied by ``q_weight + weight_offset`` or ``k_weight + weight_offset`` ([d], float32 or the queries' dtype; None:
    the norm alone) before its rotation, in the same pass.  ``inv_freq`` None: no rotation.  Returns the queries.
    """
    _cuda(key_cache, "key_cache")
    _cuda(value_cache, "value_cache")
    _cuda(positions, "positions")
    _cuda(slot_mapping, "slot_mapping")
    shape, dtype = key_cache.shape, query.dtype
    if len(shape) != 4 or value_cache.shape != shape:
        raise ValueError("caches must be [N, H_kv, bs, d]")
    num_blocks, hkv, bs, d = shape
    query_out, strides, rot, code = _rope_inputs(query, key, value, inv_freq, layout, query_out, hkv, d, stream)
    t = query.shape[0]
    if key_cache.dtype is not dtype or value_cache.dtype is not dtype:
        raise ValueError("query, key, value and caches must share a dtype")
    if positions.dtype is not torch.int32 or positions.shape != (t,):
        raise ValueError("positions: int32 [T]")
    if slot_mapping.dtype is not torch.int64 or slot_mapping.shape != (t,):
        raise ValueError("slot_mapping: int64 [T]")
    weight_dtype = None
    for w in (q_weight, k_weight):
        if w is None:
            continue
        _cuda(w, "weights")
        if w.shape != (d,) or (w.dtype is not torch.float32 and w.dtype is not dtype) or weight_dtype not in (None, w.dtype):
            raise ValueError("weights: [d], float32 or the queries' dtype, the same for both")
        weight_dtype = w.dtype
    dev = key_cache.device
    _one_device(dev, query, key, value, value_cache, q_weight, k_weight, inv_freq, positions, slot_mapping, query_out)
    _launch(library().pa_norm_rope_write_kv, dev, stream, query_out.data_ptr(), query.data_ptr(), key.data_ptr(),
            value.data_ptr(), key_cache.data_ptr(), value_cache.data_ptr(), None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), inv_freq.data_ptr() if rot else None, positions.data_ptr(),
            slot_mapping.data_ptr(), *strides, t, query.shape[1], hkv, d, rot, code, float(factor), float(eps),
            float(weight_offset), _TORCH_DTYPES.get(weight_dtype, 0), bs, num_blocks, _dtype_code(query))
    return query_out


def attend_tree_workspace_size(num_tokens: int, num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                               block_size: int, max_blocks_per_seq: int, dtype: torch.dtype) -> int:
    """Bytes of scratch that ``attend_tree`` wants for these sizes, on the current device."""
    return int(library().pa_attend_tree_workspace_size(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                       max_blocks_per_seq, _TORCH_DTYPES[dtype]))


def attend_tree(query: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor, tree_mask: torch.Tensor,
                block_tables: torch.Tensor, context_lens: torch.Tensor, q_offsets: torch.Tensor, scale: Optional[float] = None,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``pa_attend_tree``: query ``[T, H_q, d]`` (f16/bf16) holds the nodes of each request, the last
    ``q_offsets[b + 1] - q_offsets[b]`` of its ``context_lens[b]`` positions; each row attends the positions before the
    nodes, and the nodes whose bits its row of ``tree_mask`` (int64 [T, words]) has, over the cache ``[N, H_kv, bs, d]`` of
    the same dtype.  A row that sees nothing gets zeros; rows behind ``q_offsets[B]`` of ``out`` are left as they were.
    ``workspace`` defaults to a fresh one.
    """
    for name, t in (("query", query), ("key_cache", key_cache), ("value_cache", value_cache), ("tree_mask", tree_mask)):
        _cuda(t, name)
    _need(key_cache.dim() == 4 and value_cache.shape == key_cache.shape, "caches must be [N, H_kv, bs, d]")
    num_blocks, hkv, bs, d = key_cache.shape
    _need(query.dim() == 3 and query.shape[2] == d, "query must be [T, H_q, d]")
    _need(query.dtype == key_cache.dtype == value_cache.dtype, "query and caches must share a dtype")
    _runs(block_tables, context_lens, q_offsets)
    t, hq, _ = query.shape
    _need(tree_mask.dtype == torch.int64 and tree_mask.dim() == 2 and tree_mask.shape[0] == t, "tree_mask: int64 [T, words]")
    dev = key_cache.device
    if out is None:
        out = _fresh(tuple(query.shape), query.dtype, dev, stream)
    _cuda(out, "out")
    _need(out.shape == query.shape and out.dtype == query.dtype, "out must match query")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    b, width = block_tables.shape
    code = _dtype_code(query)
    if workspace is None:
        size_of = library().pa_attend_tree_workspace_size
        if dev.index == torch._C._cuda_getDevice():
            need = size_of(t, b, hq, hkv, d, bs, width, code)
        else:
            with torch.cuda.device(dev):
                need = size_of(t, b, hq, hkv, d, bs, width, code)
        workspace = _fresh(max(int(need), 256), torch.uint8, dev, stream)
    _cuda(workspace, "workspace")
    _one_device(dev, query, value_cache, tree_mask, block_tables, context_lens, q_offsets, out, workspace)
    _launch(library().pa_attend_tree, dev, stream, out.data_ptr(), query.data_ptr(), key_cache.data_ptr(),
            value_cache.data_ptr(), tree_mask.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(),
            q_offsets.data_ptr(), b, t, hq, hkv, d, bs, width, num_blocks, tree_mask.shape[1], float(scale), code,
            workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def accept_tree(parents: torch.Tensor, tokens: torch.Tensor, choices: torch.Tensor, q_offsets: torch.Tensor,
                max_accepted: int, out: Optional[TreePath] = None, stream=None) -> TreePath:
    """``pa_accept_tree``: from each request's node 0 on to the first child whose token (``tokens`` [T]) is the target's
    choice at the node (``choices`` [T]; int32 or int64, as ``tokens``), up to ``max_accepted`` nodes; and the choice at the last one.
    """
    t, b = _nodes(parents, q_offsets)
    _cuda(tokens, "tokens")
    _cuda(choices, "choices")
    dtype = tokens.dtype
    if (dtype is not torch.int64 and dtype is not torch.int32) or choices.dtype is not dtype or tokens.shape != (t,) or choices.shape != (t,):
        raise ValueError("tokens and choices: int32 or int64 [T], of one dtype")
    dev, depth = parents.device, int(max_accepted)
    _need(1 <= depth <= MAX_TREE_NODES, "max_accepted must be 1 to 1024")
    out = _outputs(out, TreePath, (((b, depth), torch.int32), ((b,), torch.int32), ((b,), dtype)), dev, stream)
    _one_device(dev, tokens, choices, q_offsets, *out)
    _launch(library().pa_accept_tree, dev, stream, out.accepted.data_ptr(), out.num_accepted.data_ptr(),
            out.next_tokens.data_ptr(), parents.data_ptr(), tokens.data_ptr(), choices.data_ptr(), q_offsets.data_ptr(), b, t,
            depth, tokens.element_size())
    return out


def _layer_pointers(caches, name: str):
    """(addresses of the layers' caches, shape, dtype, device): one [L, N, H_kv, bs, d] tensor, or a sequence of [N, H_kv, bs, d]."""
    if isinstance(caches, torch.Tensor):
        _cuda(caches, name)
        shape = caches.shape
        if len(shape) != 5 or shape[0] < 1:
            raise ValueError(f"{name}: [layers, N, H_kv, bs, d], or a sequence of [N, H_kv, bs, d]")
        first, step = caches.data_ptr(), caches.stride(0) * caches.element_size()
        # (a layer without elements has no stride to speak of: the library refuses its sizes)
        return array("Q", range(first, first + shape[0] * step, step) if step else [first] * shape[0]), shape[1:], caches.dtype, caches.device
    _need(len(caches) >= 1, f"{name}: a cache per layer")
    like = caches[0]
    for c in caches:
        _cuda(c, name)
        if c.dim() != 4 or c.shape != like.shape or c.dtype is not like.dtype or c.device != like.device:
            raise ValueError(f"{name}: caches [N, H_kv, bs, d] of one shape, dtype and device")
    return array("Q", [c.data_ptr() for c in caches]), like.shape, like.dtype, like.device


def compact_tree(key_caches, value_caches, slot_mapping: torch.Tensor, q_offsets: torch.Tensor, accepted: torch.Tensor,
                 num_accepted: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor, free_blocks: torch.Tensor,
                 num_free: torch.Tensor, out: Optional[TreeState] = None, stream=None) -> TreeState:
    """``pa_compact_tree``: moves the accepted nodes (``accepted`` int32 [B, depth], ascending, ``num_accepted`` [B] of them) to
    the places behind the request's cached positions in every layer's caches (one tensor [layers, N, H_kv, bs, d], or a sequence of
    [N, H_kv, bs, d] tensors, each for keys and values; a cache that layers share is listed once), shortens the requests to them and gives the blocks behind back to ``free_blocks``.
    ``slot_mapping`` and ``q_offsets`` are ``advance_tables``'.  ``out``: two tensors as ``TreeState`` to write to, which may be
    ``context_lens`` and ``num_free``.
    """
    keys, shape, dtype, dev = _layer_pointers(key_caches, "key_caches")
    values, vshape, vdtype, vdev = _layer_pointers(value_caches, "value_caches")
    if len(keys) != len(values) or shape != vshape or dtype is not vdtype or dev != vdev:
        raise ValueError("key_caches and value_caches must match")
    if dtype is not torch.bfloat16 and dtype is not torch.float16 and dtype is not torch.float32:
        raise ValueError("caches: float32, float16 or bfloat16")
    num_blocks, hkv, bs, d = shape
    _int32s("q_offsets accepted num_accepted block_tables context_lens free_blocks num_free", q_offsets, accepted, num_accepted,
            block_tables, context_lens, free_blocks, num_free)
    _cuda(slot_mapping, "slot_mapping")
    if slot_mapping.dtype is not torch.int64 or slot_mapping.dim() != 1:
        raise ValueError("slot_mapping: int64 [T]")
    if block_tables.dim() != 2 or accepted.dim() != 2:
        raise ValueError("block_tables: int32 [B, max_blocks], accepted: int32 [B, depth]")
    b, width = block_tables.shape
    if accepted.shape[0] != b or num_accepted.shape != (b,) or context_lens.shape != (b,) or q_offsets.shape != (b + 1,):
        raise ValueError("accepted [B, depth], num_accepted and context_lens [B], q_offsets [B + 1]")
    if free_blocks.shape != (num_blocks,) or num_free.numel() != 1:
        raise ValueError("free_blocks: int32 [num_blocks], num_free: int32 [1]")
    out = _outputs(out, TreeState, (((b,), torch.int32), (tuple(num_free.shape), torch.int32)), dev, stream)
    _one_device(dev, slot_mapping, q_offsets, accepted, num_accepted, block_tables, context_lens, free_blocks, num_free, *out)
    _launch(library().pa_compact_tree, dev, stream, keys.buffer_info()[0], values.buffer_info()[0], len(keys), slot_mapping.data_ptr(), q_offsets.data_ptr(),
            accepted.data_ptr(), num_accepted.data_ptr(), block_tables.data_ptr(), context_lens.data_ptr(), free_blocks.data_ptr(),
            num_free.data_ptr(), out.context_lens.data_ptr(), out.num_free.data_ptr(), b, slot_mapping.shape[0], accepted.shape[1],
            hkv, d, bs, width, num_blocks, _TORCH_DTYPES[dtype])
    return out

"""Binding of the operators of a drafted (speculative) step: block tables and slot maps from
request lengths, rotary positions with the cache write, tree attention, acceptance.

As the rest of the binding, each function checks devices, types, shapes and contiguity, and
forwards pointers to the library on torch's current stream of the tensors' device. Everything
stays on the GPU: no call synchronises, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

from typing import Optional, Sequence

from . import (PARTITION_AUTO, PA_ERR_WORKSPACE, PA_OK, PagedAttnError, _dtype_code, _lib, _torch,
               pa_decode_desc, pa_rotary_desc)


def _refuse(x, name, dtype, dev, shape):
    if x.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    if x.dtype is not dtype:
        raise TypeError(f"{name} has dtype {x.dtype}, expected {dtype}")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(x, name, dtype, dev, shape=None):
    """Device pointer of a contiguous tensor of this type (and shape) on device ``dev``."""
    if x.get_device() != dev or x.dtype is not dtype or not x.is_contiguous() or \
            (shape is not None and x.shape != shape):
        _refuse(x, name, dtype, dev, shape)
    return x.data_ptr()


def _opt(x, name, dtype, dev, shape=None):
    return None if x is None else _ptr(x, name, dtype, dev, shape)


def _launch(fn, what: str, dev: int, stream, args) -> None:
    """Calls a library function on device ``dev``, with ``stream`` or that device's current
    stream as its last argument."""
    torch = _torch()
    if stream is None:
        # the handle alone: a Stream object would cost more than the launch's other checks
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError("stream belongs to another device than the tensors")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != PA_OK:
        raise PagedAttnError(st, what)


def _device(x, name) -> int:
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros, v_zeros, dev):
    """(cache dtype code, pointers of the pools, pointers of scales and zero points)."""
    torch = _torch()
    shape, dt = k_cache.shape, k_cache.dtype
    if len(shape) != 4:
        raise ValueError("the caches must be [num_blocks, num_kv_heads, B, d]")
    pools = _ptr(k_cache, "k_cache", dt, dev), _ptr(v_cache, "v_cache", dt, dev, shape)
    if k_scales is v_scales is k_zeros is v_zeros is None:
        return _dtype_code(dt), pools, (None, None, None, None)
    bh, f32, i32 = shape[:2], torch.float32, torch.int32
    return _dtype_code(dt), pools, (
        _opt(k_scales, "k_scales", f32, dev, bh), _opt(v_scales, "v_scales", f32, dev, bh),
        _opt(k_zeros, "k_zeros", i32, dev, bh), _opt(v_zeros, "v_zeros", i32, dev, bh))


def build_step(context_lens, new_lens, blocks_held, block_tables, free_blocks, queue_state, *,
               block_size: int, num_blocks: int, total_lens, query_start, blocks_held_out,
               queue_state_out, slot_mapping, positions=None, parents=None, tree_mask=None,
               status=None, stream=None) -> None:
    """A step's block tables, slot map, positions and ancestor masks from request lengths.

    Sequence s has context_lens[s] cached tokens in blocks_held[s] blocks and brings
    new_lens[s] tokens; the blocks it lacks are taken, in sequence order, from the front of
    the free queue: ``free_blocks`` is a ring, ``queue_state`` its [front index, count].
    All int32 CUDA tensors. Outputs, none of which may overlap another buffer: total_lens [S],
    query_start [S + 1], blocks_held_out [S], queue_state_out [2], slot_mapping int64 [rows]
    (-1 behind the last sequence), positions [rows] (context + number of ancestors), tree_mask
    [rows, words] (bit j % 32 of word j / 32: the row sees row j of its sequence), status [1]
    (0, or the PA_DEVERR_* bits for which the step was refused as a whole). block_tables gets
    the new entries. ``parents`` [rows]: index within the sequence of each row's parent, -1
    for none; without it rows form a chain.
    """
    torch = _torch()
    i32, dev = torch.int32, _device(context_lens, "context_lens")
    S, rows = context_lens.shape[0], slot_mapping.shape[0]
    words = 0 if tree_mask is None else tree_mask.shape[-1]
    if block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [S, max_blocks]")
    args = (
        _ptr(context_lens, "context_lens", i32, dev, (S,)),
        _ptr(new_lens, "new_lens", i32, dev, (S,)),
        _ptr(blocks_held, "blocks_held", i32, dev, (S,)),
        _opt(parents, "parents", i32, dev, (rows,)),
        _ptr(block_tables, "block_tables", i32, dev), _ptr(free_blocks, "free_blocks", i32, dev),
        _ptr(queue_state, "queue_state", i32, dev, (2,)), S, block_tables.shape[1], block_size,
        num_blocks, free_blocks.numel(), rows, words,
        _ptr(total_lens, "total_lens", i32, dev, (S,)),
        _ptr(query_start, "query_start", i32, dev, (S + 1,)),
        _ptr(blocks_held_out, "blocks_held_out", i32, dev, (S,)),
        _ptr(queue_state_out, "queue_state_out", i32, dev, (2,)),
        _ptr(slot_mapping, "slot_mapping", torch.int64, dev, (rows,)),
        _opt(positions, "positions", i32, dev, (rows,)),
        _opt(tree_mask, "tree_mask", i32, dev, (rows, words)),
        _opt(status, "status", i32, dev, (1,)))
    _launch(_lib.paged_build_step, "paged_build_step", dev, stream, args)


def release_blocks(keep_lens, blocks_held, block_tables, free_blocks, queue_state, *,
                   block_size: int, blocks_held_out, queue_state_out, status=None,
                   stream=None) -> None:
    """Returns the blocks behind each sequence's first keep_lens[s] tokens to the back of the
    free queue, in sequence and table order (0 ends a sequence). Buffers as in
    ``build_step``; free_blocks is written."""
    torch = _torch()
    i32, dev = torch.int32, _device(keep_lens, "keep_lens")
    S = keep_lens.shape[0]
    if block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("block_tables must be [S, max_blocks]")
    args = (
        _ptr(keep_lens, "keep_lens", i32, dev, (S,)),
        _ptr(blocks_held, "blocks_held", i32, dev, (S,)),
        _ptr(block_tables, "block_tables", i32, dev), _ptr(free_blocks, "free_blocks", i32, dev),
        _ptr(queue_state, "queue_state", i32, dev, (2,)), S, block_tables.shape[1], block_size,
        free_blocks.numel(), _ptr(blocks_held_out, "blocks_held_out", i32, dev, (S,)),
        _ptr(queue_state_out, "queue_state_out", i32, dev, (2,)),
        _opt(status, "status", i32, dev, (1,)))
    _launch(_lib.paged_release_blocks, "paged_release_blocks", dev, stream, args)


def _rows(x, name, dtype, dev, T, d):
    """(pointer, token stride) of rows [T, heads, d] that may be strided along T."""
    s0, s1, s2 = x.stride()
    if x.get_device() != dev or x.dtype is not dtype:
        _refuse(x, name, dtype, dev, None)
    heads = x.shape[1]
    if s2 != 1 or (s1 != d and heads > 1):
        raise ValueError(f"{name} rows must be contiguous [heads, d]")
    return x.data_ptr(), s0 if T > 1 else heads * d  # a single row has no stride of its own


def rotary_and_cache(q, k, v, q_out, k_cache, v_cache, positions, slot_mapping, inv_freq, *,
                     sections: Optional[Sequence[int]] = None, adjacent_pairs: bool = False,
                     k_scales=None, v_scales=None, k_zeros=None, v_zeros=None,
                     stream=None) -> None:
    """Rotary positions on q and k, fused with the slot-mapped cache write of k and v.

    q, q_out [T, Hq, d] and k, v [T, Hkv, d] (rows may be strided along T; q_out may be q),
    fp32 or bf16; inv_freq fp32 [R / 2] turns the first R channels of every head: channel i
    with i + R / 2, or 2i with 2i + 1 (adjacent_pairs). positions int32 [T], or [axes, T] with
    ``sections`` = frequencies of each axis (time, height, width). A token with a negative
    slot is padding: nothing of it is read or written."""
    torch = _torch()
    T, Hq, d = q.shape
    NB, Hkv, B, cd = k_cache.shape
    dev, half = _device(q, "q"), inv_freq.shape[0]
    if k.shape != (T, Hkv, d) or v.shape != k.shape or cd != d:
        raise ValueError("k / v do not match q and the cache")
    if q_out.shape != q.shape:
        raise ValueError("q_out must match q")
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    sec = (half,) if sections is None else tuple(sections)
    if positions.dim() > 2 or len(sec) != axes or not 1 <= axes <= 4:
        raise ValueError("positions must be [T], or [axes, T] with a section for each of 1 to 4 axes")
    code, pools, side = _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros, v_zeros, dev)
    dt = q.dtype
    (qp, qs), (kp, ks) = _rows(q, "q", dt, dev, T, d), _rows(k, "k", dt, dev, T, d)
    (vp, vs), (op, os_) = _rows(v, "v", dt, dev, T, d), _rows(q_out, "q_out", dt, dev, T, d)
    desc = pa_rotary_desc(T, Hq, Hkv, d, 2 * half, axes, sec, adjacent_pairs, B, NB, qs, ks, vs,
                          os_, _dtype_code(dt), code)
    _launch(_lib.rotary_and_cache, "rotary_and_cache", dev, stream, (
        qp, kp, vp, op, *pools,
        _ptr(positions, "positions", torch.int32, dev, (T,) if positions.dim() == 1 else (axes, T)),
        _ptr(slot_mapping, "slot_mapping", torch.int64, dev, (T,)),
        _ptr(inv_freq, "inv_freq", torch.float32, dev, (half,)), desc, *side))


def _tree_desc(q, k_cache, block_tables) -> pa_decode_desc:
    _, Hq, d = q.shape
    NB, Hkv, B, cd = k_cache.shape
    if cd != d:
        raise ValueError("head_dim of q and cache differ")
    qd = _dtype_code(q.dtype)
    return pa_decode_desc(block_tables.shape[0], Hq, Hkv, d, B, block_tables.shape[1], NB,
                          PARTITION_AUTO, qd, _dtype_code(k_cache.dtype), qd)


def tree_workspace_size(q, k_cache, block_tables, *, max_query_len: int,
                        max_context_len: int) -> int:
    """Workspace bytes of a ``paged_attn_tree`` call with tensors of these shapes and types."""
    return int(_lib.paged_attn_tree_workspace_size(
        _tree_desc(q, k_cache, block_tables), q.shape[0], max_query_len,
        max_context_len))


def paged_attn_tree(q, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask,
                    scale: float, out, *, max_query_len: int, max_context_len: int,
                    k_scales=None, v_scales=None, k_zeros=None, v_zeros=None, lse_out=None,
                    workspace=None, stream=None):
    """Attention of a step's drafted tokens over the paged cache.

    q, out [T, Hq, d]: rows query_start[s] .. query_start[s+1]-1 belong to sequence s and are
    the last tokens of context_lens[s], their K/V in the cache already. Row i sees every
    position before the rows and, of the rows, those whose bit is set in tree_mask int32
    [T, words] (bit j % 32 of word j / 32; 1 to 8 words). Rows behind the last sequence are
    left alone. workspace: uint8 of at least ``tree_workspace_size(...)`` bytes, one per call
    in flight. Other arguments as in ``paged_attn_prefill``."""
    torch = _torch()
    dev, i32 = _device(q, "q"), torch.int32
    desc = _tree_desc(q, k_cache, block_tables)
    T, Hq, _ = q.shape
    S = desc.num_seqs
    _, pools, side = _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros, v_zeros, dev)
    words = tree_mask.shape[-1]
    args = (
        _ptr(q, "q", q.dtype, dev), *pools, _ptr(block_tables, "block_tables", i32, dev),
        _ptr(context_lens, "context_lens", i32, dev, (S,)),
        _ptr(query_start, "query_start", i32, dev, (S + 1,)),
        _ptr(tree_mask, "tree_mask", i32, dev, (T, words)), words, T, max_query_len, scale,
        _ptr(out, "out", q.dtype, dev, q.shape), desc, max_context_len, *side,
        _opt(lse_out, "lse_out", torch.float32, dev, (T, Hq)),
        None if workspace is None else _ptr(workspace, "workspace", workspace.dtype, dev),
        0 if workspace is None else workspace.numel() * workspace.element_size())
    try:
        _launch(_lib.paged_attn_tree, "paged_attn_tree", dev, stream, args)
    except PagedAttnError as e:
        if e.status == PA_ERR_WORKSPACE:
            need = _lib.paged_attn_tree_workspace_size(desc, T, max_query_len,
                                                       max_context_len)
            raise PagedAttnError(e.status, f"paged_attn_tree needs {need} workspace bytes") from None
        raise
    return out


def tree_verify(parents, draft_tokens, target_tokens, query_start, context_lens, *, accepted,
                num_accepted, next_tokens, kept_lens, stream=None) -> None:
    """The accepted path of each draft tree under greedy choice.

    parents int32 [T], draft_tokens and target_tokens int64 [T] (each row's token, and the
    model's choice after it), query_start int32 [S + 1], context_lens int32 [S] (rows
    included). From row 0 on, the lowest child whose token is the one chosen after its
    parent is accepted. Outputs: accepted int32 [S, max_accept] (rows, then -1), num_accepted
    int32 [S], next_tokens int64 [S], kept_lens int32 [S]."""
    torch = _torch()
    i32, i64, dev = torch.int32, torch.int64, _device(query_start, "query_start")
    T, S = parents.shape[0], query_start.shape[0] - 1
    if accepted.dim() != 2:
        raise ValueError("accepted must be [S, max_accept]")
    A = accepted.shape[1]
    args = (
        _ptr(parents, "parents", i32, dev, (T,)),
        _ptr(draft_tokens, "draft_tokens", i64, dev, (T,)),
        _ptr(target_tokens, "target_tokens", i64, dev, (T,)),
        _ptr(query_start, "query_start", i32, dev, (S + 1,)),
        _ptr(context_lens, "context_lens", i32, dev, (S,)), S, T, A,
        _ptr(accepted, "accepted", i32, dev, (S, A)),
        _ptr(num_accepted, "num_accepted", i32, dev, (S,)),
        _ptr(next_tokens, "next_tokens", i64, dev, (S,)),
        _ptr(kept_lens, "kept_lens", i32, dev, (S,)))
    _launch(_lib.tree_verify, "tree_verify", dev, stream, args)


def compact_accepted(k_cache, v_cache, block_tables, context_lens, query_start, accepted,
                     num_accepted, *, k_scales=None, v_scales=None, k_zeros=None, v_zeros=None,
                     stream=None) -> None:
    """Moves the K/V of the accepted rows to the positions right behind the context, in place
    (``accepted`` and ``num_accepted`` as ``tree_verify`` gives them)."""
    torch = _torch()
    i32, dev, S = torch.int32, _device(k_cache, "k_cache"), context_lens.shape[0]
    code, pools, side = _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros, v_zeros, dev)
    NB, Hkv, B, d = k_cache.shape
    if accepted.dim() != 2 or block_tables.dim() != 2 or block_tables.shape[0] != S:
        raise ValueError("accepted must be [S, max_accept] and block_tables [S, max_blocks]")
    A = accepted.shape[1]
    _launch(_lib.compact_accepted, "compact_accepted", dev, stream, (
        *pools, _ptr(block_tables, "block_tables", i32, dev),
        _ptr(context_lens, "context_lens", i32, dev, (S,)),
        _ptr(query_start, "query_start", i32, dev, (S + 1,)),
        _ptr(accepted, "accepted", i32, dev, (S, A)),
        _ptr(num_accepted, "num_accepted", i32, dev, (S,)), S, A, block_tables.shape[1], Hkv, d, B,
        NB, code, *side))

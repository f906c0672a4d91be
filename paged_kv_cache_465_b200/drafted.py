"""Binding of the operators of a drafted (speculative) step: block tables and slot maps from
request lengths, rotary positions with the cache write, tree attention, acceptance.

As the rest of the binding, each function checks devices, types, shapes and contiguity, and
forwards pointers to the library on torch's current stream of the tensors' device. Everything
stays on the GPU: no call synchronises, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

import importlib.util
import os
from typing import Optional, Sequence

from .build import helper_path
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
    raise ValueError(f"{name} must be contiguous (its rows, where they may be strided)")


# Replaced by the native helper's functions on their first call: it needs torch, which this
# package does not import before it is given a tensor.
def _ptrs(*args):
    """(dev, tensor, name, dtype, shape, ...) -> device pointers; a tensor may be None, and a
    shape (any)."""
    _load_helper()
    return _ptrs(*args)


def _rows(*args):
    """(dev, tensor, name, dtype, shape) -> (device pointer, stride) of rows [T, heads, d] that
    may be strided along T."""
    _load_helper()
    return _rows(*args)


def _load_helper() -> None:
    global _ptrs, _rows
    path = helper_path(_torch())
    if not os.path.exists(path):
        raise ImportError(
            f"{path}, the checks of tensors for this torch and Python, is missing: build it with "
            "`python paged_kv_cache_465_b200/build.py`")
    spec = importlib.util.spec_from_file_location(__package__ + "._tensors", path)
    helper = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(helper)
    helper.on_refusal(_refuse)
    _ptrs, _rows = helper.ptrs, helper.rows


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
    """(cache dtype code, its shape, pointers of the pools, of scales and zero points)."""
    torch = _torch()
    shape, dt = k_cache.shape, k_cache.dtype
    if len(shape) != 4:
        raise ValueError("the caches must be [num_blocks, num_kv_heads, B, d]")
    pools = _ptrs(dev, k_cache, "k_cache", dt, None, v_cache, "v_cache", dt, shape)
    if k_scales is v_scales is k_zeros is v_zeros is None:
        return _dtype_code(dt), shape, pools, (None, None, None, None)
    bh, f32, i32 = shape[:2], torch.float32, torch.int32
    return _dtype_code(dt), shape, pools, _ptrs(
        dev, k_scales, "k_scales", f32, bh, v_scales, "v_scales", f32, bh,
        k_zeros, "k_zeros", i32, bh, v_zeros, "v_zeros", i32, bh)


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
    for none; without it rows form a chain. With no sequences (S = 0) every output is
    written too: no rows, no slots, the queue passed on.
    """
    torch = _torch()
    i32, dev = torch.int32, _device(context_lens, "context_lens")
    S, rows = context_lens.shape[0], slot_mapping.shape[0]
    words = 0 if tree_mask is None else tree_mask.shape[-1]
    width, s1, r1, one, two = block_tables.shape[-1], (S,), (rows,), (1,), (2,)
    ins = _ptrs(dev, context_lens, "context_lens", i32, s1, new_lens, "new_lens", i32, s1,
                blocks_held, "blocks_held", i32, s1, parents, "parents", i32, r1,
                block_tables, "block_tables", i32, (S, width),
                free_blocks, "free_blocks", i32, None, queue_state, "queue_state", i32, two)
    outs = _ptrs(dev, total_lens, "total_lens", i32, s1, query_start, "query_start", i32, (S + 1,),
                 blocks_held_out, "blocks_held_out", i32, s1,
                 queue_state_out, "queue_state_out", i32, two,
                 slot_mapping, "slot_mapping", torch.int64, r1, positions, "positions", i32, r1,
                 tree_mask, "tree_mask", i32, (rows, words), status, "status", i32, one)
    _launch(_lib.paged_build_step, "paged_build_step", dev, stream, (
        *ins, S, width, block_size, num_blocks, free_blocks.numel(), rows, words, *outs))


def release_blocks(keep_lens, blocks_held, block_tables, free_blocks, queue_state, *,
                   block_size: int, blocks_held_out, queue_state_out, status=None,
                   stream=None) -> None:
    """Returns the blocks behind each sequence's first keep_lens[s] tokens to the back of the
    free queue, in sequence and table order (0 ends a sequence). Buffers as in
    ``build_step``; free_blocks is written."""
    torch = _torch()
    i32, dev = torch.int32, _device(keep_lens, "keep_lens")
    S, width = keep_lens.shape[0], block_tables.shape[-1]
    s1 = (S,)
    ins = _ptrs(dev, keep_lens, "keep_lens", i32, s1, blocks_held, "blocks_held", i32, s1,
                block_tables, "block_tables", i32, (S, width),
                free_blocks, "free_blocks", i32, None, queue_state, "queue_state", i32, (2,))
    outs = _ptrs(dev, blocks_held_out, "blocks_held_out", i32, s1,
                 queue_state_out, "queue_state_out", i32, (2,), status, "status", i32, (1,))
    _launch(_lib.paged_release_blocks, "paged_release_blocks", dev, stream, (
        *ins, S, width, block_size, free_blocks.numel(), *outs))


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
    qshape, dt, dev = q.shape, q.dtype, _device(q, "q")
    T, Hq, d = qshape
    code, (NB, Hkv, B, cd), pools, side = _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros,
                                                      v_zeros, dev)
    if cd != d:
        raise ValueError("head_dim of q and cache differ")
    half, ps = inv_freq.shape[0], positions.shape
    axes = 1 if len(ps) == 1 else ps[0]
    sec = (half,) if sections is None else tuple(sections)
    if len(ps) > 2 or len(sec) != axes or not 1 <= axes <= 4:
        raise ValueError("positions must be [T], or [axes, T] with a section for each of 1 to 4 axes")
    qp, qs = _rows(dev, q, "q", dt, qshape)
    op, os_ = _rows(dev, q_out, "q_out", dt, qshape)
    kp, ks = _rows(dev, k, "k", dt, (T, Hkv, d))
    vp, vs = _rows(dev, v, "v", dt, (T, Hkv, d))
    desc = pa_rotary_desc(T, Hq, Hkv, d, 2 * half, axes, sec, adjacent_pairs, B, NB, qs, ks, vs,
                          os_, _dtype_code(dt), code)
    _launch(_lib.rotary_and_cache, "rotary_and_cache", dev, stream, (
        qp, kp, vp, op, *pools,
        *_ptrs(dev, positions, "positions", torch.int32, (T,) if len(ps) == 1 else (axes, T),
               slot_mapping, "slot_mapping", torch.int64, (T,),
               inv_freq, "inv_freq", torch.float32, (half,)), desc, *side))


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
    qshape, dt, S, words = q.shape, q.dtype, desc.num_seqs, tree_mask.shape[-1]
    T = qshape[0]
    _, _, pools, side = _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros, v_zeros, dev)
    (qp, op, bt, cl, qs, mp, lp) = _ptrs(
        dev, q, "q", dt, None, out, "out", dt, qshape, block_tables, "block_tables", i32, None,
        context_lens, "context_lens", i32, (S,), query_start, "query_start", i32, (S + 1,),
        tree_mask, "tree_mask", i32, (T, words),
        lse_out, "lse_out", torch.float32, qshape[:2])
    wp, wn = None, 0
    if workspace is not None:
        wp, = _ptrs(dev, workspace, "workspace", workspace.dtype, None)
        wn = workspace.numel() * workspace.element_size()
    args = (qp, *pools, bt, cl, qs, mp, words, T, max_query_len, scale, op, desc, max_context_len,
            *side, lp, wp, wn)
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
    A, t1, s1 = accepted.shape[1], (T,), (S,)
    ins = _ptrs(dev, parents, "parents", i32, t1, draft_tokens, "draft_tokens", i64, t1,
                target_tokens, "target_tokens", i64, t1, query_start, "query_start", i32, None,
                context_lens, "context_lens", i32, s1)
    outs = _ptrs(dev, accepted, "accepted", i32, (S, A), num_accepted, "num_accepted", i32, s1,
                 next_tokens, "next_tokens", i64, s1, kept_lens, "kept_lens", i32, s1)
    _launch(_lib.tree_verify, "tree_verify", dev, stream, (*ins, S, T, A, *outs))


def compact_accepted(k_cache, v_cache, block_tables, context_lens, query_start, accepted,
                     num_accepted, *, k_scales=None, v_scales=None, k_zeros=None, v_zeros=None,
                     stream=None) -> None:
    """Moves the K/V of the accepted rows to the positions right behind the context, in place
    (``accepted`` and ``num_accepted`` as ``tree_verify`` gives them)."""
    torch = _torch()
    i32, dev, S = torch.int32, _device(k_cache, "k_cache"), context_lens.shape[0]
    code, (NB, Hkv, B, d), pools, side = _cache_ptrs(k_cache, v_cache, k_scales, v_scales, k_zeros,
                                                     v_zeros, dev)
    if accepted.dim() != 2:
        raise ValueError("accepted must be [S, max_accept]")
    A, width, s1 = accepted.shape[1], block_tables.shape[-1], (S,)
    ptrs = _ptrs(dev, block_tables, "block_tables", i32, (S, width),
                 context_lens, "context_lens", i32, s1, query_start, "query_start", i32, (S + 1,),
                 accepted, "accepted", i32, (S, A), num_accepted, "num_accepted", i32, s1)
    _launch(_lib.compact_accepted, "compact_accepted", dev, stream, (
        *pools, *ptrs, S, A, width, Hkv, d, B, NB, code, *side))

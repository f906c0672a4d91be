"""The operators of a drafted step, from their definitions (test infrastructure only).

Bookkeeping in Python loops over sequences and tokens, floating-point steps in float64; only
the cache conversions, which the library defines in float32, are float32 (and so bit-exact).
Block allocation follows ``oracle.paged.RefAllocator`` (FIFO queue, sequence order): [KVPaged]
"PagedAttention: OS virtual-memory style management", [KVFail] Key Points.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

from .attention import decode_values, gather_kv
from .codecs import bf16_encode, e4m3_decode, e4m3_encode, int8_encode


def ref_ancestors(parents: Sequence[int]) -> List[List[int]]:
    """Each row's ancestors and itself; a parent that is not before its child counts as none."""
    see = []
    for i, p in enumerate(parents):
        see.append((see[p] if 0 <= p < i else []) + [i])
    return see


def mask_words(rows: Sequence[Sequence[int]], words: int) -> np.ndarray:
    """int32 [len(rows), words]: bit j % 32 of word j / 32 set for every j of a row."""
    m = np.zeros((len(rows), words), dtype=np.uint32)
    for i, js in enumerate(rows):
        for j in js:
            m[i, j // 32] |= np.uint32(1 << (j % 32))
    return m.view(np.int32)


def ref_build_step(context, new, held, tables, ring, queue, block_size: int, num_blocks: int,
                   rows: int, parents=None, words: int = 0):
    """(tables, held, queue, total_lens, query_start, slots, positions, mask) after the step,
    or None when it has to be refused as a whole."""
    S, width = tables.shape
    tables, held = tables.copy(), [int(h) for h in held]
    head, count = int(queue[0]), int(queue[1])
    cap = len(ring)
    if not (0 <= head < cap and 0 <= count <= cap) or min(context) < 0 or min(new) < 0:
        return None
    if sum(int(n) for n in new) > rows:
        return None
    qs, slots = [0], np.full(rows, -1, dtype=np.int64)
    positions, mask = np.zeros(rows, dtype=np.int32), np.zeros((rows, max(words, 1)), dtype=np.int32)
    for s in range(S):
        c, n = int(context[s]), int(new[s])
        if held[s] < 0 or held[s] > width or held[s] * block_size < c or \
                c + n > width * block_size or (words and n > 32 * words):
            return None
        while held[s] * block_size < c + n:
            if count == 0:
                return None
            tables[s, held[s]] = ring[head]
            held[s] += 1
            head, count = (head + 1) % cap, count - 1
        r0 = qs[-1]
        par = list(range(-1, n - 1)) if parents is None else [int(p) for p in parents[r0:r0 + n]]
        see = ref_ancestors(par)
        for i in range(n):
            b = int(tables[s, (c + i) // block_size])
            slots[r0 + i] = b * block_size + (c + i) % block_size if 0 <= b < num_blocks else -1
            positions[r0 + i] = c + len(see[i]) - 1
        if words:
            mask[r0:r0 + n] = mask_words(see, words)
        qs.append(r0 + n)
    total = np.asarray(context, dtype=np.int64) + np.asarray(new, dtype=np.int64)
    return (tables, np.array(held, dtype=np.int32), np.array([head, count], dtype=np.int32),
            total.astype(np.int32), np.array(qs, dtype=np.int32), slots, positions, mask)


def ref_release(keep, held, tables, ring, queue, block_size: int):
    """(ring, held, queue) afterwards, or None when it has to be refused."""
    ring, held = ring.copy(), [int(h) for h in held]
    head, count, cap = int(queue[0]), int(queue[1]), len(ring)
    if not (0 <= head < cap and 0 <= count <= cap) or min(keep) < 0:
        return None
    for s in range(len(held)):
        if held[s] < 0 or held[s] > tables.shape[1]:
            return None
        kept = min(held[s], -(-int(keep[s]) // block_size))
        for b in tables[s, kept:held[s]]:
            if count == cap:
                return None
            ring[(head + count) % cap] = b
            count += 1
        held[s] = kept
    return ring, np.array(held, dtype=np.int32), np.array([head, count], dtype=np.int32)


def ref_turn(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, sections: Sequence[int],
             adjacent: bool) -> np.ndarray:
    """Rows x [T, heads, d] (float64) turned by their positions [axes, T], pair by pair."""
    y = x.copy()
    half, i = len(inv_freq), 0
    for axis, size in enumerate(sections):
        for _ in range(size):
            a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
            th = positions[axis].astype(np.float64) * np.float64(inv_freq[i])
            c, s = np.cos(th)[:, None], np.sin(th)[:, None]
            y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
            y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
            i += 1
    assert i == half
    return y


def ref_tree(q: np.ndarray, query_start, see: Sequence[Sequence[Sequence[int]]], k_cache, v_cache,
             block_tables, context_lens, scale: float, num_kv_heads: int, q_dtype: str,
             kv_dtype: str, k_scales=None, v_scales=None, k_zeros=None, v_zeros=None):
    """Attention of drafted rows, float64: see[s][i] lists the rows of sequence s that its row i
    sees beside the context before them. Returns out [T, Hq, d], lse [T, Hq], the
    softmax-weighted mean of |V| (what a rounding of the weights can move) and the largest
    scale * sum |q K| of each row (what a rounding of the products can move). Rows of no
    sequence are NaN. Keys that a row does not see are left out, not masked."""
    T, Hq, d = q.shape
    G = Hq // num_kv_heads
    qv = decode_values(q, q_dtype)
    out, absv = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d))
    lse, big = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for s in range(len(context_lens)):
        r0, n = int(query_start[s]), int(query_start[s + 1]) - int(query_start[s])
        ctx = int(context_lens[s])
        if n == 0:
            continue
        for kvh in range(num_kv_heads):
            K, V = gather_kv(k_cache, v_cache, block_tables[s], ctx, kvh, kv_dtype, k_scales,
                             v_scales, k_zeros, v_zeros)
            for i in range(n):
                keys = np.concatenate([np.arange(ctx - n), ctx - n + np.array(see[s][i], dtype=int)
                                       ]).astype(int)
                hs = slice(kvh * G, (kvh + 1) * G)
                if len(keys) == 0:
                    out[r0 + i, hs], lse[r0 + i, hs] = 0.0, -np.inf
                    continue
                x = qv[r0 + i, hs]
                z = scale * (x @ K[keys].T)
                big[r0 + i, hs] = abs(scale) * (np.abs(x) @ np.abs(K[keys]).T).max(-1)
                m = z.max(-1, keepdims=True)
                e = np.exp(z - m)
                l = e.sum(-1, keepdims=True)
                out[r0 + i, hs] = e @ V[keys] / l
                absv[r0 + i, hs] = e @ np.abs(V[keys]) / l
                lse[r0 + i, hs] = (m + np.log(l))[:, 0]
    return out, lse, absv, big


def ref_verify(parents, draft, target, query_start, context_lens, max_accept: int):
    """(paths, next tokens, kept lengths)."""
    paths, nxt, kept = [], [], []
    for s in range(len(context_lens)):
        r0, n = int(query_start[s]), int(query_start[s + 1]) - int(query_start[s])
        path, want, cur = [], -1, 0
        while n and len(path) < max_accept:
            path.append(cur)
            want = int(target[r0 + cur])
            kids = [i for i in range(cur + 1, n)
                    if int(parents[r0 + i]) == cur and int(draft[r0 + i]) == want]
            if not kids:
                break
            cur = kids[0]
        paths.append(path)
        nxt.append(want)
        kept.append(int(context_lens[s]) - n + len(path))
    return paths, nxt, kept


def stored_codes(x: np.ndarray, dtype: str, scale=None, zero=None) -> np.ndarray:
    """float32 values as a cache holds them (float32 division, as the cache write defines)."""
    x = np.asarray(x, dtype=np.float32)
    if dtype == "f32":
        return x
    if dtype == "bf16":
        return bf16_encode(x)
    y = x / np.asarray(scale, dtype=np.float32)
    return e4m3_encode(y) if dtype == "fp8" else int8_encode(y, zero)


def ref_compact(cache: np.ndarray, block_tables, context_lens, query_start, paths, dtype: str,
                scales: Optional[np.ndarray] = None, zeros: Optional[np.ndarray] = None
                ) -> np.ndarray:
    """The pool (storage codes [NB, H, B, d]) after every path's rows have moved, in order."""
    pool = cache.copy()
    B = pool.shape[2]
    for s, path in enumerate(paths):
        n = int(query_start[s + 1]) - int(query_start[s])
        base = int(context_lens[s]) - n
        for i, p in enumerate(path):
            (b0, o0), (b1, o1) = ((int(block_tables[s][t // B]), t % B) for t in (base + p, base + i))
            if p == i:
                continue
            for h in range(pool.shape[1]):
                codes = pool[b0, h, o0].copy()
                if scales is not None:
                    z0, z1 = (0, 0) if zeros is None else (zeros[b0, h], zeros[b1, h])
                    if scales[b0, h] != scales[b1, h] or z0 != z1:
                        v = e4m3_decode(codes) if dtype == "fp8" else codes.astype(np.float64) - z0
                        v = v.astype(np.float32) * np.float32(scales[b0, h])
                        codes = stored_codes(v, dtype, scales[b1, h], z1)
                pool[b1, h, o1] = codes
    return pool

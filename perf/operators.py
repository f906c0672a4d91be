"""Cases for the operators of a drafted (speculative) step over the paged KV cache.

A serving step that drafts tokens goes through four operators, each measured alone:

* ``build``   block tables, slot map, positions and ancestor masks from request lengths (after
              the blocks of ended or shortened sequences went back to the free queue);
* ``rotary``  rotary positions (one or several axes) on q and k, fused with the cache write;
* ``tree``    attention of a tree of drafted tokens over the paged cache;
* ``accept``  the longest drafted path that the model agrees with, and its K/V moved to the
              positions right after the context.

``run`` computes an operator in plain torch operations, or, where ``own`` is true, with this
repository's entry points. Lengths follow from the case alone (spread over its range), values
from the seed. Layouts are the library's: pools [blocks][kv heads][block tokens][128], int32
block tables, int64 slots.
"""
import math

import torch

own = False

D = 128  # head dimension of every configuration measured here


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one request, a short context and a small tree: latency
        dict(name="tree_single", op="tree", seqs=1, hq=32, hkv=8, bs=16, kv="bf16", ctx_lo=250,
             ctx_hi=250, n_lo=8, n_hi=8),
        # a small batch of requests at every stage, trees of different sizes
        dict(name="tree_b32_bf16", op="tree", seqs=32, hq=32, hkv=8, bs=16, kv="bf16", ctx_lo=1,
             ctx_hi=4096, n_lo=1, n_hi=16),
        # a full batch on an fp8 cache, short drafts
        dict(name="tree_b256_fp8", op="tree", seqs=256, hq=32, hkv=8, bs=16, kv="fp8", ctx_lo=16,
             ctx_hi=8192, n_lo=8, n_hi=8),
        # few requests with very long contexts
        dict(name="tree_long_bf16", op="tree", seqs=8, hq=64, hkv=8, bs=16, kv="bf16",
             ctx_lo=131072, ctx_hi=131072, n_lo=16, n_hi=16),
        # int8 cache in 32-token blocks, odd lengths, large trees
        dict(name="tree_int8_odd", op="tree", seqs=13, hq=16, hkv=2, bs=32, kv="int8", ctx_lo=901,
             ctx_hi=20001, n_lo=5, n_hi=63),
        # a plain decode step's bookkeeping: one new token for each of 256 sequences
        dict(name="build_decode", op="build", seqs=256, bs=16, ctx_lo=16, ctx_hi=8192, n_lo=1,
             n_hi=1, tree=False, ended=0),
        # a large drafted step after some sequences ended
        dict(name="build_tree", op="build", seqs=1021, bs=16, ctx_lo=1, ctx_hi=4096, n_lo=1,
             n_hi=64, tree=True, ended=37),
        # a decode step's tokens: latency
        dict(name="rotary_step", op="rotary", tokens=37, pad=3, hq=32, hkv=8, bs=16, kv="bf16",
             axes=1, rot=128, adjacent=False, far=8192),
        # eight 2048-token prompts with time / height / width positions
        dict(name="rotary_prompt_3axes", op="rotary", tokens=16384, pad=100, hq=32, hkv=8, bs=16,
             kv="bf16", axes=3, rot=128, adjacent=False, far=131072),
        # a chunk into an fp8 cache, the first half of each head rotated in adjacent pairs
        dict(name="rotary_chunk_fp8", op="rotary", tokens=8191, pad=0, hq=64, hkv=8, bs=16,
             kv="fp8", axes=1, rot=64, adjacent=True, far=131072),
        # acceptance for a small batch of small trees
        dict(name="accept_b32_bf16", op="accept", seqs=32, hkv=8, bs=16, kv="bf16", ctx_lo=1,
             ctx_hi=300, n_lo=1, n_hi=16, deep=8),
        # acceptance for a full batch of large trees on an fp8 cache
        dict(name="accept_b256_fp8", op="accept", seqs=256, hkv=8, bs=16, kv="fp8", ctx_lo=16,
             ctx_hi=500, n_lo=64, n_hi=64, deep=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "build", "rotary", "accept"])
    bs = rng.choice([8, 16, 16, 32])
    kv = rng.choice(["bf16", "fp8", "int8"])
    group = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 8, 8])
    if op == "tree":
        seqs = _log(rng, 1, 256)
        n_hi = _log(rng, 1, 64)
        # as many padded (token, kv head) keys as the longest listed case at most, and a
        # quarter of its (query row, key) pairs
        hi = min(131072, (1 << 20) * 8 // (seqs * hkv), (1 << 27) // (seqs * hkv * n_hi * group))
        hi = _log(rng, min(40, hi), max(40, hi))
        return dict(op=op, seqs=seqs, hq=hkv * group, hkv=hkv, bs=bs, kv=kv,
                    ctx_lo=rng.randint(1, max(1, hi // 2)), ctx_hi=hi,
                    n_lo=rng.randint(0, n_hi) if seqs > 1 else n_hi, n_hi=n_hi)
    if op == "build":
        n_hi = _log(rng, 1, 64)
        return dict(op=op, seqs=_log(rng, 1, 1021), bs=bs, ctx_lo=rng.randint(1, 64),
                    ctx_hi=_log(rng, 64, 4096), n_lo=rng.randint(0, n_hi), n_hi=n_hi,
                    tree=rng.random() < 0.5, ended=rng.randint(0, 64))
    if op == "rotary":
        axes = rng.choice([1, 1, 3])
        return dict(op=op, tokens=_log(rng, 1, 8191), pad=rng.randint(0, 40), hq=hkv * group,
                    hkv=hkv, bs=bs, kv=kv, axes=axes, rot=rng.choice([64, 96, 128]),
                    adjacent=rng.random() < 0.5, far=_log(rng, 1000, 1000000))
    n_hi = _log(rng, 1, 64)
    return dict(op=op, seqs=_log(rng, 1, 256), hkv=hkv, bs=bs, kv=kv, ctx_lo=rng.randint(1, 100),
                ctx_hi=_log(rng, 100, 500), n_lo=rng.randint(0, n_hi), n_hi=n_hi,
                deep=rng.randint(1, 16))


def _spread(lo, hi, count, step):
    """`count` whole numbers spread evenly over the logarithm of [lo, hi], out of order."""
    at = [(k + 0.5) / count for k in range(count)]
    v = [lo + int((math.expm1(math.log1p(hi - lo) * a))) for a in at]
    v[-1] = hi
    return [v[(k * step + count // 3) % count] for k in range(count)] if math.gcd(step, count) == 1 else v


def _lens(c):
    """(tokens cached before the step, new tokens) of each sequence."""
    base = _spread(c["ctx_lo"], c["ctx_hi"], c["seqs"], 7)
    new = [c["n_lo"] + (5 * k + 3) % (c["n_hi"] - c["n_lo"] + 1) for k in range(c["seqs"])]
    if max(new) == 0:
        new[0] = 1
    return base, new


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _starts(new):
    qs = [0]
    for n in new:
        qs.append(qs[-1] + n)
    return qs


def _pool(g, kv, nb, hkv, bs):
    """K and V pools with values N(0, 1) in the cache's type, and its scales / zero points."""
    s = dict(k_scales=None, v_scales=None, k_zeros=None, v_zeros=None)
    for n in "kv":
        shape = (nb, hkv, bs, D)
        if kv == "bf16":
            s[n + "_cache"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
            continue
        # a block's scale follows its largest value: they differ from block to block
        sc = (3.5 + torch.rand(nb, hkv, device="cuda", generator=g) * 1.5) / (448 if kv == "fp8" else 128)
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        y = x / sc[:, :, None, None]
        if kv == "fp8":
            s[n + "_cache"] = y.clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            z = torch.randint(-20, 21, (nb, hkv), device="cuda", generator=g, dtype=torch.int32)
            s[n + "_cache"] = (y.round_() + z[:, :, None, None]).clamp_(-128, 127).to(torch.int8)
            s[n + "_zeros"] = z
        s[n + "_scales"] = sc
    return s


def _parents(g, new):
    """A tree for each sequence: node 0 is its root, every later node hangs on an earlier one
    (as often as not the one before it)."""
    i = torch.cat([torch.arange(n, device="cuda") for n in new])
    u = torch.rand(i.numel(), device="cuda", generator=g)
    far = (torch.rand(i.numel(), device="cuda", generator=g) * i).long().clamp_(max=10**6)
    p = torch.where(u < 0.5, i - 1, torch.minimum(far, i - 1))
    return torch.where(i == 0, torch.full_like(i, -1), p).int()


def _tables(g, base, new, bs):
    """Block tables that hold context and new tokens, over a shuffled pool with spare blocks."""
    need = [-(-(b + n) // bs) for b, n in zip(base, new)]
    nb = sum(need) + 2
    perm = torch.randperm(nb - 1, device="cuda", generator=g).int()  # the last block stays unused
    bt = torch.full((len(base), max(need)), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(max(need), device="cuda")
    held = _ints(need)
    bt[col[None, :] < held[:, None]] = perm[: sum(need)]
    return bt, nb


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "rotary":
        t, nb = c["tokens"], -(-(c["tokens"] + 1) // c["bs"]) + 2
        dt = torch.bfloat16
        s["q"] = torch.empty(t, c["hq"], D, dtype=dt, device="cuda").normal_(generator=g)
        kv = torch.empty(t, 2 * c["hkv"], D, dtype=dt, device="cuda").normal_(generator=g)
        s["k"], s["v"] = kv[:, : c["hkv"]], kv[:, c["hkv"]:]  # rows of one projection
        s["q_out"] = torch.zeros_like(s["q"])
        s.update(_pool(g, c["kv"], nb, c["hkv"], c["bs"]))
        slots = torch.randperm((nb - 1) * c["bs"], device="cuda", generator=g)[:t]
        pad = torch.randperm(t, device="cuda", generator=g)[: min(c["pad"], t - 1)]
        slots[pad] = -1
        s["slots"] = slots
        s["positions"] = torch.randint(0, c["far"], (c["axes"], t), device="cuda", generator=g,
                                       dtype=torch.int32)
        h = c["rot"] // 2
        s["inv_freq"] = 1.0 / 10000.0 ** (torch.arange(h, device="cuda").float() / h)
        # a quarter of the pairs for time, the others shared by height and width
        a = h // 4
        s["sections"] = [h] if c["axes"] == 1 else [a, (h - a) // 2, h - a - (h - a) // 2]
        s["axis"] = _ints([k for k, m in enumerate(s["sections"]) for _ in range(m)], torch.int64)
        return s
    base, new = _lens(c)
    qs = _starts(new)
    total = qs[-1]
    if c["op"] == "build":
        S, bs = c["seqs"], c["bs"]
        ended = min(c["ended"], S // 2)
        keep = [0 if k < ended else base[k] for k in range(S)]
        held = [-(-(b + (k % 3 == 0) * bs) // bs) for k, b in enumerate(base)]  # some hold a spare
        width = max(-(-(b + n) // bs) for b, n in zip(base, new)) + 2
        nb = S * width + 5
        perm = torch.randperm(nb, device="cuda", generator=g).int()
        bt = torch.full((S, width), -1, dtype=torch.int32, device="cuda")
        used = sum(held)
        bt[torch.arange(width, device="cuda")[None, :] < _ints(held)[:, None]] = perm[:used]
        # the queue is a ring; its front stands near the end, so that it wraps
        ring = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
        head, count = nb - 3, nb - used
        ring[(head + torch.arange(count, device="cuda")) % nb] = perm[used:]
        rows = total + 11  # a step of fixed width has padding rows
        s.update(block_tables=bt, held=_ints(held), ring=ring, queue=_ints([head, count]),
                 keep=_ints(keep), context=_ints(keep), new=_ints(new), rows=rows, num_blocks=nb,
                 width=width, words=2)
        s["parents"] = torch.cat([_parents(g, new), _ints([-1] * 11)]) if c["tree"] else None
        for n, shape, dt in (("held_mid", S, torch.int32), ("queue_mid", 2, torch.int32),
                             ("held_out", S, torch.int32), ("queue_out", 2, torch.int32),
                             ("total_lens", S, torch.int32), ("query_start", S + 1, torch.int32),
                             ("slots", rows, torch.int64), ("positions", rows, torch.int32),
                             ("mask", (rows, 2), torch.int32), ("status", 2, torch.int32)):
            s[n] = torch.zeros(shape, dtype=dt, device="cuda")
        return s
    s["block_tables"], nb = _tables(g, base, new, c["bs"])
    s.update(_pool(g, c["kv"], nb, c["hkv"], c["bs"]))
    s["context_lens"] = _ints([b + n for b, n in zip(base, new)])
    s["query_start"] = _ints(qs)
    s["max_query"] = max(new)
    s["max_context"] = max(b + n for b, n in zip(base, new))
    s["parents"] = _parents(g, new)
    if c["op"] == "tree":
        rows = total + (2 if c["seqs"] > 1 else 0)  # a batch has padding rows
        s["q"] = torch.empty(rows, c["hq"], D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["mask"] = torch.zeros(rows, 2, dtype=torch.int32, device="cuda")
        s["mask"][:total] = _ancestors(s["parents"], s["query_start"], 2)[0]
        s["scale"] = 1.0 / math.sqrt(D)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(rows, c["hq"], device="cuda")
        return s
    # acceptance: the model agrees with a node's first child three times out of four
    s["draft"] = torch.randint(0, 50, (total,), device="cuda", generator=g)
    first = torch.full((total,), total, device="cuda")
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(s["query_start"][1:].long(), row, right=True)
    up = s["query_start"].long()[seq] + s["parents"].long()
    child = s["parents"] >= 0
    first.scatter_reduce_(0, up[child], row[child], "amin")
    agree = (torch.rand(total, device="cuda", generator=g) < 0.75) & (first < total)
    other = torch.randint(0, 50, (total,), device="cuda", generator=g)
    s["target"] = torch.where(agree, s["draft"][first.clamp(max=total - 1)], other)
    S, a = c["seqs"], c["deep"]
    s["accepted"] = torch.zeros(S, a, dtype=torch.int32, device="cuda")
    s["num_accepted"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    s["next_tokens"] = torch.zeros(S, dtype=torch.int64, device="cuda")
    s["kept_lens"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"tree": _own_tree, "build": _own_build, "rotary": _own_rotary,
                "accept": _own_accept}[op](state)
    return {"tree": _plain_tree, "build": _plain_build, "rotary": _plain_rotary,
            "accept": _plain_accept}[op](state)


def _shown(s):
    """The pools as numbers: fp8 codes are numbers already, int8 codes the values they hold."""
    if s["k_zeros"] is None:
        return [s["k_cache"], s["v_cache"]]
    return [((s[n + "_cache"] - s[n + "_zeros"][:, :, None, None])
             * s[n + "_scales"][:, :, None, None]).bfloat16() for n in "kv"]


def _own_tree(s):
    import paged_kv_cache_465_b200 as pa
    if "workspace" not in s:  # a program keeps its workspace from step to step
        s["workspace"] = torch.empty(max(16, pa.tree_workspace_size(
            s["q"], s["k_cache"], s["block_tables"], max_query_len=s["max_query"],
            max_context_len=s["max_context"])), dtype=torch.uint8, device="cuda")
    pa.paged_attn_tree(s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                       s["query_start"], s["mask"], s["scale"], s["out"],
                       max_query_len=s["max_query"], max_context_len=s["max_context"],
                       k_scales=s["k_scales"], v_scales=s["v_scales"], k_zeros=s["k_zeros"],
                       v_zeros=s["v_zeros"], lse_out=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _own_build(s):
    import paged_kv_cache_465_b200 as pa
    c = s["case"]
    # the tables are extended in place: every pass starts from those of the state
    if "tables" not in s:
        s["tables"] = torch.empty_like(s["block_tables"])
    bt = s["tables"].copy_(s["block_tables"])
    pa.release_blocks(s["keep"], s["held"], bt, s["ring"], s["queue"], block_size=c["bs"],
                      blocks_held_out=s["held_mid"], queue_state_out=s["queue_mid"],
                      status=s["status"][:1])
    pa.build_step(s["context"], s["new"], s["held_mid"], bt, s["ring"], s["queue_mid"],
                  block_size=c["bs"], num_blocks=s["num_blocks"], total_lens=s["total_lens"],
                  query_start=s["query_start"], blocks_held_out=s["held_out"],
                  queue_state_out=s["queue_out"], slot_mapping=s["slots"],
                  positions=s["positions"], parents=s["parents"],
                  tree_mask=s["mask"] if c["tree"] else None, status=s["status"][1:])
    return [bt] + [s[n] for n in ("ring", "held_out", "queue_out", "total_lens", "query_start",
                                  "slots", "positions", "mask", "status")]


def _own_rotary(s):
    import paged_kv_cache_465_b200 as pa
    pa.rotary_and_cache(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"],
                        s["positions"], s["slots"], s["inv_freq"], sections=s["sections"],
                        adjacent_pairs=s["case"]["adjacent"], k_scales=s["k_scales"],
                        v_scales=s["v_scales"], k_zeros=s["k_zeros"], v_zeros=s["v_zeros"])
    return [s["q_out"]] + _shown(s)


def _own_accept(s):
    import paged_kv_cache_465_b200 as pa
    pa.tree_verify(s["parents"], s["draft"], s["target"], s["query_start"], s["context_lens"],
                   accepted=s["accepted"], num_accepted=s["num_accepted"],
                   next_tokens=s["next_tokens"], kept_lens=s["kept_lens"])
    pa.compact_accepted(s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                        s["query_start"], s["accepted"], s["num_accepted"],
                        k_scales=s["k_scales"], v_scales=s["v_scales"], k_zeros=s["k_zeros"],
                        v_zeros=s["v_zeros"])
    return [s[n] for n in ("accepted", "num_accepted", "next_tokens", "kept_lens")] + _shown(s)


def _rows(query_start, rows):
    """Sequence and place in it of every token row (rows behind the last sequence: live false)."""
    t = torch.arange(rows, device=query_start.device)
    seq = torch.searchsorted(query_start[1:].long(), t, right=True)
    live = seq < query_start.numel() - 1
    seq = seq.clamp(max=query_start.numel() - 2)
    return seq, t - query_start.long()[seq], live


def _ancestors(parents, query_start, words):
    """([rows, words] int32 bits of each row's ancestors and itself, number of ancestors)."""
    rows = parents.numel()
    seq, i, live = _rows(query_start, rows)
    up = torch.where((parents >= 0) & live, parents.long() + query_start.long()[seq], -1)
    see = torch.zeros(rows, 32 * words, dtype=torch.bool, device=parents.device)
    see.scatter_(1, i.clamp(0, 32 * words - 1)[:, None], live[:, None])
    for _ in range(6):  # each round doubles how far up a row has looked: 64 nodes at most
        there = up.clamp(min=0)
        see = see | (see[there] & (up >= 0)[:, None])
        up = torch.where(up >= 0, up[there], -1)
    depth = see.sum(1) - 1
    bit = 2 ** torch.arange(32, device=parents.device)
    packed = (see.view(rows, words, 32) * bit).sum(-1)
    return torch.where(packed >= 2**31, packed - 2**32, packed).int(), depth


def _values(cache, blk, off, scales, zeros):
    """Float values [..., kv heads, D] of the cache at (blk, off); fp8 and int8 dequantised."""
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[blk, :, off]
    x = (x.view(cache.dtype) if cache.dtype == torch.float8_e4m3fn else x).float()
    if zeros is not None:
        x = x - zeros[blk][..., None]
    return x if scales is None else x * scales[blk][..., None]


def _plain_tree(s):
    c = s["case"]
    S, N, L, G, hkv = c["seqs"], s["max_query"], s["max_context"], c["hq"] // c["hkv"], c["hkv"]
    qs, ctx = s["query_start"].long(), s["context_lens"].long()
    n, rows = qs[1:] - qs[:-1], s["q"].shape[0]
    t = torch.arange(L, device="cuda")
    blk = s["block_tables"].clamp(min=0).long()[:, t // c["bs"]]
    off = (t % c["bs"]).expand(S, L)
    k = _values(s["k_cache"], blk, off, s["k_scales"], s["k_zeros"])
    i = torch.arange(N, device="cuda")
    at = (qs[:-1, None] + i).clamp(max=rows - 1)
    q = s["q"][at].float().view(S, N, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, hkv, N * G, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).view(S, hkv, N, G, L)
    z *= s["scale"]
    j = t[None, :] - (ctx - n)[:, None]  # which drafted token a key is
    word = (j.clamp(0, 63) // 32)[:, None, :].expand(S, N, L)
    bit = (s["mask"][at].gather(2, word) >> (j.clamp(min=0) % 32)[:, None, :].int()) & 1
    see = ((j < 0)[:, None, :] | (bit == 1)) & (t[None, :] < ctx[:, None])[:, None, :]
    z.masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    z = z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    v = _values(s["v_cache"], blk, off, s["v_scales"], s["v_zeros"])
    v = torch.where((t[None, :] < ctx[:, None])[..., None, None], v, 0.0)
    o = torch.matmul(z.view(S, hkv, N * G, L), v.permute(0, 2, 1, 3)).view(S, hkv, N, G, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 2, 1, 3, 4).reshape(S, N, c["hq"], D)
    lse = (m + l.log())[..., 0].permute(0, 2, 1, 3).reshape(S, N, c["hq"])
    seq, place, live = _rows(s["query_start"], rows)
    place = place.clamp(max=N - 1)
    out = torch.where(live[:, None, None], o[seq, place], 0.0)
    return out.to(s["q"].dtype), torch.where(live[:, None], lse[seq, place], 0.0)


def _plain_build(s):
    c = s["case"]
    bs, bt, ring, rows, width = c["bs"], s["block_tables"], s["ring"], s["rows"], s["width"]
    cap = ring.numel()
    col = torch.arange(width, device="cuda")
    # blocks of ended sequences go back, in table order, to the back of the queue
    held = s["held"].long()
    kept = torch.minimum(held, (s["keep"].long() + bs - 1) // bs)
    back = held - kept
    head, count = s["queue"].long()
    at = (back.cumsum(0) - back)[:, None] + col - kept[:, None]
    goes = (col >= kept[:, None]) & (col < held[:, None])
    place = torch.where(goes, (head + count + at) % cap, cap)
    ring = torch.cat([ring, ring[:1]]).scatter(0, place.flatten(), bt.flatten())[:cap]
    count = count + back.sum()
    # new blocks in sequence order from its front
    base, n = s["context"].long(), s["new"].long()
    total = base + n
    need = ((total + bs - 1) // bs - kept).clamp(min=0)
    first = need.cumsum(0) - need
    j = col - kept[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    bt = torch.where(fresh, ring[(head + first[:, None] + j.clamp(min=0)) % cap], bt)
    used = need.sum()
    query_start = torch.cat([n.new_zeros(1), n.cumsum(0)]).int()
    seq, i, live = _rows(query_start, rows)
    pos = base[seq] + i
    slots = bt[seq, (pos // bs).clamp(max=width - 1)].long() * bs + pos % bs
    place, mask = i, s["mask"]
    if c["tree"]:
        mask, place = _ancestors(s["parents"], query_start, 2)
        mask = torch.where(live[:, None], mask, 0)
    positions = torch.where(live, base[seq] + place, 0).int()
    return [bt, ring, (kept + need).int(), torch.stack([(head + used) % cap, count - used]).int(),
            total.int(), query_start, torch.where(live, slots, -1), positions, mask,
            torch.zeros_like(s["status"])]


def _turn(x, cos, sin, rot, adjacent):
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if adjacent else (y[..., : rot // 2], y[..., rot // 2: rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if adjacent else torch.cat([u, w], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _stored(x, like, scales, zeros):
    """Values as a cache holds them: cast, or quantised with the destination's scale."""
    if scales is None:
        return x.to(like)
    y = x / scales[..., None]
    if zeros is None:
        return y.clamp(-448, 448).to(like).view(torch.uint8)
    return (y.round() + zeros[..., None]).clamp(-128, 127).to(like)


def _put(cache, blk, off, live, x, scales, zeros):
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    sc, zp = (None if p is None else p[blk] for p in (scales, zeros))
    raw[blk, :, off] = torch.where(live[..., None, None], _stored(x, cache.dtype, sc, zp),
                                   raw[blk, :, off])


def _plain_rotary(s):
    c = s["case"]
    angle = (s["positions"].double()[s["axis"]] * s["inv_freq"].double()[:, None]).T[:, None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    live = s["slots"] >= 0
    # padding rows rewrite what the last slot, which no token has, holds already
    slot = torch.where(live, s["slots"], s["k_cache"].shape[0] * c["bs"] - 1)
    blk, off = slot // c["bs"], slot % c["bs"]
    q = _turn(s["q"], cos, sin, c["rot"], c["adjacent"]).to(s["q"].dtype)
    k = _turn(s["k"], cos, sin, c["rot"], c["adjacent"])
    _put(s["k_cache"], blk, off, live, k, s["k_scales"], s["k_zeros"])
    _put(s["v_cache"], blk, off, live, s["v"].float(), s["v_scales"], s["v_zeros"])
    return [torch.where(live[:, None, None], q, 0.0)] + _shown(s)


def _plain_accept(s):
    c = s["case"]
    S, N, A, total = c["seqs"], s["max_query"], c["deep"], s["parents"].numel()
    qs = s["query_start"].long()
    n = qs[1:] - qs[:-1]
    i = torch.arange(N, device="cuda")
    at = (qs[:-1, None] + i).clamp(max=total - 1)
    there = i < n[:, None]
    parents, draft, target = s["parents"].long()[at], s["draft"][at], s["target"][at]
    cur, alive = torch.zeros(S, 1, dtype=torch.int64, device="cuda"), n[:, None] > 0
    path, last = [], torch.full((S, 1), -1, device="cuda")
    for _ in range(A):  # one node of the path a round
        path.append(torch.where(alive, cur, -1))
        want = target.gather(1, cur)
        last = torch.where(alive, want, last)
        fits = (parents == cur) & (draft == want) & there
        child = torch.where(fits, i, N).amin(1, keepdim=True)
        alive = alive & (child < N)
        cur = torch.where(alive, child, cur)
    accepted = torch.cat(path, 1)
    count = (accepted >= 0).sum(1)
    base = s["context_lens"].long() - n
    # all moved rows are read before the first is written
    live = accepted >= 0
    spare = (s["k_cache"].shape[0] - 1) * c["bs"]

    def where_is(pos):
        width = s["block_tables"].shape[1]
        b = s["block_tables"].long().gather(1, (pos // c["bs"]).clamp(max=width - 1))
        slot = torch.where(live, b * c["bs"] + pos % c["bs"], spare)
        return slot // c["bs"], slot % c["bs"]

    src = where_is(base[:, None] + accepted.clamp(min=0))
    dst = where_is(base[:, None] + torch.arange(A, device="cuda"))
    for name in "kv":
        cache, sc, zp = s[name + "_cache"], s[name + "_scales"], s[name + "_zeros"]
        x = _values(cache, *src, sc, zp)
        if sc is None:
            _put(cache, *dst, live, x, sc, zp)
            continue
        # codes move as they are between blocks of one scale (and zero point)
        raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        codes, old = raw[src[0], :, src[1]], raw[dst[0], :, dst[1]]
        same = sc[src[0]] == sc[dst[0]]
        if zp is not None:
            same = same & (zp[src[0]] == zp[dst[0]])
        new = _stored(x, cache.dtype, sc[dst[0]], None if zp is None else zp[dst[0]])
        raw[dst[0], :, dst[1]] = torch.where(live[..., None, None],
                                             torch.where(same[..., None], codes, new), old)
    return [accepted.int(), count.int(), last[:, 0], (base + count).int()] + _shown(s)


# ---------------------------------------------------------------------------------------
# what a pass cannot do without, and its results in 64 bits
# ---------------------------------------------------------------------------------------
_SIZE = {"bf16": 2, "fp8": 1, "int8": 1}
_PARAMS = {"bf16": 0, "fp8": 4, "int8": 8}  # scale and zero point of a (block, kv head)


def work(case):
    c = case
    if c["op"] == "rotary":
        t = c["tokens"] - min(c["pad"], c["tokens"] - 1)
        b = t * (2 * c["hq"] * D * 2 + 2 * c["hkv"] * D * (2 + _SIZE[c["kv"]])
                 + 4 * c["axes"] + 2 * _PARAMS[c["kv"]] * c["hkv"] // c["bs"])
        return {"bytes": b + 8 * c["tokens"], "flops": 3 * t * (c["hq"] + c["hkv"]) * c["rot"]}
    base, new = _lens(c)
    total = sum(new)
    if c["op"] == "build":
        fresh = sum(-(-(b + n) // c["bs"]) - -(-b // c["bs"]) for b, n in zip(base, new))
        tree = 4 + 8 if c["tree"] else 0
        return {"bytes": total * (8 + 4 + tree) + c["seqs"] * (4 * 4 + 4 * 4) + 8 * fresh,
                "flops": total}
    if c["op"] == "accept":
        moved = c["seqs"] * min(c["deep"], 2) * 2 * c["hkv"] * D * _SIZE[c["kv"]]
        return {"bytes": total * (4 + 8 + 8) + c["seqs"] * (4 * c["deep"] + 24) + 2 * moved,
                "flops": total}
    blocks = sum(-(-(b + n) // c["bs"]) for b, n in zip(base, new))
    keys = sum(b + n for b, n in zip(base, new))
    return {"bytes": keys * 2 * c["hkv"] * D * _SIZE[c["kv"]]
            + blocks * (4 + 2 * c["hkv"] * _PARAMS[c["kv"]])
            + total * (c["hq"] * (2 * D * 2 + 4) + 8) + 8 * c["seqs"],
            "flops": 4 * D * c["hq"] * sum(n * (b + 1) for b, n in zip(base, new))}


def exact(case, seed):
    c = case
    if c["op"] == "build":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"tree": _exact_tree, "rotary": _exact_rotary, "accept": _exact_accept}[c["op"]](c, s)


def _exact_value(cache, b, off, scales, zeros):
    raw = cache.view(torch.uint8)[b, :, off].view(torch.float8_e4m3fn) if cache.dtype == torch.float8_e4m3fn else cache[b, :, off]
    x = raw.double()
    if zeros is not None:
        x = x - zeros[b].double()[..., None]
    return x if scales is None else x * scales[b].double()[..., None]


def _exact_tree(c, s):
    G = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    qs, lens, par = s["query_start"].tolist(), s["context_lens"].tolist(), s["parents"].tolist()
    for k in range(c["seqs"]):
        r0, r1, ctx = qs[k], qs[k + 1], lens[k]
        n = r1 - r0
        if n == 0:
            continue
        see = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):  # a parent comes before its children
            if par[r0 + i] >= 0:
                see[i] = see[par[r0 + i]]
            see[i, i] = True
        t = torch.arange(ctx, device="cuda")
        b = s["block_tables"][k].long()[t // c["bs"]]
        keys = _exact_value(s["k_cache"], b, t % c["bs"], s["k_scales"], s["k_zeros"])
        vals = _exact_value(s["v_cache"], b, t % c["bs"], s["v_scales"], s["v_zeros"])
        for h in range(c["hkv"]):
            q = s["q"][r0:r1, h * G:(h + 1) * G].double()
            z = s["scale"] * torch.einsum("ngd,td->ngt", q, keys[:, h])
            z[:, :, ctx - n:] = torch.where(see.cuda()[:, None, :], z[:, :, ctx - n:], -math.inf)
            lse[r0:r1, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[r0:r1, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), vals[:, h])
    return out, lse


def _exact_held(s, n):
    """What a pool holds, in 64 bits: fp8 in units of its scales, int8 as values."""
    x = s[n + "_cache"].double()
    if s["k_zeros"] is None:
        return x
    return (x - s[n + "_zeros"].double()[:, :, None, None]) * s[n + "_scales"].double()[:, :, None, None]


def _exact_to(s, n, x, b):
    """Values x [rows, kv heads, D] as blocks b hold them (fp8 unrounded, within its range)."""
    if s["k_scales"] is None:
        return x
    sc = s[n + "_scales"][b].double()[..., None]
    if s["k_zeros"] is None:
        return (x / sc).clamp(-448, 448)
    z = s[n + "_zeros"][b].double()[..., None]
    return ((x / sc).round().add(z).clamp(-128, 127) - z) * sc


def _exact_rotary(c, s):
    half = c["rot"] // 2
    bounds = [sum(s["sections"][: a + 1]) for a in range(c["axes"])]
    axis = [next(a for a, e in enumerate(bounds) if i < e) for i in range(half)]
    # the angles as complex numbers of length one
    theta = s["positions"][axis].double().T * s["inv_freq"].double()[None, :]
    spin = torch.polar(torch.ones_like(theta), theta)

    def turned(x):
        x = x.double()
        pair = x[..., : c["rot"]]
        pair = pair.unflatten(-1, (half, 2)) if c["adjacent"] else pair.unflatten(-1, (2, half)).transpose(-1, -2)
        y = torch.view_as_real(torch.complex(pair[..., 0], pair[..., 1]) * spin[:, None, :])
        y = y.flatten(-2) if c["adjacent"] else y.transpose(-1, -2).flatten(-2)
        return torch.cat([y, x[..., c["rot"]:]], -1)

    live = (s["slots"] >= 0).nonzero()[:, 0]
    b, off = s["slots"][live] // c["bs"], s["slots"][live] % c["bs"]
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    q[live] = turned(s["q"])[live]
    pools = []
    for n, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        pool = _exact_held(s, n)
        pool[b, :, off] = _exact_to(s, n, x[live], b)
        pools.append(pool)
    return [q] + pools


def _exact_accept(c, s):
    qs, lens = s["query_start"].tolist(), s["context_lens"].tolist()
    par, draft, target = s["parents"].tolist(), s["draft"].tolist(), s["target"].tolist()
    bt = s["block_tables"].tolist()
    moves = []
    for k in range(c["seqs"]):
        r0, n = qs[k], qs[k + 1] - qs[k]
        base, cur, path = lens[k] - n, 0, []
        while n and len(path) < c["deep"]:
            path.append(cur)
            nxt = [i for i in range(n) if par[r0 + i] == cur and draft[r0 + i] == target[r0 + cur]]
            if not nxt:
                break
            cur = nxt[0]
        for i, node in enumerate(path):
            f, t = base + node, base + i
            moves.append((bt[k][f // c["bs"]], f % c["bs"], bt[k][t // c["bs"]], t % c["bs"]))
    m = torch.tensor(moves, device="cuda")
    pools = []
    for n in "kv":
        pool = _exact_held(s, n)
        x = _exact_value(s[n + "_cache"], m[:, 0], m[:, 1], s[n + "_scales"], s[n + "_zeros"])
        pool[m[:, 2], :, m[:, 3]] = _exact_to(s, n, x, m[:, 2])
        pools.append(pool)
    return [None] * 4 + pools

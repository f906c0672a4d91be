"""GPU tests of the operators of a drafted step against the float64 oracle (oracle/drafted.py).

Bookkeeping, cache contents and moved rows are exact. Attention and rotary outputs are held
to bounds derived from the formats' roundings (half a step: bf16 2^-8, fp32 2^-24, E4M3 2^-4
relative, int8 half a code) and the arithmetic of the path, element by element:

* attention, weights w_t = softmax, A = sum w_t |V_t|: a score's products and sums in float32
  move it by at most dz = 2 (d + 4) 2^-24 scale sum |q K| (a tensor-core sum may drop what a
  rounding would keep, hence the 2), its exponent's argument by 2^-22 of its size (at most
  2^-16 for |z| below 64) and the approximate exponential by 2^-21; both numerator and
  denominator feel that, and their sums round 2^-24 per key: E = 2 (e^dz - 1 + 2^-16 + 2^-21) +
  ctx 2^-23. The tensor-core path also rounds each weight to bf16: 2^-8. The output is rounded
  once: |out - ref| <= (2^-8 + E) A + 2^-8 |ref|, with 2^-24 and no 2^-8 A on the fp32 path.
* lse: |dz| + 2^-15 + ctx 2^-23 + 2^-21 |lse|.
* rotary: the reduced angle is off by 2^-24 of a turn (3.8e-7), sin and cos by 2^-23, each
  product and sum by 2^-24: 2^-20 (|x| + |y|) covers them, then one rounding of the format.
"""
import math

import numpy as np
import pytest

from oracle import drafted
from oracle.codecs import e4m3_decode, int8_decode
from tests.gpu_common import cache_codes, to_f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_465_b200 as pa
    pa.set_decode_impl("auto")
    assert pa.device_error() == 0
    yield pa
    pa.set_decode_impl("auto")


def cuda(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def random_parents(rng, n):
    """Half the rows hang on the row before them, the others anywhere before; row 0 on none."""
    return [-1] + [i - 1 if rng.random() < 0.5 else int(rng.integers(0, i)) for i in range(1, n)]


# ---------------------------------------------------------------------------------------
# block tables, slot maps, masks
# ---------------------------------------------------------------------------------------
def build(pa, context, new, held, tables, ring, queue, B, nb, rows, parents=None, words=0):
    S = len(context)
    o = dict(total_lens=cuda(np.full(S, -7)), query_start=cuda(np.full(S + 1, -7)),
             blocks_held_out=cuda(np.full(S, -7)), queue_state_out=cuda([-7, -7]),
             slot_mapping=cuda(np.full(rows, -7), torch.int64), positions=cuda(np.full(rows, -7)),
             status=cuda([-7]))
    if words:
        o["tree_mask"] = cuda(np.full((rows, words), -7))
    bt = cuda(tables)
    pa.build_step(cuda(context), cuda(new), cuda(held), bt, cuda(ring), cuda(queue), block_size=B,
                  num_blocks=nb, parents=None if parents is None else cuda(parents), **o)
    return bt.cpu().numpy(), {k: v.cpu().numpy() for k, v in o.items()}


def queue_case(rng, S, B, ctx_hi, new_hi, spare=1):
    """Random lengths with their tables over a shuffled pool, the rest of it in a ring that wraps."""
    context = rng.integers(0, ctx_hi + 1, S)
    new = rng.integers(0, new_hi + 1, S)
    held = -(-context // B) + rng.integers(0, spare + 1, S)
    width = int(max(held.max(), (-(-(context + new) // B)).max())) + 1
    nb = int(held.sum()) + int((-(-(context + new) // B)).sum()) + 3
    perm = rng.permutation(nb)
    tables = np.full((S, width), -1)
    at = 0
    for s in range(S):
        tables[s, :held[s]] = perm[at:at + held[s]]
        at += held[s]
    head, count = nb - 2, nb - at
    ring = np.full(nb, -1)
    ring[(head + np.arange(count)) % nb] = perm[at:]
    return context, new, held, tables, ring, [head, count], nb


@pytest.mark.parametrize("S,B,ctx,new,rows_more", [
    (1, 16, 40, 1, 0), (1, 8, 0, 1, 5), (3, 32, 100, 5, 2), (64, 16, 300, 1, 0),
    (257, 8, 90, 64, 13), (1500, 16, 60, 3, 1), (5, 16, 50, 4000, 100), (2100, 32, 40, 2, 0)])
@pytest.mark.parametrize("tree", [False, True])
def test_build_step(pa, S, B, ctx, new, rows_more, tree):
    rng = np.random.default_rng(S * 1000 + B)
    context, n, held, tables, ring, queue, nb = queue_case(rng, S, B, ctx, new)
    rows = int(n.sum()) + rows_more
    if rows == 0:
        n[0], rows = 1, 1
    words = 0 if n.max() > 256 else int(-(-max(int(n.max()), 1) // 32))
    parents = None
    if tree:
        parents = sum((random_parents(rng, k) for k in n if k), []) + [123456] * (rows - int(n.sum()))
    ref = drafted.ref_build_step(context, n, held, tables, ring, queue, B, nb, rows, parents, words)
    bt, o = build(pa, context, n, held, tables, ring, queue, B, nb, rows, parents, words)
    assert pa.device_error() == 0 and o["status"][0] == 0
    names = ("blocks_held_out", "queue_state_out", "total_lens", "query_start", "slot_mapping",
             "positions")
    assert np.array_equal(bt, ref[0])
    for k, r in zip(names, ref[1:7]):
        assert np.array_equal(o[k], r), k
    if words:
        assert np.array_equal(o["tree_mask"], ref[7])


def test_build_step_whole_queue_and_no_tokens(pa):
    """The last free block may be taken; a step of no tokens changes nothing."""
    t = np.array([[3, -1, -1], [5, -1, -1]])
    bt, o = build(pa, [16, 10], [17, 6], [1, 1], t, [0, 1, 2, 4], [2, 2], 16, 6, 23, words=1)
    assert pa.device_error() == 0 and o["status"][0] == 0
    assert bt.tolist() == [[3, 2, 4], [5, -1, -1]] and o["queue_state_out"].tolist() == [0, 0]
    bt, o = build(pa, [16, 10], [0, 0], [1, 1], t, [0, 1, 2, 4], [2, 2], 16, 6, 4, words=1)
    assert pa.device_error() == 0 and np.array_equal(bt, t)
    assert o["slot_mapping"].tolist() == [-1] * 4 and o["query_start"].tolist() == [0, 0, 0]
    assert not o["positions"].any() and not o["tree_mask"].any()


@pytest.mark.parametrize("rows", [0, 5, 2500])
@pytest.mark.parametrize("words", [0, 2])
def test_build_step_of_no_sequences(pa, rows, words):
    """An idle step of fixed width writes every output: no slot, no rows, the queue as it was."""
    none = np.zeros(0)
    bt, o = build(pa, none, none, none, np.zeros((0, 3)), [4, 1, 0, 2], [3, 2], 16, 6, rows, words=words)
    assert pa.device_error() == 0 and o["status"].tolist() == [0]
    assert o["query_start"].tolist() == [0] and o["queue_state_out"].tolist() == [3, 2]
    assert (o["slot_mapping"] == -1).all() and not o["positions"].any()
    assert not words or not o["tree_mask"].any()
    _, o = build(pa, none, none, none, np.zeros((0, 3)), [4, 1, 0, 2], [4, 2], 16, 6, rows, words=words)
    assert pa.device_error() == 0x200 and o["status"].tolist() == [0x200]
    assert (o["slot_mapping"] == -1).all() and o["queue_state_out"].tolist() == [4, 2]


def test_release_blocks_of_no_sequences(pa):
    """The queue is passed on: a program that chains queue states does not go back to an old one."""
    ring, out, status = cuda([4, 1, 0, 2]), cuda([-7, -7]), cuda([-7])
    pa.release_blocks(cuda([]), cuda([]), cuda(np.zeros((0, 3))), ring, cuda([3, 2]), block_size=16,
                      blocks_held_out=cuda([]), queue_state_out=out, status=status)
    assert out.tolist() == [3, 2] and status.tolist() == [0] and ring.tolist() == [4, 1, 0, 2]
    assert pa.device_error() == 0


def test_an_idle_step_writes_nothing_to_the_cache(pa):
    """A fixed-width step of two sequences, then one of none into the same buffers: the second
    step's rows reach no cache row."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = lambda h: torch.randn(4, h, 64, device="cuda", generator=g).bfloat16()  # noqa: E731
    kc, vc = (torch.randn(6, 2, 16, 64, device="cuda", generator=g).bfloat16() for _ in range(2))
    o = dict(query_start=cuda(np.full(3, -7)), queue_state_out=cuda([-7, -7]),
             slot_mapping=cuda(np.full(4, -7), torch.int64), positions=cuda(np.full(4, -7)))

    def step(S, queue):
        new = {n: cuda(np.full(S, -7)) for n in ("total_lens", "blocks_held_out")}
        pa.build_step(cuda([16, 3][:S]), cuda([1, 2][:S]), cuda([1, 1][:S]), cuda(np.array([[3, -1], [5, -1]])[:S]),
                      cuda([4, 1, 0, 2]), queue, block_size=16, num_blocks=6, **new,
                      **dict(o, query_start=o["query_start"][:S + 1]))
        pa.rotary_and_cache(x(4), x(2), x(2), x(4), kc, vc, o["positions"], o["slot_mapping"],
                            torch.ones(32, device="cuda"))
    step(2, cuda([3, 2]))
    assert o["slot_mapping"].tolist() == [32, 83, 84, -1] and o["queue_state_out"].tolist() == [0, 1]
    before, queue = (kc.clone(), vc.clone()), o["queue_state_out"].clone()
    step(0, queue)
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    assert torch.equal(o["queue_state_out"], queue) and pa.device_error() == 0


@pytest.mark.parametrize("why,bit", [("blocks", 0x100), ("rows", 0x20), ("one_too_long", 0x80), ("queue_head", 0x200),
                                     ("queue_count", 0x200), ("negative", 0x8), ("table", 0x8),
                                     ("held", 0x8), ("wide", 0x80)])
def test_build_step_refuses_as_a_whole(pa, why, bit):
    S, B, nb, rows = 300, 16, 2000, 1200
    context, n = np.full(S, 16), np.full(S, 3)
    held, tables = np.ones(S, dtype=int), np.full((S, 4), -1)
    tables[:, 0] = np.arange(S)
    ring, queue = np.arange(nb), [5, 400]
    if why == "blocks":
        queue = [5, 299]
    elif why == "rows":
        n[:] = 4
        n[150] = 5
    elif why == "one_too_long":   # for the mask (256), and for the rows with it
        n[7] = 304
        tables = np.pad(tables, ((0, 0), (0, 40)), constant_values=-1)
    elif why == "queue_head":
        queue = [nb, 400]
    elif why == "queue_count":
        queue = [0, nb + 1]
    elif why == "negative":
        n[299] = -1
    elif why == "table":
        n[200] = 49
    elif why == "held":
        context[100] = 17
    elif why == "wide":
        n[33] = 33
    bt, o = build(pa, context, n, held, tables, ring, queue, B, nb, rows, words=1 if why == "wide" else 8)
    assert pa.device_error() == bit and o["status"][0] == bit
    assert np.array_equal(bt, tables) and np.array_equal(o["blocks_held_out"], held)
    assert o["queue_state_out"].tolist() == queue and np.array_equal(o["total_lens"], context)
    assert not o["query_start"].any() and (o["slot_mapping"] == -1).all()
    assert not o["positions"].any() and not o["tree_mask"].any()
    assert pa.device_error() == 0


def test_build_step_flags_bad_rows(pa):
    """A parent not before its child and a block id outside the pool are recorded; the other
    rows are not affected."""
    t = np.array([[2, -1], [77, -1]])
    bt, o = build(pa, [14, 3], [4, 2], [1, 1], t, [900, 1, 2, 3], [0, 3], 16, 5, 7,
                  [-1, 3, 0, 2, -1, -9, 0], 1)
    assert pa.device_error() == 0x80 | 0x1 and o["status"][0] == 0
    assert o["slot_mapping"].tolist() == [46, 47, -1, -1, -1, -1, -1]
    assert o["positions"].tolist() == [14, 14, 15, 16, 3, 3, 0]
    assert o["tree_mask"][:, 0].tolist() == [1, 2, 5, 13, 1, 2, 0]
    assert bt.tolist() == [[2, 900], [77, -1]]


@pytest.mark.parametrize("S,B,ctx", [(1, 16, 100), (64, 8, 300), (65, 16, 50), (1500, 32, 200),
                                     (9500, 16, 20)])
def test_release_blocks(pa, S, B, ctx):
    rng = np.random.default_rng(S)
    context, _, held, tables, ring, queue, nb = queue_case(rng, S, B, ctx, 0, spare=2)
    keep = np.where(rng.random(S) < 0.4, 0, rng.integers(0, ctx + 40, S))
    ref = drafted.ref_release(keep, held, tables, ring, queue, B)
    rg, ho, qo, st = cuda(ring), cuda(np.full(S, -7)), cuda([-7, -7]), cuda([-7])
    pa.release_blocks(cuda(keep), cuda(held), cuda(tables), rg, cuda(queue), block_size=B,
                      blocks_held_out=ho, queue_state_out=qo, status=st)
    assert pa.device_error() == 0 and st.item() == 0
    for got, r in zip((rg, ho, qo), ref):
        assert np.array_equal(got.cpu().numpy(), r)


@pytest.mark.parametrize("why,bit", [("negative", 0x8), ("held", 0x8), ("full", 0x200), ("head", 0x200)])
def test_release_blocks_refuses_as_a_whole(pa, why, bit):
    keep, held, tables = [0, 16, 5], [2, 2, 1], np.arange(9).reshape(3, 3)
    ring, queue = np.arange(6), [4, 3]
    if why == "negative":
        keep = [0, -1, 5]
    elif why == "held":
        held = [2, 4, 1]
    elif why == "full":
        queue = [4, 4]
    else:
        queue = [-1, 3]
    rg, ho, qo, st = cuda(ring), cuda([-7] * 3), cuda([-7, -7]), cuda([-7])
    pa.release_blocks(cuda(keep), cuda(held), cuda(tables), rg, cuda(queue), block_size=16,
                      blocks_held_out=ho, queue_state_out=qo, status=st)
    assert pa.device_error() == bit and st.item() == bit
    assert rg.tolist() == list(ring) and ho.tolist() == held and qo.tolist() == queue


def test_bookkeeping_refuses_shared_buffers(pa):
    z = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    held, queue, slots = z(2), z(2), torch.zeros(4, dtype=torch.int64, device="cuda")
    def go(**kw):
        a = dict(total_lens=z(2), query_start=z(3), blocks_held_out=z(2), queue_state_out=z(2),
                 slot_mapping=slots, positions=z(4))
        a.update(kw)
        pa.build_step(z(2), z(2), held, z(6).view(2, 3), z(9), queue, block_size=16, num_blocks=9, **a)
    for kw in (dict(blocks_held_out=held), dict(queue_state_out=queue), dict(total_lens=held),
               dict(positions=slots.view(torch.int32)[4:])):
        with pytest.raises(pa.PagedAttnError):
            go(**kw)
    for kw in (dict(query_start=z(2)), dict(positions=z(3)), dict(status=z(2)),
               dict(tree_mask=z(4).view(4, 1).t()), dict(total_lens=z(4)[::2])):
        with pytest.raises(ValueError):
            go(**kw)
    with pytest.raises(TypeError):
        go(slot_mapping=z(4))
    with pytest.raises(pa.PagedAttnError):
        pa.release_blocks(z(2), held, z(6).view(2, 3), z(9), queue, block_size=16,
                          blocks_held_out=held, queue_state_out=z(2))


# ---------------------------------------------------------------------------------------
# rotary positions with the cache write
# ---------------------------------------------------------------------------------------
def pool(rng, kv, nb, hkv, B, d):
    """Random pool codes with scales and zero points that differ from block to block."""
    o = dict(k_scales=None, v_scales=None, k_zeros=None, v_zeros=None)
    for n in "kv":
        x = rng.standard_normal((nb, hkv, B, d)).astype(np.float32)
        if kv in ("fp8", "int8"):
            o[n + "_scales"] = ((3.0 + 2 * rng.random((nb, hkv))) / (448 if kv == "fp8" else 128)
                                ).astype(np.float32)
        if kv == "int8":
            o[n + "_zeros"] = rng.integers(-20, 21, (nb, hkv)).astype(np.int32)
        sc, zp = (None if o[n + p] is None else o[n + p][:, :, None, None] for p in ("_scales", "_zeros"))
        o[n] = drafted.stored_codes(x, kv, sc, zp)
    return o


def on_gpu(o):
    """The pool of ``pool`` as the library's tensors."""
    def codes(x):
        t = torch.from_numpy(np.ascontiguousarray(x.view(np.int16) if x.dtype == np.uint16 else x).copy())
        return (t.view(torch.bfloat16) if x.dtype == np.uint16 else t).cuda()
    side = {k: None if o[k] is None else torch.from_numpy(o[k].copy()).cuda()
            for k in ("k_scales", "v_scales", "k_zeros", "v_zeros")}
    return codes(o["k"]), codes(o["v"]), side


def rotary_case(pa, indt, kv, T, hq, hkv, d, rot, sections, adjacent, B, far, layout="rows", pad=2):
    rng = np.random.default_rng(T * 7 + rot + d)
    dt = torch.float32 if indt == "f32" else torch.bfloat16
    nb = -(-T // B) + 2
    o = pool(rng, kv, nb, hkv, B, d)
    kc, vc, side = on_gpu(o)
    x = torch.randn(T, hq + 2 * hkv, d, generator=torch.Generator().manual_seed(T)).to(dt).cuda()
    if layout == "projection":   # q, k and v are slices of one projection's rows
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (y.contiguous() for y in (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]))
    slots = rng.permutation(nb * B)[:T].astype(np.int64)
    slots[rng.permutation(T)[:min(pad, T - 1)]] = -1 - rng.integers(0, 5)
    live = slots >= 0
    pos = rng.integers(-far if far < 100 else 0, far, (len(sections), T)).astype(np.int32)
    inv = (1.0 / 10000.0 ** (np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    ref_q, ref_k = (drafted.ref_turn(to_f64(y), pos, inv, sections, adjacent) for y in (q, k))
    size = lambda y: 2.0 ** -20 * (np.abs(to_f64(y)).max(-1, keepdims=True) * 2)  # noqa: E731
    sq, sk, v64 = size(q), size(k), to_f64(v).astype(np.float32)
    if layout == "in place":
        q_out = q
        before = q.clone()
    else:
        q_out = torch.full_like(q.contiguous(), 7.0)
        before = q_out.clone()
    pa.rotary_and_cache(q, k, v, q_out, kc, vc, cuda(pos if len(sections) > 1 else pos[0]),
                        cuda(slots, torch.int64), cuda(inv, torch.float32),
                        sections=None if len(sections) == 1 else sections, adjacent_pairs=adjacent,
                        **side)
    assert pa.device_error() == 0
    err = np.abs(to_f64(q_out) - ref_q)[live]
    assert (err <= (sq + (F32 if indt == "f32" else BF16) * np.abs(ref_q))[live]).all()
    assert torch.equal(q_out[~torch.from_numpy(live).cuda()], before[~torch.from_numpy(live).cuda()])
    # the cache: v bit for bit; k within the roundings of its format; everything else untouched
    for name, got, x64 in (("k", cache_codes(kc), ref_k), ("v", cache_codes(vc), None)):
        b, off = slots[live] // B, slots[live] % B
        new = got[b, :, off]
        sc, zp = (None if o[name + p] is None else o[name + p][b][..., None] for p in ("_scales", "_zeros"))
        if name == "v":
            assert np.array_equal(new, drafted.stored_codes(v64[live], kv, sc, zp))
        else:
            x, tol = x64[live], sk[live]
            if kv == "f32":
                assert (np.abs(new - x) <= tol + F32 * np.abs(x)).all()
            elif kv == "bf16":
                val = (new.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
                assert (np.abs(val - x) <= tol + BF16 * np.abs(x)).all()
            elif kv == "fp8":
                y = np.clip(x / sc, -448, 448)
                step = np.maximum(E4M3 * np.abs(y), 2.0 ** -10)
                assert (np.abs(e4m3_decode(new) - y) <= step * (1 + 1e-6) + tol / sc).all()
            else:
                y = np.clip(x / sc, -128 - zp, 127 - zp)
                assert (np.abs(int8_decode(new, zp) - y) <= 0.5 + 1e-6 + tol / sc).all()
        got = got.copy()
        got[b, :, off] = o[name][b, :, off]
        assert np.array_equal(got, o[name]), "slots that no token has"


@pytest.mark.parametrize("indt,kv", [("bf16", "bf16"), ("bf16", "fp8"), ("bf16", "int8"), ("f32", "f32"),
                                     ("f32", "bf16"), ("f32", "fp8"), ("f32", "int8")])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_types(pa, indt, kv, adjacent):
    rotary_case(pa, indt, kv, 53, 8, 2, 128, 128, [16, 24, 24], adjacent, 16, 4000)


@pytest.mark.parametrize("T,hq,hkv,d,rot,sections,B", [
    (1, 1, 1, 64, 64, [32], 8), (1, 32, 8, 128, 128, [64], 16), (7, 3, 3, 64, 16, [8], 32),
    (300, 16, 1, 256, 256, [128], 16), (40, 4, 4, 128, 96, [0, 24, 0, 24], 8), (9, 64, 8, 128, 112, [56], 16),
    (5, 2, 1, 256, 48, [1, 23], 32)])
@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_shapes(pa, T, hq, hkv, d, rot, sections, B, adjacent):
    rotary_case(pa, "bf16", "bf16", T, hq, hkv, d, rot, sections, adjacent, B, 4000)


@pytest.mark.parametrize("layout", ["projection", "in place"])
@pytest.mark.parametrize("indt", ["bf16", "f32"])
def test_rotary_layouts(pa, layout, indt):
    rotary_case(pa, indt, "bf16", 33, 8, 2, 128, 64, [32], False, 16, 4000, layout)


@pytest.mark.parametrize("far", [10, 1 << 20, (1 << 31) - 1])
def test_rotary_far_positions(pa, far):
    """The angle of a far position is reduced in float64 (far 10: negative positions too)."""
    rotary_case(pa, "f32", "f32", 64, 2, 1, 64, 64, [32], False, 16, far)


def test_rotary_bad_slots_and_zero_points(pa):
    T, hq, hkv, d, B, nb = 3, 2, 2, 64, 16, 4
    q, k = (torch.randn(T, h, d, device="cuda").bfloat16() for h in (hq, hkv))
    kc, vc = (torch.zeros(nb, hkv, B, d, dtype=torch.int8, device="cuda") for _ in range(2))
    sc, zp = torch.full((nb, hkv), 0.01, device="cuda"), torch.zeros(nb, hkv, dtype=torch.int32, device="cuda")
    zp[1, 1] = 200
    out, inv = torch.zeros_like(q), torch.ones(32, device="cuda")
    slots = cuda([nb * B, 5, B + 5], torch.int64)
    pa.rotary_and_cache(q, k, k, out, kc, vc, cuda([1, 2, 3]), slots, inv, k_scales=sc, v_scales=sc,
                        k_zeros=zp, v_zeros=zp)
    assert pa.device_error() == pa.PA_DEVERR_SLOT | pa.PA_DEVERR_ZERO
    assert not out[0].any() and out[1:].any()
    assert kc[0, :, 5].any() and kc[1, 0, 5].any() and not kc[1, 1].any() and not kc[2:].any()
    with pytest.raises(ValueError):
        pa.rotary_and_cache(q, k, k, q.flatten()[8:].new_zeros(1).expand(T, hq, d), kc, vc, cuda([1, 2, 3]),
                            slots, inv, k_scales=sc, v_scales=sc, k_zeros=zp, v_zeros=zp)
    buf = torch.zeros(T * hq * d + 64, device="cuda").bfloat16()
    with pytest.raises(pa.PagedAttnError):   # q_out overlaps q without being q
        pa.rotary_and_cache(buf[:T * hq * d].view(T, hq, d), k, k, buf[64:].view(T, hq, d), kc, vc,
                            cuda([1, 2, 3]), slots, inv, k_scales=sc, v_scales=sc, k_zeros=zp, v_zeros=zp)


# ---------------------------------------------------------------------------------------
# tree attention
# ---------------------------------------------------------------------------------------
class Tree:
    """A step's tensors: context of base[s] tokens and new[s] rows per sequence."""

    def __init__(self, seed, base, new, hq, hkv, d, B, kv, parents=True, see=None, pad=2, words=None):
        rng = self.rng = np.random.default_rng(seed)
        self.base, self.new, self.hq, self.hkv, self.d, self.B, self.kv = base, new, hq, hkv, d, B, kv
        S = len(base)
        self.ctx = np.array(base) + np.array(new)
        self.qs = np.concatenate([[0], np.cumsum(new)])
        self.T = int(self.qs[-1]) + pad
        need = -(-self.ctx // B)
        nb = int(need.sum()) + 2
        perm = rng.permutation(nb)
        self.bt = np.full((S, int(max(need.max(), 1)) + 1), -1)
        at = 0
        for s in range(S):
            self.bt[s, :need[s]] = perm[at:at + need[s]]
            at += need[s]
        self.o = pool(rng, kv, nb, hkv, B, d)
        self.see = see if see is not None else [drafted.ref_ancestors(random_parents(rng, n) if n else [])
                                                for n in new]
        self.words = words or max(1, -(-max(new) // 32))
        self.scale = 1 / math.sqrt(d)
        f32 = kv == "f32"
        q = torch.randn(self.T, hq, d, generator=torch.Generator().manual_seed(seed))
        self.q = q.cuda() if f32 else q.bfloat16().cuda()
        self.max_q, self.max_ctx = max(new), int(self.ctx.max())
        self.device()

    def device(self):
        self.kc, self.vc, self.side = on_gpu(self.o)
        rows = [js for s in self.see for js in s]
        self.mask = cuda(np.concatenate([drafted.mask_words(rows, self.words) if rows else
                                         np.zeros((0, self.words), dtype=np.int32),
                                         np.full((self.T - len(rows), self.words), -1)]))
        self.dbt, self.dctx, self.dqs = cuda(self.bt), cuda(self.ctx), cuda(self.qs)

    def workspace(self, pa):
        n = pa.tree_workspace_size(self.q, self.kc, self.dbt, max_query_len=self.max_q,
                                   max_context_len=self.max_ctx)
        return torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere

    def run(self, pa, impl="auto", out=None, lse=None, ws=None):
        out = torch.full_like(self.q, 3.0) if out is None else out
        lse = torch.full((self.T, self.hq), 3.0, device="cuda") if lse is None else lse
        pa.set_decode_impl(impl)
        try:
            pa.paged_attn_tree(self.q, self.kc, self.vc, self.dbt, self.dctx, self.dqs, self.mask, self.scale,
                               out, max_query_len=self.max_q, max_context_len=self.max_ctx, lse_out=lse,
                               workspace=self.workspace(pa) if ws is None else ws, **self.side)
        finally:
            pa.set_decode_impl("auto")
        return out, lse

    def ref(self):
        q = self.q.cpu()
        codes = q.numpy() if self.kv == "f32" else q.view(torch.int16).numpy().view(np.uint16)
        with np.errstate(invalid="ignore"):
            return drafted.ref_tree(codes, self.qs, self.see, self.o["k"], self.o["v"], self.bt, self.ctx,
                                    self.scale, self.hkv, "f32" if self.kv == "f32" else "bf16", self.kv,
                                    self.o["k_scales"], self.o["v_scales"], self.o["k_zeros"], self.o["v_zeros"])

    def check(self, pa, impl="auto", got=None):
        out, lse = self.run(pa, impl) if got is None else got
        assert pa.device_error() == 0
        ref, rl, absv, big = self.ref()
        n = int(self.qs[-1])
        assert (out[n:] == 3).all() and (lse[n:] == 3).all(), "rows behind the last sequence"
        o, l = to_f64(out)[:n], to_f64(lse)[:n]
        dz = (2 * (self.d + 4) * F32 * big[:n])
        ctx = np.repeat(self.ctx, self.new)[:, None]
        E = 2 * (np.expm1(dz) + 2.0 ** -16 + 2.0 ** -21) + ctx * 2.0 ** -23
        tc = impl != "simt" and self.kv != "f32" and self.d == 128 and self.hq // self.hkv in (1, 2, 4, 8, 16)
        rnd = F32 if self.kv == "f32" else BF16
        tol = (E + (BF16 if tc else 0.0))[..., None] * absv[:n] + rnd * np.abs(ref[:n])
        fin = np.isfinite(ref[:n])
        assert np.array_equal(np.isfinite(o), fin)
        assert (np.abs(o - ref[:n])[fin] <= tol[fin] + 1e-30).all(), \
            float((np.abs(o - ref[:n]) / np.maximum(tol, 1e-30))[fin].max())
        fl = np.isfinite(rl[:n])
        assert np.array_equal(l[~fl], rl[:n][~fl], equal_nan=True)
        tl = dz + 2.0 ** -15 + ctx * 2.0 ** -23 + 2.0 ** -21 * np.abs(rl[:n])
        assert (np.abs(l[fl] - rl[:n][fl]) <= tl[fl]).all()
        return out, lse


IMPLS = ["simt", "auto"]


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_tree_types_and_blocks(pa, impl, kv, B):
    """Contexts that end inside blocks and key tiles, one-token trees, sequences without rows."""
    Tree(B, [0, 1, 63, 64, 65, 500, 129, 31], [3, 1, 2, 9, 1, 16, 0, 33], 8, 2, 128, B, kv).check(pa, impl)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (4, 2), (8, 2), (16, 2), (32, 2), (12, 4), (10, 2)])
@pytest.mark.parametrize("impl", IMPLS)
def test_tree_groups(pa, impl, hq, hkv):
    """Groups of 1, 2, 4, 8 and 16 (tensor cores) and 3 and 5 (CUDA cores); several row tiles."""
    Tree(hq, [70, 300, 5], [40, 7, 130], hq, hkv, 128, 16, "bf16").check(pa, impl)


@pytest.mark.parametrize("kv,d", [("f32", 64), ("f32", 128), ("f32", 256), ("bf16", 64), ("bf16", 256),
                                  ("fp8", 64), ("int8", 256)])
def test_tree_other_shapes(pa, kv, d):
    Tree(d, [33, 700, 0], [6, 3, 17], 4, 2, d, 16, kv).check(pa)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_tree_long_context_split(pa, impl, kv):
    """Few sequences with long contexts: every one is cut between many CTAs."""
    Tree(5, [9000, 130], [5, 2], 4, 1, 128, 16, kv).check(pa, impl)


def test_tree_many_sequences(pa):
    """More sequences than a warp holds or a CTA has threads, ragged, many of them idle."""
    rng = np.random.default_rng(0)
    S = 700
    base = rng.integers(0, 90, S).tolist()
    new = np.where(rng.random(S) < 0.4, 0, rng.integers(1, 5, S)).tolist()
    Tree(6, base, new, 8, 2, 128, 16, "bf16").check(pa)
    Tree(7, base, new, 8, 2, 128, 8, "fp8").check(pa)


@pytest.mark.parametrize("impl", IMPLS)
def test_tree_largest_draft(pa, impl):
    """256 rows, eight mask words, beside a single row."""
    Tree(8, [20, 100], [256, 1], 4, 1, 128, 16, "bf16").check(pa, impl)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tree_masks_of_any_kind(pa, impl, kv):
    """Masks need not be a tree's: later rows, not itself, none, all; also a row that sees
    nothing at all (no context either): out 0, lse -inf."""
    rng = np.random.default_rng(3)
    see = [[sorted(rng.permutation(n)[:rng.integers(0, n + 1)].tolist()) for _ in range(n)]
           for n in (70, 5, 66)]
    see[0][0], see[1][2], see[2][65] = [], [], list(range(66))
    t = Tree(9, [200, 0, 62], [70, 5, 66], 8, 2, 128, 16, kv, see=see, words=4)
    out, lse = t.check(pa, impl)
    assert (out[72] == 0).all() and (lse[72] == -math.inf).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tree_nan_and_infinity_where_nobody_looks(pa, impl, kv):
    """NaN and infinities in drafted rows that a row does not see, behind the context, in
    unused blocks and in unseen scales do not reach it; rows that see them get them."""
    see = [[[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4]], [[i] for i in range(40)]]
    t = Tree(10, [59, 130], [5, 40], 8, 2, 128, 16, kv, see=see, pad=1)
    nan, inf = (0x7f, None) if kv == "fp8" else (0x7fc0, 0x7f80)
    at = lambda s, i: (t.bt[s, (t.base[s] + i) // 16], slice(None), (t.base[s] + i) % 16)  # noqa: E731
    t.o["k"][at(0, 3)] = nan
    t.o["v"][at(0, 4)][..., 5] = nan
    t.o["v"][at(1, 7)] = nan
    if inf:
        t.o["v"][at(0, 2)][..., 9] = inf
        t.o["v"][at(0, 1)][..., 9] = inf | 0x8000
        t.o["k"][at(1, 11)] = inf
    used = {int(b) for row in t.bt for b in row if b >= 0}
    for b in set(range(t.o["k"].shape[0])) - used:
        t.o["k"][b] = t.o["v"][b] = nan
    for s in range(2):   # behind the context, in the last block
        b, off = t.bt[s, (t.ctx[s] - 1) // 16], t.ctx[s] % 16
        if off:
            t.o["k"][b, :, off:] = t.o["v"][b, :, off:] = nan
    t.device()
    out, lse = t.run(pa, impl)
    assert pa.device_error() == 0
    ref, rl, *_ = t.ref()
    o, n = to_f64(out), int(t.qs[-1])
    assert np.array_equal(np.isnan(o[:n]), np.isnan(ref[:n]))
    assert np.array_equal(np.isposinf(o[:n]), np.isposinf(ref[:n]))
    assert np.array_equal(np.isneginf(o[:n]), np.isneginf(ref[:n]))
    fin = np.isfinite(ref[:n])
    assert np.abs(o[:n][fin] - ref[:n][fin]).max() <= 2e-2 * 4   # (2^-8 + E) A + 2^-8 |ref|, A <= 4
    assert fin[0].all() and not fin[3].any() and fin[4, :, :5].all() and not fin[4, :, 5].any()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_tree_scale_of_either_sign(pa, impl, scale):
    t = Tree(11, [100, 0], [9, 4], 8, 2, 128, 16, "bf16")
    t.scale = scale
    t.check(pa, impl)


@pytest.mark.parametrize("impl", IMPLS)
def test_tree_rescales_a_growing_maximum(pa, impl):
    """Scores that keep growing along the context make the running maximum move often."""
    t = Tree(12, [700], [6], 8, 2, 128, 16, "bf16")
    k = torch.from_numpy(t.o["k"].view(np.int16)).view(torch.bfloat16).float()
    pos = torch.zeros(k.shape[0], 16)
    for b, blk in enumerate(t.bt[0]):
        if blk >= 0:
            pos[blk] = torch.arange(16) + 16 * b
    k = k * (pos / 100)[:, None, :, None]
    t.o["k"] = k.bfloat16().view(torch.int16).numpy().view(np.uint16)
    t.device()
    t.check(pa, impl)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_tree_bad_blocks_are_skipped_and_flagged(pa, impl, kv):
    """Keys of an unusable block are left out: the result is that of a context without them."""
    t = Tree(13, [160], [4], 8, 2, 128, 16, kv)
    _, whole = t.run(pa, impl)
    assert pa.device_error() == 0
    bt = t.bt.copy()
    bt[0, 3], bt[0, 7] = t.o["k"].shape[0], -5
    t.dbt = cuda(bt)
    out, lse = t.run(pa, impl)
    assert pa.device_error() == pa.PA_DEVERR_BLOCK_ID
    keep = [b for b in range(t.bt.shape[1]) if b not in (3, 7)]
    short = Tree(13, [160], [4], 8, 2, 128, 16, kv)
    short.bt = t.bt[:, keep]
    short.base, short.ctx = [128], np.array([132])
    short.max_ctx = 132
    short.device()
    o2, l2 = short.run(pa, impl)
    assert pa.device_error() == 0
    n = 4   # both are within their bound of one reference, and differ from the whole context's
    assert (lse[:n] < whole[:n]).all()
    assert torch.allclose(out[:n].float(), o2[:n].float(), rtol=4 * BF16, atol=2e-2)
    assert torch.allclose(lse[:n], l2[:n], atol=1e-4)
    if kv == "int8":
        t.dbt = cuda(t.bt)
        t.side["v_zeros"][int(t.bt[0, 2]), 0] = 128
        t.run(pa, impl)
        assert pa.device_error() == pa.PA_DEVERR_ZERO


@pytest.mark.parametrize("impl", IMPLS)
def test_tree_inconsistent_ranges_are_skipped_and_flagged(pa, impl):
    for what in ("descending", "past", "context", "long"):
        t = Tree(14, [50, 60, 70], [3, 4, 5], 8, 2, 128, 16, "bf16", pad=0)
        want, _ = t.run(pa, impl)
        if what == "descending":
            t.dqs = cuda([0, 3, 2, 12])
            skip, keep = slice(2, 12), slice(0, 2)
        elif what == "past":
            t.dqs = cuda([0, 3, 7, 13])
            skip, keep = slice(7, 12), slice(0, 7)
        elif what == "context":
            t.dctx = cuda([53, 3, 75])
            skip, keep = slice(3, 7), slice(0, 3)
        else:
            t.dctx = cuda([53, 4000, 75])
            skip, keep = slice(3, 7), slice(0, 3)
        out, _ = t.run(pa, impl)
        assert pa.device_error() == pa.PA_DEVERR_QUERY, what
        assert torch.equal(out[keep], want[keep]), what
        if what != "descending":
            assert (out[skip] == 3).all(), what


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("impl", IMPLS)
def test_tree_results_repeat_and_do_not_depend_on_placement(pa, impl, kv):
    t = Tree(15, [900, 17, 2500, 60], [8, 16, 3, 1], 8, 2, 128, 16, kv)
    o1, l1 = t.run(pa, impl)
    for _ in range(3):
        o2, l2 = t.run(pa, impl)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    perm = t.rng.permutation(t.o["k"].shape[0])
    for n in ("k", "v", "k_scales", "v_scales"):
        if t.o[n] is not None:
            x = np.empty_like(t.o[n])
            x[perm] = t.o[n]
            t.o[n] = x
    t.bt = np.where(t.bt >= 0, perm[np.maximum(t.bt, 0)], -1)
    t.device()
    o2, l2 = t.run(pa, impl)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("new", [40, 5])
def test_tree_drafts_across_the_parts_of_a_context(pa, kv, new):
    """A small batch is cut every 128 tokens: drafts that end, begin and lie across a cut, and a
    part that holds nothing but drafts."""
    Tree(21, [100, 88, 127, 128, 250, 384, 0], [new] * 7, 4, 1, 128, 8, kv).check(pa)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_tree_lengths_far_below_the_longest_allowed(pa, impl, kv):
    """A table and a longest context made for more than the batch has: most parts are empty, and
    rows of one part meet rows of several."""
    t = Tree(22, [30, 700, 3, 260], [4, 9, 1, 2], 8, 2, 128, 16, kv)
    t.bt = np.concatenate([t.bt, np.full((4, 900), -1)], 1)
    t.max_ctx = 16 * 900
    t.device()
    t.check(pa, impl)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("new", [5, 40])
def test_tree_long_parts(pa, kv, new):
    """A step with very many (padding) rows does not cut its contexts: a CTA takes a long one
    stretch by stretch, with drafts that lie across a stretch's end."""
    t = Tree(25, [12000, 5100, 5120, 40], [new] * 4, 4, 1, 128, 16, kv, pad=100000)
    assert t.workspace(pa).numel() == 16
    t.check(pa)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["fp8", "int8"])
def test_tree_scales_of_either_sign_that_differ_between_blocks(pa, impl, kv):
    """Block scales times powers of two from 2^-6 to 2^6 with signs, growing and shrinking along a
    context: weights that carry them stay within the format they are rounded to."""
    t = Tree(23, [330, 40, 500], [6, 8, 3], 8, 2, 128, 16, kv)
    rng = np.random.default_rng(24)
    for n, e in (("k_scales", 2), ("v_scales", 6)):
        shape = t.o[n].shape
        t.o[n] *= (rng.choice([-1.0, 1.0], shape) * 2.0 ** rng.integers(-e, e + 1, shape)).astype(np.float32)
    t.device()
    t.check(pa, impl)


def within(t, out, lse, rows=None, floor=0.0, weight=BF16):
    """Rows of a step against the oracle under the bounds above, with no slack but ``floor`` and
    weights rounded by ``weight``; infinities and NaN of the outputs where the oracle has values
    that are not finite."""
    with np.errstate(all="ignore"):
        ref, rl, absv, big = t.ref()
    n = int(t.qs[-1])
    pick = np.arange(n) if rows is None else np.asarray(rows)
    o, l = to_f64(out)[pick], to_f64(lse)[pick]
    ref, rl, absv, big = (x[pick] for x in (ref, rl, absv, big))
    ctx = np.repeat(t.ctx, t.new)[pick][:, None]
    dz = 2 * (t.d + 4) * F32 * big
    fin, fl = np.isfinite(ref), np.isfinite(rl)
    assert np.array_equal(np.isfinite(o), fin) and np.array_equal(np.isfinite(l), fl)
    with np.errstate(all="ignore"):
        E = 2 * (np.expm1(dz) + 2.0 ** -16 + 2.0 ** -21) + ctx * 2.0 ** -23
        tol = (weight + E)[..., None] * absv + BF16 * np.abs(ref) + floor
        assert (np.abs(o - ref)[fin] <= tol[fin]).all(), float((np.abs(o - ref) / tol)[fin].max())
        tl = dz + 2.0 ** -15 + ctx * 2.0 ** -23 + 2.0 ** -21 * np.abs(rl)
        assert (np.abs(l - rl)[fl] <= tl[fl]).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("bad", [math.inf, math.nan, 1e30])
@pytest.mark.parametrize("new", [8, 16, 24, 150])
def test_tree_scales_of_blocks_that_a_row_does_not_see(pa, impl, kv, bad, new):
    """A block of drafts with a huge, infinite or NaN scale takes nothing from rows that do not
    see it, also where it shares a step of keys with context blocks; rows that see it get it."""
    base = [24, 40, 200]
    half = new // 2
    see = [[list(range(i + 1)) if i < half else list(range(0, half // 2)) + list(range(half, i + 1))
            for i in range(new)] for _ in base]
    t = Tree(29, base, [new] * 3, 8, 2, 128, 8, kv, see=see)
    # the block with drafts half .. : the first half's rows see none of it where it begins there
    at = half // 8 * 8 + (8 if half % 8 else 0)
    if new == 8:     # one block of drafts: rows 0 to 3 see the context alone
        at, t.see = 0, [[[] if i < 4 else list(range(i + 1)) for i in range(8)] for _ in base]
    seen = [[any(at <= j < at + 8 for j in js) for js in s] for s in t.see]
    for s in range(3):
        b = t.bt[s, (base[s] + at) // 8]
        t.o["v_scales"][b] = bad
        if s == 1 and not math.isinf(bad):
            t.o["k_scales"][b] = math.nan
    t.device()
    out, lse = t.run(pa, impl)
    assert pa.device_error() == 0
    seen = np.array([x for s in seen for x in s])
    assert seen.any() and not seen.all()
    within(t, out, lse, np.flatnonzero(~seen))
    assert np.isfinite(to_f64(out)[:len(seen)][~seen]).all()
    if not math.isnan(bad):
        finite = math.isfinite(bad)
        keep = [i for i in np.flatnonzero(seen) if i // new != 1]
        if finite:
            # A weight times its V scale is held in f16 relative to a power of two of at most twice
            # the largest scale, times 2^7: to half a step of 2^-24, or 2^-31 of that scale. Where
            # the huge block's codes are 0 this is what is left of the others' |code| <= 448 (the
            # sum of weights that divides them is at least 1).
            within(t, out, lse, keep, floor=float(t.ctx.max()) * 448 * 2.0 ** -31 * bad)
        else:
            assert not np.isfinite(to_f64(out)[keep]).any()
    else:
        assert np.isnan(to_f64(out)[:len(seen)][seen]).all()


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("e", [-100, 114])
def test_tree_scales_near_the_ends_of_float32(pa, impl, kv, e):
    """V scales about 2^(e - 7): weights that carry them stay within the format they are rounded to
    (and, with a few hundred tokens, sums of values of 2^(e + 2) within float32)."""
    t = Tree(30, [300, 3], [6, 40], 8, 2, 128, 16, kv)
    t.o["v_scales"] *= np.float32(2.0 ** e)
    t.device()
    out, lse = t.run(pa, impl)
    assert pa.device_error() == 0
    within(t, out, lse)


@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("new", [8, 40])
def test_tree_weights_over_codes_are_f16(pa, kv, new):
    """Over one-byte codes a weight times its V scale is held in f16: to 2^-11 of itself, or half a
    step of 2^-24 relative to 2^-7 v_ref, v_ref at most twice the largest V scale (2^-31 of it for
    a code of 1; codes reach 448). The sum of the weights that divides them is at least 1. In
    channels that cancel, bf16 weights would pass the bound."""
    t = Tree(33, [2, 5, 40, 300], [new] * 4, 8, 2, 128, 16, kv)
    out, lse = t.run(pa)
    assert pa.device_error() == 0
    top = float(np.abs(t.o["v_scales"]).max())
    within(t, out, lse, floor=float(t.ctx.max()) * 448 * 2.0 ** -31 * top, weight=2.0 ** -11)


@pytest.mark.parametrize("impl", IMPLS)
@pytest.mark.parametrize("kv,e", [("bf16", 116), ("bf16", -100)] +
                         [(kv, e) for kv in ("fp8", "int8") for e in (118, 124, -100, -124)])
@pytest.mark.parametrize("new", [3, 33])
def test_tree_query_rows_of_any_size(pa, impl, kv, e, new):
    """Query rows near both ends of bf16's range, with a scale that brings their scores back (for a
    bf16 cache as far as sums of 128 products stay within float32); every other row is small."""
    t = Tree(31, [70, 300], [new, 2], 8, 2, 128, 16, kv)
    t.q[::2] *= 2.0 ** e
    t.scale *= 2.0 ** -e
    if e < 0:
        t.q[1::2] *= 2.0 ** (e - 2)
    out, lse = t.run(pa, impl)
    assert pa.device_error() == 0
    within(t, out, lse)


def test_tree_two_calls_at_once_and_other_streams(pa):
    """Calls on two streams with a workspace each, and on a side stream, give the same results."""
    a, b = Tree(16, [3000, 40], [8, 5], 8, 2, 128, 16, "bf16"), Tree(17, [700] * 9, [4] * 9, 8, 2, 128, 16, "fp8")
    ra, rb = a.run(pa), b.run(pa)
    bufs = [(t, torch.empty_like(t.q), torch.empty(t.T, t.hq, device="cuda"), t.workspace(pa)) for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (t, o, l, w), st in zip(bufs, streams):
            with torch.cuda.stream(st):
                t.run(pa, out=o, lse=l, ws=w)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    for (t, o, l, _), (r, rl) in zip(bufs, (ra, rb)):
        n = int(t.qs[-1])
        assert torch.equal(o[:n], r[:n]) and torch.equal(l[:n], rl[:n])


def test_tree_refusals(pa):
    t = Tree(18, [2000], [3], 8, 2, 128, 16, "bf16")   # long enough to be split on either path
    ok = dict(max_query_len=3, max_context_len=2003, workspace=t.workspace(pa))
    def go(q=t.q, kc=t.kc, bt=t.dbt, ctx=t.dctx, qs=t.dqs, mask=t.mask, out=None, **kw):
        a = dict(ok)
        a.update(kw)
        pa.paged_attn_tree(q, kc, t.vc, bt, ctx, qs, mask, 0.1, torch.empty_like(t.q) if out is None else out, **a)
    go()
    for kw in (dict(workspace=None), dict(workspace=t.workspace(pa)[:-1])):
        with pytest.raises(pa.PagedAttnError) as e:
            go(**kw)
        assert e.value.status == pa.PA_ERR_WORKSPACE
    for kw in (dict(max_query_len=33), dict(max_query_len=2004), dict(max_context_len=5000)):
        with pytest.raises(pa.PagedAttnError):
            go(**kw)
    for kw in (dict(q=t.q[:, :, :64]), dict(ctx=cuda([53, 1])), dict(qs=cuda([0, 1, 3])), dict(mask=t.mask[1:]),
               dict(out=torch.empty_like(t.q)[1:]), dict(bt=t.dbt.cpu()), dict(q=t.q.transpose(0, 1)),
               dict(kc=t.kc[:, :, ::2]), dict(lse_out=torch.empty(3, 8, device="cuda"))):
        with pytest.raises(ValueError):
            go(**kw)
    with pytest.raises(TypeError):
        go(ctx=t.dctx.long())
    assert pa.device_error() == 0


# ---------------------------------------------------------------------------------------
# acceptance
# ---------------------------------------------------------------------------------------
def verify(pa, par, draft, target, qs, ctx, A):
    S = len(ctx)
    o = dict(accepted=cuda(np.full((S, A), -7)), num_accepted=cuda(np.full(S, -7)),
             next_tokens=cuda(np.full(S, -7), torch.int64), kept_lens=cuda(np.full(S, -7)))
    pa.tree_verify(cuda(par), cuda(draft, torch.int64), cuda(target, torch.int64), cuda(qs), cuda(ctx), **o)
    return {k: v.cpu().numpy() for k, v in o.items()}


@pytest.mark.parametrize("sizes,A,vocab", [([1], 1, 2), ([5, 0, 1, 64], 8, 3), ([256, 33, 200], 40, 2),
                                           ([100] * 9, 1, 2), ([31, 32, 33, 63, 65, 0, 0, 2], 64, 2),
                                           ([256], 256, 1), ([3] * 300, 2, 4)])
@pytest.mark.parametrize("chain", [False, True])
def test_verify(pa, sizes, A, vocab, chain):
    rng = np.random.default_rng(sum(sizes) + A)
    par = sum(([-1] + list(range(n - 1)) if chain else random_parents(rng, n) for n in sizes if n), [])
    T, qs = sum(sizes), np.concatenate([[0], np.cumsum(sizes)])
    big = 1 << 40   # tokens are 64-bit
    draft, target = (rng.integers(0, vocab, T) * big + 5 for _ in range(2))
    ctx = np.array(sizes) + rng.integers(0, 50, len(sizes))
    paths, nxt, kept = drafted.ref_verify(par, draft, target, qs, ctx, A)
    o = verify(pa, par, draft, target, qs, ctx, A)
    assert pa.device_error() == 0
    for s, p in enumerate(paths):
        assert o["accepted"][s].tolist() == p + [-1] * (A - len(p))
    assert o["num_accepted"].tolist() == [len(p) for p in paths]
    assert o["next_tokens"].tolist() == nxt and o["kept_lens"].tolist() == kept


def test_verify_flags_bad_sequences(pa):
    T = 300
    par, tok = [-1] + list(range(T - 1)), [4] * T
    o = verify(pa, par, tok, tok, [0, 3, 2, 300, 301], [10, 10, 400, 10], 4)
    assert pa.device_error() == pa.PA_DEVERR_QUERY | pa.PA_DEVERR_TREE
    assert o["num_accepted"].tolist() == [3, 0, 0, 0] and o["kept_lens"].tolist() == [10, 10, 400, 10]
    assert o["next_tokens"].tolist() == [4, -1, -1, -1] and (o["accepted"][1:] == -1).all()


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("f32", 64), ("fp8", 128), ("int8", 128), ("fp8", 64),
                                  ("bf16", 256), ("int8", 256)])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_compact(pa, kv, d, B):
    rng = np.random.default_rng(d + B)
    new, base = [1, 40, 0, 256, 17, 64], [3, 77, 9, 0, 15, 200]
    t = Tree(B, base, new, 3, 3, d, B, kv, see=[[[] for _ in range(n)] for n in new], words=8)
    paths = []
    for n in new:
        k = int(rng.integers(1, n + 1)) if n else 0
        paths.append(sorted(rng.permutation(n)[:k].tolist()))
    paths[3] = sorted(set(paths[3]) | {0, 1, 2, 255})
    paths[4] = list(range(17))                       # everything stays in place
    A = max(len(p) for p in paths) + 3
    acc = cuda([p + [-1] * (A - len(p)) for p in paths])
    if kv in ("fp8", "int8"):                        # some blocks share a scale
        t.o["k_scales"][::2] = 0.01
        t.device()
    pa.compact_accepted(t.kc, t.vc, t.dbt, t.dctx, t.dqs, acc, cuda([len(p) for p in paths]), **t.side)
    assert pa.device_error() == 0
    for name, got in (("k", t.kc), ("v", t.vc)):
        ref = drafted.ref_compact(t.o[name], t.bt, t.ctx, t.qs, paths, kv, t.o[name + "_scales"],
                                  t.o[name + "_zeros"])
        assert np.array_equal(cache_codes(got), ref)
        if kv != "f32":
            assert not np.array_equal(ref, t.o[name])


def test_compact_bad_paths_move_nothing(pa):
    """Not ascending, past the rows, longer than the rows, a negative row: nothing moves; a bad
    block id skips its row."""
    new, base = [8, 8, 8, 8, 8], [20, 20, 20, 20, 20]
    t = Tree(3, base, new, 2, 2, 128, 16, "bf16")
    acc = cuda([[0, 2, 2, -1], [0, 8, -1, -1], [0, 1, 2, 3], [0, -1, 3, 4], [1, 2, 5, 7]])
    before = t.kc.clone()
    pa.compact_accepted(t.kc, t.vc, t.dbt, t.dctx, t.dqs, acc, cuda([3, 2, 5, 3, 0]))
    assert pa.device_error() == pa.PA_DEVERR_TREE and torch.equal(t.kc, before)
    bt = t.bt.copy()
    bt[4, 1] = 1 << 20
    pa.compact_accepted(t.kc, t.vc, cuda(bt), t.dctx, t.dqs, acc, cuda([0, 0, 0, 0, 4]))
    assert pa.device_error() == pa.PA_DEVERR_BLOCK_ID and torch.equal(t.kc, before)
    pa.compact_accepted(t.kc, t.vc, t.dbt, cuda([28, 28, 28, 28, 1000]), t.dqs, acc, cuda([0, 0, 0, 0, 4]))
    assert pa.device_error() == pa.PA_DEVERR_CONTEXT and torch.equal(t.kc, before)


# ---------------------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------------------
class Loop:
    """A drafting loop over PagedKVCache with everything on the GPU. A made-up model: a token's
    q, k, v come from fixed tables, the model's choice after a row from the sign of its output;
    drafts are drawn beforehand."""

    def __init__(self, pa, kv="bf16", S=3, hq=4, hkv=2, d=128, B=16, rows=24, words=1, A=6):
        from paged_kv_cache_465_b200.cache import PagedKVCache
        self.pa, self.S, self.d, self.hq, self.rows, self.A = pa, S, d, hq, rows, A
        self.cache = PagedKVCache(128, hkv, d, kv, B, order=np.random.default_rng(1).permutation(128))
        if kv == "fp8":   # scales are fixed before the first write, one for the pool
            self.cache.k_scales.fill_(0.02)
            self.cache.v_scales.fill_(0.02)
        g = torch.Generator(device="cuda").manual_seed(3)
        self.vocab = 5
        self.tables_q, self.tables_k, self.tables_v = (
            torch.randn(self.vocab, h, d, generator=g, device="cuda").bfloat16() for h in (hq, hkv, hkv))
        i = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.bt = torch.full((S, 32), -1, dtype=torch.int32, device="cuda")
        self.ring, self.queue = self.cache.free_ring()
        self.lens, self.held, self.new = i(S), i(S), i(S)
        self.total, self.qs, self.held2, self.queue2 = i(S), i(S + 1), i(S), i(2)
        self.slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.pos, self.mask, self.par, self.status = i(rows), i(rows, words), i(rows), i(1)
        self.tok = torch.zeros(rows, dtype=torch.int64, device="cuda")
        self.target = torch.zeros_like(self.tok)
        self.q = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(rows, hq, device="cuda")
        self.inv = 1.0 / 10000.0 ** (torch.arange(d // 2, device="cuda").float() / (d // 2))
        self.acc, self.nacc, self.kept = i(S, A), i(S), i(S)
        self.nxt = torch.zeros(S, dtype=torch.int64, device="cuda")
        self.ws = torch.empty(self.cache.tree_workspace_bytes(self.q, self.bt, max_query_len=32 * words,
                                                              max_context_len=512), dtype=torch.uint8, device="cuda")
        self.words = words

    def step(self):
        pa, c = self.pa, self.cache
        pa.build_step(self.lens, self.new, self.held, self.bt, self.ring, self.queue, block_size=c.block_size,
                      num_blocks=c.num_blocks, total_lens=self.total, query_start=self.qs,
                      blocks_held_out=self.held2, queue_state_out=self.queue2, slot_mapping=self.slots,
                      positions=self.pos, parents=self.par, tree_mask=self.mask, status=self.status)
        c.rotary_write(self.tables_q[self.tok], self.tables_k[self.tok], self.tables_v[self.tok], self.q,
                       self.pos, self.slots, self.inv)
        c.tree(self.q, self.bt, self.total, self.qs, self.mask, 1 / math.sqrt(self.d), self.out,
               max_query_len=32 * self.words, max_context_len=512, lse_out=self.lse, workspace=self.ws)
        self.target.copy_((self.out.float()[:, 0, :8].sum(-1) * 40).long().abs() % self.vocab)
        pa.tree_verify(self.par, self.tok, self.target, self.qs, self.total, accepted=self.acc,
                       num_accepted=self.nacc, next_tokens=self.nxt, kept_lens=self.kept)
        c.compact(self.bt, self.total, self.qs, self.acc, self.nacc)
        # what the step leaves: lengths, and the queue after the drafts' spare blocks went back
        pa.release_blocks(self.kept, self.held2, self.bt, self.ring, self.queue2, block_size=c.block_size,
                          blocks_held_out=self.held, queue_state_out=self.queue)
        self.lens.copy_(self.kept)

    def draft(self, rng, newest):
        """New trees: row 0 the newest token of its sequence, the others random drafts."""
        new = [int(rng.integers(1, 9)) for _ in range(self.S)]
        par, tok = [], []
        for s, n in enumerate(new):
            par += random_parents(rng, n)
            tok += [newest[s]] + rng.integers(0, self.vocab, n - 1).tolist()
        pad = self.rows - len(par)
        self.new.copy_(cuda(new))
        self.par.copy_(cuda(par + [-1] * pad))
        self.tok.copy_(cuda(tok + [0] * pad, torch.int64))
        return new, par, tok


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("graph", [False, True])
def test_drafting_loop_keeps_the_cache_of_plain_decoding(pa, kv, graph):
    """After a dozen drafted steps (eager, and captured once and replayed) the cache holds, position by
    position, the K and V of the accepted tokens alone, turned by their positions; no block is
    lost; and the last step's attention equals the oracle's."""
    lp = Loop(pa, kv)
    rng = np.random.default_rng(5)
    newest, history = [1, 2, 3], [[], [], []]
    if graph:   # warm up on a step of no tokens, then capture one
        lp.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lp.step()
    accepted_more = 0
    for _ in range(12):
        new, par, tok = lp.draft(rng, newest)
        g.replay() if graph else lp.step()
        torch.cuda.synchronize()
        assert pa.device_error() == 0 and lp.status.item() == 0
        qs = np.concatenate([[0], np.cumsum(new)])
        target = lp.target.tolist()
        for s in range(lp.S):
            path = [p for p in lp.acc[s].tolist() if p >= 0]
            assert path[0] == 0 and len(path) == lp.nacc[s].item()
            for a, b in zip(path, path[1:]):
                assert par[qs[s] + b] == a and tok[qs[s] + b] == target[qs[s] + a]
            history[s] += [tok[qs[s] + p] for p in path]
            newest[s] = lp.nxt[s].item()
            assert newest[s] == target[qs[s] + path[-1]]
            accepted_more += len(path) - 1
    assert accepted_more > 0   # the loop did exercise moves
    assert lp.lens.tolist() == [len(h) for h in history]
    held, bt = lp.held.tolist(), lp.bt.cpu().numpy()
    B = lp.cache.block_size
    assert held == [-(-len(h) // B) for h in history]
    head, count = lp.queue.tolist()
    ring = lp.ring.cpu().numpy()
    owned = [int(b) for s in range(lp.S) for b in bt[s, :held[s]]] + [int(ring[(head + i) % 128]) for i in range(count)]
    assert sorted(owned) == list(range(128))
    inv = lp.inv.cpu().numpy()
    for s, h in enumerate(history):
        idx = torch.tensor(h)
        k = drafted.ref_turn(to_f64(lp.tables_k)[idx], np.arange(len(h))[None], inv, [lp.d // 2], False)
        v = to_f64(lp.tables_v)[idx]
        t = np.arange(len(h))
        blk, off = bt[s, t // B], t % B
        sc = 0.02 if kv == "fp8" else 1.0
        gk, gv = (cache_codes(x)[blk, :, off] for x in (lp.cache.k_cache, lp.cache.v_cache))
        dec = (lambda c: e4m3_decode(c) * sc) if kv == "fp8" else (
            lambda c: (c.astype(np.uint32) << 16).view(np.float32).astype(np.float64))
        rel = E4M3 if kv == "fp8" else BF16
        tiny = 2.0 ** -10 * sc if kv == "fp8" else 0.0
        for got, ref in ((gk, k), (gv, v)):
            size = np.abs(ref).max(-1, keepdims=True) * 2.0 ** -19
            assert (np.abs(dec(got) - ref) <= np.maximum(rel * np.abs(ref) * (1 + 1e-6), tiny) + size).all()


def test_a_refused_step_changes_nothing_downstream(pa):
    """With the queue empty a step is refused on the GPU; the calls after it see a step of no
    tokens, and lengths, tables and pool stay."""
    lp = Loop(pa)
    rng = np.random.default_rng(9)
    lp.draft(rng, [0, 1, 2])
    lp.step()
    lens, held = lp.lens.clone(), lp.held.clone()
    count = lp.queue[1].item()
    lp.queue[1] = 0
    lp.lens.copy_(lp.held * 16)      # every block is full: any token needs a new one
    pool = lp.cache.k_cache.clone()
    full = lp.lens.clone()
    lp.draft(rng, [0, 1, 2])
    out = lp.out.clone()
    lp.step()
    assert pa.device_error() == pa.PA_DEVERR_BLOCKS and lp.status.item() == pa.PA_DEVERR_BLOCKS
    assert torch.equal(lp.lens, full) and torch.equal(lp.held, held) and torch.equal(lp.cache.k_cache, pool)
    assert lp.nacc.tolist() == [0, 0, 0] and torch.equal(lp.out, out) and count > 0 and lens.tolist()

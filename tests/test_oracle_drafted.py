"""CPU pins of the oracle's drafted-step functions, against other oracle functions, hand-worked
trees and closed forms; and refusals of the library's entry points that need no device."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import drafted
from oracle.attention import ref_prefill
from oracle.codecs import bf16_encode, e4m3_decode
from oracle.paged import RefAllocator


@pytest.fixture(scope="module")
def pa():
    from tests.test_lib_cpu import ROOT
    import importlib.util
    import os
    spec = importlib.util.spec_from_file_location(
        "_pa_build", os.path.join(ROOT, "paged_kv_cache_465_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build()
    import paged_kv_cache_465_b200 as pa
    return pa


def test_ancestors_and_masks_worked_by_hand():
    #      0
    #     / \
    #    1   2      5 hangs on the context
    #   /   / \
    #  3   4   6
    see = drafted.ref_ancestors([-1, 0, 0, 1, 2, -1, 2])
    assert see == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5], [0, 2, 6]]
    m = drafted.mask_words(see + [[31, 32, 63]], 2).view(np.uint32)
    assert m[:, 0].tolist() == [1, 3, 5, 11, 21, 32, 69, 1 << 31]
    assert m[:, 1].tolist() == [0] * 7 + [1 | 1 << 31]
    # a parent that is not before its child counts as none
    assert drafted.ref_ancestors([0, 5, 1]) == [[0], [1], [1, 2]]


@pytest.mark.parametrize("B", [8, 16, 32])
def test_build_step_takes_the_blocks_the_allocator_takes(B):
    rng = np.random.default_rng(B)
    nb, S = 200, 7
    order = rng.permutation(nb)
    al = RefAllocator(nb, B, order=order)
    lens = rng.integers(0, 60, S)
    for s in range(S):
        al.add_seq(s, int(lens[s]))
    width = 20
    tables = np.full((S, width), -1, dtype=np.int32)
    held = np.array([len(al.block_table(s)) for s in range(S)])
    for s in range(S):
        tables[s, :held[s]] = al.block_table(s)
    free = list(al.free)
    ring = np.array(free + [-1] * (nb - len(free)), dtype=np.int32)
    new = rng.integers(0, 40, S)
    got = drafted.ref_build_step(lens, new, held, tables, ring, [0, len(free)], B, nb, 400)
    slots, pairs = al.append_batch(list(range(S)), new.tolist())
    assert not pairs
    assert np.array_equal(got[5][:int(new.sum())], slots) and (got[5][int(new.sum()):] == -1).all()
    for s in range(S):
        assert got[0][s, :got[1][s]].tolist() == al.block_table(s)
    left = [int(ring[(got[2][0] + i) % nb]) for i in range(got[2][1])]
    assert left == list(al.free)
    # ending every sequence returns its blocks as the allocator does
    ring2, held2, q2 = drafted.ref_release([0] * S, got[1], got[0], ring, got[2], B)
    for s in range(S):
        al.free_seq(s)
    assert [int(ring2[(q2[0] + i) % nb]) for i in range(q2[1])] == list(al.free)
    assert not held2.any()


def test_build_step_refuses_as_a_whole():
    t = np.full((2, 4), -1, dtype=np.int32)
    t[0, 0] = 3
    args = ([5, 0], [20, 3], [1, 0], t, np.arange(6, dtype=np.int32))
    assert drafted.ref_build_step(*args, [0, 3], 16, 6, 32) is not None
    assert drafted.ref_build_step(*args, [0, 1], 16, 6, 32) is None      # short queue
    assert drafted.ref_build_step(*args, [0, 3], 16, 6, 22) is None      # more rows than there are
    assert drafted.ref_build_step(*args, [6, 3], 16, 6, 32) is None      # front outside the ring
    assert drafted.ref_build_step([5, 0], [60, 3], [1, 0], t, args[4], [0, 6], 16, 6, 99) is None
    assert drafted.ref_build_step([17, 0], [1, 3], [1, 0], t, args[4], [0, 6], 16, 6, 99) is None


@pytest.mark.parametrize("adjacent", [False, True])
def test_turn_is_a_rotation(adjacent):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    f = (1.0 / 10000 ** (np.arange(16) / 16)).astype(np.float32)
    pos = rng.integers(0, 1000, (3, 5))
    y = drafted.ref_turn(x, pos, f, [4, 6, 6], adjacent)
    assert np.array_equal(y[:, :, 32:], x[:, :, 32:])                    # the rest is untouched
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # a turn and its opposite cancel; position 0 changes nothing
    assert np.allclose(drafted.ref_turn(y, -pos, f, [4, 6, 6], adjacent), x)
    assert np.array_equal(drafted.ref_turn(x, 0 * pos, f, [4, 6, 6], adjacent), x)
    # equal positions on every axis: one axis; as complex numbers: multiplication by e^(i theta)
    p = np.repeat(pos[:1], 3, 0)
    one = drafted.ref_turn(x, pos[:1], f, [16], adjacent)
    assert np.array_equal(drafted.ref_turn(x, p, f, [4, 6, 6], adjacent), one)
    a, b = (slice(0, 32, 2), slice(1, 32, 2)) if adjacent else (slice(0, 16), slice(16, 32))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[0][:, None] * f.astype(np.float64))[:, None]
    assert np.allclose(one[..., a] + 1j * one[..., b], z)


def test_tree_of_a_chain_is_causal_prefill():
    rng = np.random.default_rng(4)
    S, B, NB, H, Hq, d = 3, 16, 20, 2, 4, 64
    k, v = (rng.standard_normal((NB, H, B, d)).astype(np.float32) for _ in range(2))
    bt = rng.permutation(NB)[:S * 4].reshape(S, 4)
    ctx, qs = [50, 7, 33], [0, 9, 16, 17]
    q = rng.standard_normal((17, Hq, d)).astype(np.float32)
    see = [drafted.ref_ancestors(range(-1, qs[s + 1] - qs[s] - 1)) for s in range(S)]
    out, lse, absv, _ = drafted.ref_tree(q, qs, see, k, v, bt, ctx, 0.125, H, "f32", "f32")
    o2, l2 = ref_prefill(q, np.array(qs), k, v, bt, ctx, 0.125, H, "f32", "f32")
    assert np.allclose(out, o2) and np.allclose(lse, l2) and (absv >= np.abs(out) - 1e-12).all()
    # sequence 1 brings its whole context: a row that sees nothing at all
    see[1][3] = []
    out, lse, *_ = drafted.ref_tree(q, qs, see, k, v, bt, ctx, 0.125, H, "f32", "f32")
    assert (out[12] == 0).all() and (lse[12] == -np.inf).all()


def test_verify_worked_by_hand():
    # two trees: 0-{1, 2}, 2-{3, 4}; and a chain of 2
    par = [-1, 0, 0, 2, 2, -1, 0]
    draft = [9, 5, 7, 1, 1, 3, 4]
    ver = lambda target, a=8: drafted.ref_verify(par, draft, target, [0, 5, 7, 7], [15, 12, 4], a)  # noqa: E731
    paths, nxt, kept = ver([7, 0, 1, 8, 6, 5, 5])
    assert paths == [[0, 2, 3], [0], []]        # of the twins 3 and 4 the first
    assert nxt == [8, 5, -1] and kept == [13, 11, 4]
    paths, nxt, kept = ver([7, 0, 1, 8, 6, 4, 5], 2)
    assert paths == [[0, 2], [0, 1], []] and nxt == [1, 5, -1] and kept == [12, 12, 4]


def test_compact_moves_in_order_and_requantises():
    rng = np.random.default_rng(1)
    pool = bf16_encode(rng.standard_normal((4, 2, 16, 8)).astype(np.float32))
    bt, ctx, qs = [[2, 0], [3, 1]], [20, 9], [0, 6, 9]
    got = drafted.ref_compact(pool, bt, ctx, qs, [[0, 2, 3, 5], [0]], "bf16")
    flat = lambda p, s, t: p[bt[s][t // 16], :, t % 16]  # noqa: E731
    for i, src in enumerate([0, 2, 3, 5]):
        assert np.array_equal(flat(got, 0, 14 + i), flat(pool, 0, 14 + src))
    assert np.array_equal(got[3], pool[3])
    # fp8: the value survives a change of scale by a power of two
    codes = rng.integers(0, 120, (4, 2, 16, 8)).astype(np.uint8)
    sc = np.ones((4, 2), dtype=np.float32)
    sc[0] = 0.5
    got = drafted.ref_compact(codes, bt, ctx, qs, [[0, 5], [0]], "fp8", sc)
    a, b = e4m3_decode(got[2, :, 15]), e4m3_decode(codes[0, :, 3])
    keep = b * 0.5 >= 2.0 ** -6
    assert np.array_equal(a[keep], b[keep] * 0.5) and keep.any()


def test_refusals_without_a_device(pa):
    lib, one, nul = pa._lib, ctypes.c_void_p(256), ctypes.c_void_p(0)
    two = ctypes.c_void_p(256 + 4096)
    apart = [ctypes.c_void_p(4096 * (i + 1)) for i in range(20)]   # addresses of separate buffers

    def build(seqs=2, width=4, bs=16, nb=8, cap=8, rows=8, words=2, **at):
        p = list(apart[:15])   # 0-6 inputs (3 parents, 4 tables), 7-14 outputs
        for k, v in at.items():
            p[int(k[1:])] = v
        return lib.paged_build_step(*p[:7], seqs, width, bs, nb, cap, rows, words, *p[7:15], nul)
    for kw in (dict(seqs=-1), dict(seqs=65536), dict(width=0), dict(bs=0), dict(nb=0), dict(cap=0),
               dict(rows=-1), dict(words=0), dict(words=9), dict(width=1 << 30)):
        assert build(**kw) == pa.PA_ERR_INVALID, kw
    for i in (0, 1, 2, 4, 5, 6, 7, 8, 9, 10, 11):                # required
        assert build(**{f"p{i}": nul}) == pa.PA_ERR_INVALID, i
    for i, j in ((4, 0), (7, 0), (7, 1), (9, 2), (10, 6), (11, 3), (12, 11), (13, 5), (14, 8)):
        assert build(**{f"p{i}": apart[j]}) == pa.PA_ERR_INVALID, (i, j)      # shared memory
    assert build(p12=ctypes.c_void_p(4096 * 12 + 63)) == pa.PA_ERR_INVALID   # partly
    assert build(seqs=0, p0=nul) == pa.PA_OK

    def release(seqs=2, width=4, bs=16, cap=8, **at):
        p = list(apart[:8])   # 0-4 inputs (3 the ring), 5-7 outputs
        for k, v in at.items():
            p[int(k[1:])] = v
        return lib.paged_release_blocks(*p[:5], seqs, width, bs, cap, *p[5:8], nul)
    for kw in (dict(seqs=-1), dict(width=0), dict(bs=0), dict(cap=0)):
        assert release(**kw) == pa.PA_ERR_INVALID, kw
    for i in range(7):
        assert release(**{f"p{i}": nul}) == pa.PA_ERR_INVALID, i
    for i, j in ((5, 1), (5, 0), (6, 4), (7, 5), (3, 2)):
        assert release(**{f"p{i}": apart[j]}) == pa.PA_ERR_INVALID, (i, j)
    assert release(seqs=0, p0=nul) == pa.PA_OK

    def rotary(T=4, hq=8, hkv=2, d=128, rot=128, axes=1, sec=(64, 0, 0, 0), nb=8, bs=16, qs=1024,
               ks=256, indt=pa.PA_BF16, cache=pa.PA_BF16, ptr=one, q_out=two, sc=nul, zp=nul,
               qos=1024):
        desc = pa.pa_rotary_desc(T, hq, hkv, d, rot, axes, (ctypes.c_int * 4)(*sec), 0, bs, nb, qs,
                                 ks, ks, qos, indt, cache)
        return lib.rotary_and_cache(ptr, ptr, ptr, q_out, ptr, ptr, ptr, ptr, ptr,
                                    ctypes.byref(desc), sc, sc, zp, zp, nul)
    for kw in (dict(T=-1), dict(hq=0), dict(hkv=0), dict(rot=0), dict(rot=24, sec=(12, 0, 0, 0)),
               dict(rot=144, sec=(72, 0, 0, 0)), dict(axes=0), dict(axes=5), dict(sec=(60, 0, 0, 0)),
               dict(axes=2, sec=(70, -6, 0, 0)), dict(qs=1000), dict(qs=1026), dict(ks=130),
               dict(ptr=nul), dict(ptr=ctypes.c_void_p(264)), dict(q_out=one, qos=2048), dict(nb=0),
               dict(cache=pa.PA_FP8_E4M3), dict(cache=pa.PA_INT8, sc=one)):
        assert rotary(**kw) == pa.PA_ERR_INVALID, kw
    for kw in (dict(d=96, rot=96, sec=(48, 0, 0, 0)), dict(indt=pa.PA_INT8), dict(cache=pa.PA_F32),
               dict(cache=7)):
        assert rotary(**kw) == pa.PA_ERR_UNSUPPORTED, kw
    assert rotary(T=0, ptr=nul) == pa.PA_OK
    assert lib.rotary_and_cache(*([one] * 9), None, nul, nul, nul, nul, nul) == pa.PA_ERR_INVALID

    d = pa.make_desc(4, 32, 8, 128, 64, 1024, pa.PARTITION_AUTO, pa.PA_BF16, pa.PA_BF16, pa.PA_BF16)

    def tree(desc=d, words=2, T=100, mq=50, scale=0.1, ctx=1024, ptr=one, ws=one, nbytes=1 << 40):
        return lib.paged_attn_tree(ptr, ptr, ptr, ptr, ptr, ptr, ptr, words, T, mq,
                                   ctypes.c_float(scale), ptr, ctypes.byref(desc), ctx, nul, nul, nul,
                                   nul, nul, ws, nbytes, nul)
    split = pa.make_desc(4, 32, 8, 128, 64, 1024, 512, pa.PA_BF16, pa.PA_BF16, pa.PA_BF16)
    fp8 = pa.make_desc(4, 32, 8, 128, 64, 1024, 0, pa.PA_BF16, pa.PA_FP8_E4M3, pa.PA_BF16)
    for kw in (dict(desc=split), dict(words=0), dict(words=9), dict(mq=65), dict(words=8, mq=257),
               dict(T=-1), dict(mq=-1), dict(ctx=49), dict(ctx=1025), dict(scale=math.nan),
               dict(scale=math.inf), dict(ptr=nul), dict(ptr=ctypes.c_void_p(264)), dict(desc=fp8)):
        assert tree(**kw) == pa.PA_ERR_INVALID, kw
    for hd in (96, 32):
        u = pa.make_desc(4, 32, 8, hd, 64, 1024, 0, pa.PA_BF16, pa.PA_BF16, pa.PA_BF16)
        assert tree(desc=u) == pa.PA_ERR_UNSUPPORTED
    assert tree(ws=nul) == pa.PA_ERR_WORKSPACE
    need = lib.paged_attn_tree_workspace_size(ctypes.byref(d), 100, 50, 1024)
    assert need > 0 and tree(nbytes=need - 1) == pa.PA_ERR_WORKSPACE
    for kw in (dict(T=0), dict(mq=0)):
        assert tree(ptr=nul, ws=nul, **kw) == pa.PA_OK
    assert lib.paged_attn_tree_workspace_size(ctypes.byref(split), 100, 50, 1024) == 0

    def verify(S=2, T=8, A=4, **at):
        p = list(apart[:9])   # 0-4 inputs, 5-8 outputs
        for k, v in at.items():
            p[int(k[1:])] = v
        return lib.tree_verify(*p[:5], S, T, A, *p[5:9], nul)
    for kw in (dict(S=-1), dict(S=65536), dict(T=-1), dict(A=0)):
        assert verify(**kw) == pa.PA_ERR_INVALID, kw
    for i in range(9):
        assert verify(**{f"p{i}": nul}) == pa.PA_ERR_INVALID, i
    for i, j in ((5, 0), (6, 3), (7, 1), (8, 4), (8, 6)):
        assert verify(**{f"p{i}": apart[j]}) == pa.PA_ERR_INVALID, (i, j)
    assert verify(S=0, p0=nul) == pa.PA_OK

    def compact(S=2, A=4, width=4, hkv=2, hd=128, bs=16, nb=8, dt=pa.PA_BF16, ptr=one, sc=nul, zp=nul):
        return lib.compact_accepted(ptr, ptr, ptr, ptr, ptr, ptr, ptr, S, A, width, hkv, hd, bs, nb,
                                    dt, sc, sc, zp, zp, nul)
    for kw in (dict(S=-1), dict(A=0), dict(A=257), dict(width=0), dict(hkv=0), dict(hd=0), dict(bs=0),
               dict(nb=0), dict(ptr=nul), dict(ptr=ctypes.c_void_p(264)), dict(dt=pa.PA_FP8_E4M3),
               dict(dt=pa.PA_INT8, sc=one)):
        assert compact(**kw) == pa.PA_ERR_INVALID, kw
    assert compact(dt=7) == pa.PA_ERR_UNSUPPORTED and compact(hd=4) == pa.PA_ERR_UNSUPPORTED
    assert compact(S=0, ptr=nul) == pa.PA_OK


def test_idle_steps_are_checked_too(pa):
    """No sequences: the buffers that are read or written all the same have to be there, and apart."""
    nul = ctypes.c_void_p(0)
    at = [ctypes.c_void_p(4096 * (i + 1)) for i in range(20)]

    def build(rows=8, **kw):
        p = [nul] * 5 + at[5:7] + [nul] + [at[8], nul] + at[10:15]   # per-sequence buffers absent
        for k, v in kw.items():
            p[int(k[1:])] = v
        return pa._lib.paged_build_step(*p[:7], 0, 4, 16, 8, 8, rows, 2, *p[7:15], nul)
    for i in (5, 6, 8, 10, 11):
        assert build(**{f"p{i}": nul}) == pa.PA_ERR_INVALID, i
    for i, j in ((10, 6), (8, 5), (11, 6), (14, 12), (13, 11)):
        assert build(**{f"p{i}": at[j]}) == pa.PA_ERR_INVALID, (i, j)

    def release(**kw):
        p = [nul] * 3 + at[3:5] + [nul] + at[6:8]
        for k, v in kw.items():
            p[int(k[1:])] = v
        return pa._lib.paged_release_blocks(*p[:5], 0, 4, 16, 8, *p[5:8], nul)
    for i in (3, 4, 6):
        assert release(**{f"p{i}": nul}) == pa.PA_ERR_INVALID, i
    for i, j in ((6, 4), (7, 3), (7, 6)):
        assert release(**{f"p{i}": at[j]}) == pa.PA_ERR_INVALID, (i, j)


def test_tree_workspace_does_not_grow_with_the_context(pa):
    """Contexts are cut into no more parts than fill the GPU, and on the tensor cores into no more
    than whose results fit 192 MB."""
    def size(T, ctx, S=8, d=128, kv=None, hq=64):
        desc = pa.make_desc(S, hq, 8, d, -(-ctx // 16), 1 << 16, pa.PARTITION_AUTO, pa.PA_BF16,
                            pa.PA_BF16 if kv is None else kv, pa.PA_BF16)
        return pa._lib.paged_attn_tree_workspace_size(ctypes.byref(desc), T, 16, ctx)
    assert 0 < size(128, 131072) == size(128, 1 << 20) <= 192 << 20
    assert size(16384, 131072, S=1024) <= 48 << 20
    assert size(16, 131072, S=1, d=64) <= 64 << 20


def test_binding_refuses_host_tensors(pa):
    import torch
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    b = lambda *n: torch.zeros(*n, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError):
        pa.build_step(i(2), i(2), i(2), i(2, 3), i(9), i(2), block_size=16, num_blocks=9,
                      total_lens=i(2), query_start=i(3), blocks_held_out=i(2), queue_state_out=i(2),
                      slot_mapping=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        pa.release_blocks(i(2), i(2), i(2, 3), i(9), i(2), block_size=16, blocks_held_out=i(2),
                          queue_state_out=i(2))
    with pytest.raises(ValueError):
        pa.rotary_and_cache(b(2, 4, 64), b(2, 2, 64), b(2, 2, 64), b(2, 4, 64), b(4, 2, 16, 64),
                            b(4, 2, 16, 64), i(2), torch.zeros(2, dtype=torch.int64), torch.ones(32))
    with pytest.raises(ValueError):
        pa.paged_attn_tree(b(2, 4, 64), b(4, 2, 16, 64), b(4, 2, 16, 64), i(1, 3), i(1), i(2), i(2, 1),
                           0.1, b(2, 4, 64), max_query_len=2, max_context_len=40)
    with pytest.raises(ValueError):
        pa.tree_verify(i(2), torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int64), i(2),
                       i(1), accepted=i(1, 4), num_accepted=i(1),
                       next_tokens=torch.zeros(1, dtype=torch.int64), kept_lens=i(1))
    with pytest.raises(ValueError):
        pa.compact_accepted(b(4, 2, 16, 64), b(4, 2, 16, 64), i(1, 3), i(1), i(2), i(1, 4), i(1))


UNREADABLE = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
import paged_kv_cache_465_b200 as pa

def i(*n): return torch.empty(*n, dtype=torch.int32, device="cuda")
def l(*n): return torch.empty(*n, dtype=torch.int64, device="cuda")
def b(*n): return torch.empty(*n, dtype=torch.bfloat16, device="cuda")

def verify(parents):
    pa.tree_verify(parents, l(4), l(4), i(2), i(1), accepted=i(1, 2), num_accepted=i(1),
                   next_tokens=l(1), kept_lens=i(1))
    return parents

def rotary(q):
    pa.rotary_and_cache(q, b(2, 2, 64), b(2, 2, 64), b(2, 4, 64), b(4, 2, 16, 64), b(4, 2, 16, 64),
                        i(2), l(2), torch.ones(32, device="cuda"))
    return q

with FakeTensorMode():
    for f, x in ((verify, i(3, 4)), (rotary, b(3, 2, 4, 64))):
        try:
            torch.func.vmap(f)(x)
        except RuntimeError as e:
            print("raised:", str(e).splitlines()[0])
"""


def test_tensors_without_readable_memory_raise(pa):
    """A tensor that a transform has batched has no pointer: an error, as any other, not the end of
    the process."""
    r = subprocess.run([sys.executable, "-W", "ignore", "-c", UNREADABLE], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]
    said = [line for line in r.stdout.splitlines() if line.startswith("raised:")]
    assert len(said) == 2 and all("storage" in line for line in said), r.stdout

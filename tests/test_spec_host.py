"""Host side of the speculative step, on CPU: draft masks, rotary frequencies, forks, the tree plan's
work list, and every refusal that needs no device."""
import ctypes
import math

import numpy as np
import pytest

import non_uniform_paged_flash_b200 as tg


# ---- masks ----

def test_tree_masks():
    off = [0, 5, 5, 7]
    parent = [-1, 0, 0, 1, -1, -1, 0]
    assert tg.tg_tree_masks(off, parent).tolist() == [1, 3, 5, 11, 16, 1, 3]
    chain = tg.tg_tree_masks([0, 64], np.arange(64) - 1)
    assert [int(m) for m in chain] == [(1 << (j + 1)) - 1 for j in range(64)]
    assert tg.tg_tree_masks([0], []).size == 0


@pytest.mark.parametrize("off,parent", [([0, 2], [-1, 1]), ([0, 2], [0, 0]), ([0, 1], [-2]), ([0, 65], [-1] * 65),
                                        ([1, 2], [-1, -1]), ([0, 3, 2], [-1, -1])])
def test_tree_masks_refusals(off, parent):
    with pytest.raises(tg.TGError) as e:
        tg.tg_tree_masks(off, parent)
    assert e.value.status == tg.TG_EINVAL


# ---- frequencies ----

def test_rope_frequencies():
    plain, s = tg.tg_rope_frequencies(64, 10000.0)
    assert s == 1.0
    np.testing.assert_allclose(plain, 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    lin, _ = tg.tg_rope_frequencies(64, 10000.0, tg.TG_ROPE_LINEAR, 4.0)
    np.testing.assert_allclose(lin, plain / 4, rtol=1e-14)
    ntk, _ = tg.tg_rope_frequencies(64, 10000.0, tg.TG_ROPE_NTK, 4.0)
    np.testing.assert_allclose(ntk[0], 1.0)                                # the fastest pair is kept
    np.testing.assert_allclose(ntk[-1], plain[-1] / 4, rtol=1e-12)          # the slowest is interpolated
    yarn, s = tg.tg_rope_frequencies(64, 10000.0, tg.TG_ROPE_YARN, 4.0, 4096)
    assert s == pytest.approx(0.1 * math.log(4.0) + 1)
    turns = 4096 * plain / (2 * math.pi)
    ratio = plain / yarn
    assert np.all(np.diff(ratio) >= -1e-12)
    np.testing.assert_allclose(ratio[turns > 40], 1.0, rtol=1e-12)
    np.testing.assert_allclose(ratio[turns < 0.7], 4.0, rtol=1e-12)
    for kind in range(4):   # a factor of one changes nothing
        np.testing.assert_allclose(tg.tg_rope_frequencies(64, 5e5, kind, 1.0, 8192)[0],
                                   tg.tg_rope_frequencies(64, 5e5)[0], rtol=1e-13)
    assert tg.tg_rope_frequencies(0)[0].size == 0
    assert tg.tg_rope_frequencies(2)[0].tolist() == [1.0]


@pytest.mark.parametrize("args", [(63,), (-2,), (64, 1.0), (64, float("nan")), (64, float("inf")), (64, 1e4, 4),
                                  (64, 1e4, -1), (64, 1e4, 1, 0.5), (64, 1e4, 1, float("nan")), (2, 1e4, 2, 2.0),
                                  (64, 1e4, 3, 2.0, 0), (64, 1e4, 3, 2.0, 4096, 1.0, 1.0), (64, 1e4, 3, 2.0, 4096, 2.0, 0.0)])
def test_rope_frequency_refusals(args):
    with pytest.raises(tg.TGError) as e:
        tg.tg_rope_frequencies(*args)
    assert e.value.status == tg.TG_EINVAL


# ---- fork ----

def _refs(a, n):
    return [tg.tg_alloc_refcount(a, p) for p in range(n)]


def test_fork_shares_full_pages_and_lists_the_rest():
    a = tg.tg_alloc_create_ordered(40, 16)
    ids, cnt = tg.tg_reserve(a, 0, [40, 20], with_counts=True)           # pages 0 1 2 | 3 4
    assert ids.tolist() == [0, 1, 2, 3, 4]
    cids, ccnt, src, dst, rows = tg.tg_fork(a, 0, 1, [35, 16], [50, 16], [1, 1])
    assert cids.tolist() == [0, 5, 6, 7, 3] and ccnt.tolist() == [4, 1]
    assert src.tolist() == [1, 2] and dst.tolist() == [5, 6] and rows.tolist() == [16, 3]
    assert _refs(a, 8) == [2, 1, 1, 2, 1, 1, 1, 1]
    # a fork of the fork, then release in any order
    g = tg.tg_fork(a, 1, 2, [50, 0], [50, 0], [3, 0])
    assert g[0].tolist() == [0, 5, 6, 8] and g[2].tolist() == [7] and g[4].tolist() == [2]
    tg.tg_release(a, 0)
    assert _refs(a, 9) == [2, 0, 0, 1, 0, 2, 2, 1, 1]
    tg.tg_release(a, 1)
    tg.tg_release(a, 2)
    assert tg.tg_alloc_free_pages(a) == 40 and _refs(a, 9) == [0] * 9
    tg.tg_alloc_destroy(a)


def test_fork_of_a_sequence_on_a_segment():
    a = tg.tg_alloc_create_ordered(40, 16)
    seg, _ = tg.tg_share_segment(a, 32, 1)
    tg.tg_reserve(a, 0, [40], prefix_segs=[seg])
    ids, _, src, dst, rows = tg.tg_fork(a, 0, 1, [40], [60], [2])
    assert ids.tolist() == [0, 1, 3, 4] and (src.tolist(), dst.tolist(), rows.tolist()) == ([2], [3], [8])
    assert tg.tg_alloc_refcount(a, 0) == 3
    for s in (1, 0):
        tg.tg_release(a, s)
    tg.tg_release_segment(a, seg)
    assert tg.tg_alloc_free_pages(a) == 40
    tg.tg_alloc_destroy(a)


def test_fork_refusals_leave_the_allocator_as_it_was():
    a = tg.tg_alloc_create_ordered(10, 16)
    tg.tg_reserve(a, 0, [40, 20])
    before, free = _refs(a, 10), tg.tg_alloc_free_pages(a)
    for args, st in (((5, 1, [1, 1], [1, 1], [0, 0]), tg.TG_ENOTFOUND), ((0, 0, [1, 1], [1, 1], [0, 0]), tg.TG_EEXIST),
                     ((0, 1, [1], [1], [0]), tg.TG_EINVAL), ((0, 1, [49, 1], [60, 1], [0, 0]), tg.TG_EINVAL),
                     ((0, 1, [40, 20], [39, 20], [0, 0]), tg.TG_EINVAL), ((0, 1, [40, 20], [40, 20], [3, 0]), tg.TG_EINVAL),
                     ((0, 1, [-1, 0], [0, 0], [0, 0]), tg.TG_EINVAL), ((0, 1, [0, 0], [0, 0], [-1, 0]), tg.TG_EINVAL),
                     ((0, 1, [40, 20], [80, 30], [0, 0]), tg.TG_ENOSPC)):
        with pytest.raises(tg.TGError) as e:
            tg.tg_fork(a, *args)
        assert e.value.status == st, args
    assert _refs(a, 10) == before and tg.tg_alloc_free_pages(a) == free
    with pytest.raises(ValueError):
        tg.tg_fork(a, 0, 1, [1], [1, 1], [0, 0])
    tg.tg_fork(a, 0, 1, [16, 0], [16, 0], [1, 0])   # the id is free after the refusals
    tg.tg_alloc_destroy(a)


def test_random_forks_conserve_pages():
    rng = np.random.default_rng(1)
    a = tg.tg_alloc_create(300, 16, 5)
    live, nxt = {}, 0
    for _ in range(400):
        if not live or rng.random() < 0.3:
            kv = rng.integers(0, 90, size=3)
            try:
                ids, cnt = tg.tg_reserve(a, nxt, kv, with_counts=True)
            except tg.TGError as e:
                assert e.status == tg.TG_ENOSPC
            else:
                live[nxt] = (kv, ids)
            nxt += 1
        elif rng.random() < 0.6:
            p = int(rng.choice(list(live)))
            kv, _ = live[p]
            held = np.array([rng.integers(0, n + 1) for n in kv])
            shared = np.array([rng.integers(0, h // 16 + 1) for h in held])
            new = held + rng.integers(0, 40, size=3)
            try:
                ids, cnt, src, dst, rows = tg.tg_fork(a, p, nxt, held, new, shared)
            except tg.TGError as e:
                assert e.status == tg.TG_ENOSPC
            else:
                assert cnt.tolist() == [-(-int(n) // 16) for n in new]
                assert int(rows.sum()) == int((held - 16 * shared).sum())
                assert set(dst) <= set(ids) and not set(dst) & set(src)
                live[nxt] = (new, ids)
            nxt += 1
        else:
            s = int(rng.choice(list(live)))
            tg.tg_release(a, s)
            del live[s]
        want = np.zeros(300, int)
        for _, ids in live.values():
            np.add.at(want, ids, 1)
        assert _refs(a, 300) == want.tolist()
        assert tg.tg_alloc_free_pages(a) == int((want == 0).sum())
    tg.tg_alloc_destroy(a)


# ---- tree plan ----

def _plan(cap, Hq, Hkv, T, D=128, workers=0, pages=1 << 20, **kw):
    B = np.asarray(cap).size // Hkv
    return tg.tg_tree_plan_create(tg.make_shape(B, Hq, Hkv, D, pages), cap, T, np.zeros(Hkv, np.int32), [0, 1 << 20],
                                  num_workers=workers, host_only=True, **kw)


@pytest.mark.parametrize("Hq,T,tokens,D,rows", [(8, 4, 4000, 128, 16), (8, 5, 4000, 128, 64), (8, 8, 4000, 128, 64),
                                                (8, 9, 4000, 128, 64), (8, 8, 1000, 128, 64), (8, 4, 1000, 128, 16),
                                                (8, 4, 200, 128, 64), (8, 4, 4000, 64, 64), (8, 33, 4000, 128, 256),
                                                (8, 17, 4000, 128, 128), (8, 16, 4000, 64, 64)])
def test_plan_kernel_by_rows_and_lengths(Hq, T, tokens, D, rows):
    assert tg.tg_tree_plan_items(_plan([tokens] * 4, Hq, 2, T, D=D))["rows"] == rows


@pytest.mark.parametrize("seed", range(12))
def test_plan_covers_every_page_once(seed):
    rng = np.random.default_rng(seed)
    Hkv, G = 2, int(rng.choice([1, 2, 4, 8]))
    B = int(rng.integers(1, 40))
    T = int(rng.integers(1, 65))
    cap = rng.choice([0, 1, 16, 17, 500, int(rng.integers(1, 9000))], size=B * Hkv)
    info = tg.tg_tree_plan_items(_plan(cap, G * Hkv, Hkv, T, workers=int(rng.choice([0, 1, 7, 400]))))
    it, off = info["items"], info["worker_off"]
    # each worker's own items, then those taken by ticket
    assert off[0] == 0 and off[-1] <= len(it) and np.all(np.diff(off) >= 0) and len(off) == info["n_workers"] + 1
    per = 256 if T * G > 128 else T * G
    rblocks = -(-T * G // per)
    slots = []
    for i in range(B * Hkv):
        for rb in range(rblocks):
            mine = it[(it[:, 0] == i) & (it[:, 4] == rb * per)]
            pages = -(-int(cap[i]) // 16)
            edges = [0] + mine[:, 2].tolist()
            assert mine[:, 1].tolist() == edges[:-1] and edges[-1] == pages     # in order, end to end
            assert mine[:, 5].tolist() == [0] * (len(mine) - 1) + [1]           # the last takes the draft
            assert all(e % 4 == 0 for e in edges[1:-1]) and np.all(mine[:, 6] == cap[i])
            if len(mine) == 1:
                assert mine[0, 3] == -1
            else:
                assert mine[:, 3].tolist() == list(range(mine[0, 3], mine[0, 3] + len(mine)))
                slots += mine[:, 3].tolist()
    assert sorted(slots) == list(range(len(slots)))


@pytest.mark.parametrize("T,workers", [(16, 296), (4, 148)])
def test_plan_shares_are_even(T, workers):
    rng = np.random.default_rng(0)
    cap = rng.integers(500, 8000, size=512)
    info = tg.tg_tree_plan_items(_plan(cap, 32, 8, T))
    it, off = info["items"], info["worker_off"]
    load = [int((it[a:b, 2] - it[a:b, 1]).sum()) for a, b in zip(off[:-1], off[1:])]
    assert info["n_workers"] == workers and max(load) <= 1.2 * np.mean(load)
    dyn = it[off[-1]:]
    left = (dyn[:, 2] - dyn[:, 1]).sum() / (it[:, 2] - it[:, 1]).sum()
    assert 0.005 < left < 0.13                            # the rest is taken by ticket
    size = dyn[:, 2] - dyn[:, 1]
    assert size.max() <= 80                               # in small items
    small = tg.tg_tree_plan_items(_plan([500] * 8, 8, 8, 4))
    assert small["worker_off"][-1] == small["n_items"]    # a small step is all static


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), tg.TG_EINVAL), (dict(T=65), tg.TG_EUNSUPPORTED), (dict(D=96), tg.TG_EUNSUPPORTED),
    (dict(Hq=6), tg.TG_EUNSUPPORTED), (dict(Hq=7), tg.TG_EINVAL), (dict(cap=[-1, 0]), tg.TG_EINVAL),
    (dict(cap=[tg.TG_MAX_HEAD_TOKENS + 1, 0]), tg.TG_EUNSUPPORTED), (dict(pages=1 << 28), tg.TG_EUNSUPPORTED),
    (dict(pages=-1), tg.TG_EINVAL), (dict(workers=-1), tg.TG_EINVAL), (dict(workers=65537), tg.TG_EUNSUPPORTED), (dict(device=-2), tg.TG_EINVAL),
    (dict(wait_limit_us=-1), tg.TG_EINVAL)])
def test_plan_refusals(kw, status):
    args = dict(cap=[30, 40], Hq=8, Hkv=2, T=4)
    args.update(kw)
    with pytest.raises(tg.TGError) as e:
        _plan(**args)
    assert e.value.status == status


def test_plan_group_refusals():
    sh = tg.make_shape(1, 8, 2, 128, 100)
    for goh, goff in (([0, 1], [0, 10]), ([0, -1], [0, 10]), ([0, 0], [10, 0]), ([0, 0], [-1, 10])):
        with pytest.raises(tg.TGError):
            tg.tg_tree_plan_create(sh, [3, 3], 4, goh, goff, host_only=True)
    with pytest.raises(ValueError):
        tg.tg_tree_plan_create(sh, [3], 4, [0, 0], [0, 10], host_only=True)


# ---- refusals of the device calls, before anything is launched ----

def test_device_calls_refuse_bad_arguments_on_the_host():
    lib = tg.load()
    one = ctypes.c_void_p(16)
    sh = tg.make_shape(1, 2, 2, 64, 10)
    norm = lambda n=1, Hq=1, Hkv=0, D=64, q=one, qs=64, eps=1e-6, rot=0, inter=0, qo=one, qos=64, pos=one, inv=one: \
        lib.tg_qk_norm_rope(n, Hq, Hkv, D, q, qs, None, 0, None, None, eps, pos, inv, rot, inter, 1.0, qo, qos, None, 0, None)
    for kw, st in ((dict(n=-1), 1), (dict(Hq=0), 1), (dict(D=4), 1), (dict(D=20), 8), (dict(D=264, qs=264, qos=264), 8),
                   (dict(rot=66), 1), (dict(rot=3), 1), (dict(rot=24), 8), (dict(eps=-1.0), 1), (dict(qs=63), 1),
                   (dict(qs=60), 1), (dict(qs=68), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(q=ctypes.c_void_p(8)), 1),
                   (dict(rot=32, pos=None), 1), (dict(rot=32, inv=None), 1)):
        assert norm(**kw) == st, kw
    assert norm(n=0) == 0
    path = lambda s=sh, sink=4, n=4, P=3, doff=one, k=one, ks=128: lib.tg_append_path_sink_recent(
        ctypes.byref(s), sink, n, doff, P, one, one, k, ks, one, 128, one, one, one, one, one, one, one, one, one, one, None)
    for kw, st in ((dict(sink=-1), 1), (dict(P=0), 1), (dict(P=65), 8), (dict(doff=None), 1), (dict(k=None), 1),
                   (dict(ks=120), 1), (dict(ks=132), 1), (dict(n=-1), 1), (dict(s=tg.make_shape(1, 2, 2, 60, 10)), 1),
                   (dict(s=tg.make_shape(1, 2, 2, 64, 10, page=8)), 1)):
        assert path(**kw) == st, kw
    assert path(s=tg.make_shape(0, 2, 2, 64, 10)) == 0
    copy = lambda pages=5, row=256, n=1, src=one, k=one, ks=None, vs=None, bad=one: lib.tg_copy_pages(
        pages, row, n, src, one, None, k, one, ks, vs, bad, None)
    for kw, st in ((dict(pages=-1), 1), (dict(row=0), 1), (dict(row=24), 8), (dict(row=8192), 8), (dict(n=-1), 1),
                   (dict(src=None), 1), (dict(k=None), 1), (dict(k=ctypes.c_void_p(8)), 1), (dict(ks=one), 1),
                   (dict(bad=None), 1)):
        assert copy(**kw) == st, kw
    assert copy(n=0, src=None) == 0
    comp = lambda s=sh, sp=5, k=one, koff=one, n=4, bad=one, tab=one: lib.tg_compact_kv(
        ctypes.byref(s), sp, k, one, one, one, one, koff, one, n, one, one, tab, one, one, one, bad, None)
    for kw, st in ((dict(sp=-1), 1), (dict(k=None), 1), (dict(k=ctypes.c_void_p(8)), 1), (dict(koff=None), 1),
                   (dict(n=-1), 1), (dict(bad=None), 1), (dict(tab=None), 1), (dict(s=tg.make_shape(1, 2, 2, 60, 10)), 1),
                   (dict(s=tg.make_shape(1, 2, 2, 4096, 10)), 8)):
        assert comp(**kw) == st, kw
    assert comp(s=tg.make_shape(0, 2, 2, 64, 10)) == 0
    # a tree call without a device plan
    plan = _plan([30, 40], 8, 2, 4)
    assert lib.tg_tree_decode(plan.handle, 1, one, one, 1024, one, 256, one, 256, one, one, one, one, one, one, 1.0, 0.0,
                              one, one, None) == 1
    assert lib.tg_tree_plan_status(plan.handle, None) == 1
    assert lib.tg_tree_plan_items(None, None, None, None, None, None, None, None) == 1
    lib.tg_tree_plan_destroy(None)


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        tg.tg_qk_norm_rope(x, None, None, None, 0.0, i, None, x, None)
    with pytest.raises(ValueError):
        tg.tg_copy_pages(i, i, None, torch.zeros(4, 16, 64), torch.zeros(4, 16, 64), i)

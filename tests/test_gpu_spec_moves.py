"""Norm + rotary positions, path append, page copy and compaction against plain 64-bit (or exact)
forms, and one speculative step through all of them followed by the ordinary decode."""
import math

import numpy as np
import pytest
import torch

import non_uniform_paged_flash_b200 as tg
from tests import _spec as sp

pytestmark = pytest.mark.gpu


def cu(a, dt=None):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dt)).cuda()


# ---- tg_qk_norm_rope ----

@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (128, 64, True), (64, 64, False), (64, 16, False),
                                         (96, 96, False), (96, 32, False), (80, 30, True), (256, 256, False),
                                         (256, 64, True), (8, 8, True), (16, 16, False), (24, 0, False), (40, 40, True)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 3), (48, 1)])
def test_norm_rope(D, rot, inter, Hq, Hkv):
    rng = np.random.default_rng(D * 7 + rot + Hq)
    for n in (1, 5):
        qkv = sp.bf16(rng, n, Hq + 2 * Hkv, D).cuda()
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        wq, wk = (sp.bf16(rng, D).cuda() for _ in range(2))
        pos = cu(rng.choice([0, 1, 17, 4095, 131071, 1000003, 2**31 - 1, -5], size=n), np.int32)
        inv, rs = tg.tg_rope_frequencies(rot, 10000.0, tg.TG_ROPE_YARN, 8.0, 4096)
        qo = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
        ko = torch.empty(n, Hkv, D, dtype=torch.bfloat16, device="cuda")
        tg.tg_qk_norm_rope(q, k, wq, wk, 1e-6, pos, cu(inv) if rot else None, qo, ko, interleaved=inter, rot_scale=rs)
        for x, w, o in ((q, wq, qo), (k, wk, ko)):
            y, tol = sp.rope_reference(x.cpu(), w.cpu(), 1e-6, pos.cpu(), inv, inter, rs)
            assert bool(((o.double().cpu() - y).abs() <= tol).all())


def test_norm_rope_one_side_in_place_no_weight():
    """A side alone, written over its strided input, without a norm; zeros stay zeros under the norm;
    infinities and NaN stay in their head."""
    rng = np.random.default_rng(3)
    inv, _ = tg.tg_rope_frequencies(128)
    pos = cu(np.arange(40) * 1001, np.int32)
    big = sp.bf16(rng, 40, 12, 128).cuda()
    x = big[:, 2:10]
    y, tol = sp.rope_reference(x.cpu(), None, 0.0, pos.cpu(), inv, False, 1.0)
    before = big.clone()
    tg.tg_qk_norm_rope(None, x, None, None, 0.0, pos, cu(inv), None, x)
    assert bool(((x.double().cpu() - y).abs() <= tol).all())
    assert torch.equal(big[:, :2], before[:, :2]) and torch.equal(big[:, 10:], before[:, 10:])
    one = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(4, 3, 128, dtype=torch.bfloat16, device="cuda")
    z[1, 1, 3], z[2, 2, 4] = float("nan"), float("inf")
    o = torch.empty_like(z)
    tg.tg_qk_norm_rope(z, None, one, None, 1e-6, pos[:4], cu(inv), o, None)
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[1, 1] = bad[2, 2] = True
    assert bool((o.cpu()[~bad] == 0).all()) and bool(torch.isnan(o.cpu()[bad]).any(-1).all())


def test_norm_rope_refusals():
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    o, w = torch.empty_like(q), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    pos, inv = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(64, dtype=torch.float64, device="cuda")
    for bad in (dict(q=q.float()), dict(q_weight=w[:64]), dict(position=pos[:3]), dict(inv_freq=inv.float()),
                dict(q_out=o[:, :1]), dict(position=pos.long()), dict(q=q.cpu()), dict(q_out=None)):
        args = dict(q=q, k=None, q_weight=w, k_weight=None, eps=1e-6, position=pos, inv_freq=inv, q_out=o, k_out=None)
        with pytest.raises(ValueError):
            tg.tg_qk_norm_rope(**{**args, **bad})
    for kw, st in ((dict(inv_freq=inv[:60]), tg.TG_EUNSUPPORTED), (dict(eps=-1.0), tg.TG_EINVAL)):
        args = dict(q=q, k=None, q_weight=w, k_weight=None, eps=1e-6, position=pos, inv_freq=inv, q_out=o, k_out=None)
        with pytest.raises(tg.TGError) as e:
            tg.tg_qk_norm_rope(**{**args, **kw})
        assert e.value.status == st
    e0 = q[:0]
    tg.tg_qk_norm_rope(e0, None, w, None, 1e-6, pos[:0], inv, o[:0], None)


# ---- tg_append_path_sink_recent ----

@pytest.mark.parametrize("D,P,sink", [(128, 1, 4), (64, 3, 0), (128, 8, 4), (72, 13, 2), (128, 29, 100), (64, 64, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_path_append(D, P, sink, in_place):
    """Heads below, at and crossing their budgets, budgets of 0, 1 and less than the path (so that the
    path replaces its own tokens); paths of length 0 to P with repeats."""
    rng = np.random.default_rng(D + P)
    B, Hkv = 9, 3
    BH = B * Hkv
    budget = rng.choice([0, 1, 2, 5, 15, 16, 17, 33, 70], size=BH).astype(np.int32)
    kv = np.array([rng.integers(0, b + 1) if rng.random() < .6 else b for b in budget], np.int32)
    s = np.maximum(0, np.minimum(sink, budget - 1))
    cursor = np.where(kv == budget, rng.integers(0, 1000, BH) % np.maximum(1, budget - s), 0).astype(np.int32)
    ids, off, pool = sp.tables(rng, -(-budget.astype(np.int64) // 16))
    nd = rng.integers(1, 65, size=B)
    doff = np.concatenate([[0], np.cumsum(nd)]).astype(np.int32)
    plen = rng.integers(0, P + 1, size=B).astype(np.int32)
    plen[0], plen[1] = P, 0
    path = np.stack([rng.integers(0, m, size=P) for m in nd]).astype(np.int32)
    for b in range(B):
        path[b, plen[b]:] = -77   # places past the path are not read as tokens
    kvd = sp.bf16(rng, int(doff[-1]), 2 * Hkv, D).cuda()
    kp, vp = (sp.bf16(rng, pool, 16, D).cuda() for _ in range(2))
    kept, n_ref, c_ref, slots = sp.path_reference(sink, doff, path, plen, budget, kv, cursor, Hkv)
    exp = []
    for pages, new in ((kp, kvd[:, :Hkv]), (vp, kvd[:, Hkv:])):
        e = pages.cpu().view(-1, D).clone()
        for i in range(BH):
            for slot, tok in kept[i].items():
                e[sp.head_rows(ids, off, i, slot + 1)[-1]] = new[tok, i % Hkv].cpu()
        exp.append(e.view(pages.shape))
    n_d, c_d = cu(kv), cu(cursor)
    n_o, c_o = (n_d, c_d) if in_place else (torch.empty_like(n_d), torch.empty_like(c_d))
    slot_out = torch.full((BH, P), 99, dtype=torch.int32, device="cuda")
    shape = tg.make_shape(B, Hkv, Hkv, D, pool)
    table = cu(ids if ids.size else np.zeros(1, np.int32))
    tg.tg_append_path_sink_recent(shape, sink, cu(doff), cu(path), cu(plen), kvd[:, :Hkv], kvd[:, Hkv:], kp, vp, table,
                                  cu(off), cu(budget), n_d, c_d, n_o, c_o, slot_out)
    torch.cuda.synchronize()
    assert np.array_equal(slot_out.cpu().numpy(), slots)
    assert np.array_equal(n_o.cpu().numpy(), n_ref) and np.array_equal(c_o.cpu().numpy(), c_ref)
    assert torch.equal(kp.cpu(), exp[0]) and torch.equal(vp.cpu(), exp[1])


def test_path_append_equals_single_appends():
    rng = np.random.default_rng(5)
    B, Hkv, D, P = 4, 2, 128, 6
    BH = B * Hkv
    budget = np.array([20, 40, 3, 33, 17, 16, 64, 5], np.int32)
    kv = np.array([18, 40, 3, 30, 17, 12, 1, 5], np.int32)
    ids, off, pool = sp.tables(rng, -(-budget // 16))
    kvd = sp.bf16(rng, B * P, 2 * Hkv, D).cuda()
    kp, vp = (sp.bf16(rng, pool, 16, D).cuda() for _ in range(2))
    kp2, vp2 = kp.clone(), vp.clone()
    n1, c1 = cu(kv), cu(np.zeros(BH, np.int32))
    n2, c2 = n1.clone(), c1.clone()
    shape = tg.make_shape(B, Hkv, Hkv, D, pool)
    path = cu(np.tile(np.arange(P), (B, 1)), np.int32)
    slots = torch.empty(BH, P, dtype=torch.int32, device="cuda")
    tg.tg_append_path_sink_recent(shape, 4, cu(np.arange(B + 1) * P, np.int32), path, cu(np.full(B, P), np.int32),
                                  kvd[:, :Hkv], kvd[:, Hkv:], kp, vp, cu(ids), cu(off), cu(budget), n1, c1, n1, c1, slots)
    one = torch.empty(BH, dtype=torch.int32, device="cuda")
    for t in range(P):
        row = kvd.view(B, P, 2 * Hkv, D)[:, t]
        tg.tg_append_sink_recent(shape, 4, row[:, :Hkv].contiguous(), row[:, Hkv:].contiguous(), kp2, vp2, cu(ids),
                                 cu(off), cu(budget), n2, c2, one)
    torch.cuda.synchronize()
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2) and torch.equal(n1, n2) and torch.equal(c1, c2)


def test_path_append_bad_heads_are_left():
    """A path index outside the draft, a page outside the pool, a bad path length: the heads concerned
    stay as they were, the others are appended."""
    rng = np.random.default_rng(6)
    B, Hkv, D, P = 4, 2, 64, 3
    BH = B * Hkv
    budget = np.full(BH, 40, np.int32)
    ids, off, pool = sp.tables(rng, -(-budget // 16))
    ids = ids.copy()
    ids[off[7]] = pool            # head 7: sequence 3
    kvd = sp.bf16(rng, B * 4, 2 * Hkv, D).cuda()
    kp, vp = (sp.bf16(rng, pool, 16, D).cuda() for _ in range(2))
    k0 = kp.clone()
    path = np.array([[0, 1, 2], [0, 4, 1], [0, 1, 2], [0, 1, 2]], np.int32)   # sequence 1 names token 4 of 4
    plen = np.array([3, 3, 4, 3], np.int32)                                    # sequence 2: longer than max_path
    n, c = cu(np.full(BH, 10), np.int32), cu(np.zeros(BH), np.int32)
    slots = torch.empty(BH, P, dtype=torch.int32, device="cuda")
    tg.tg_append_path_sink_recent(tg.make_shape(B, Hkv, Hkv, D, pool), 4, cu(np.arange(B + 1) * 4, np.int32), cu(path),
                                  cu(plen), kvd[:, :Hkv], kvd[:, Hkv:], kp, vp, cu(ids), cu(off), cu(budget), n, c, n, c,
                                  slots)
    torch.cuda.synchronize()
    good = [0, 1, 6]
    assert n.cpu().tolist() == [13 if i in good else 10 for i in range(BH)]
    assert all(slots.cpu()[i].tolist() == ([10, 11, 12] if i in good else [-1] * 3) for i in range(BH))
    changed = (kp != k0).any(-1).view(-1).nonzero().view(-1).cpu().tolist()
    assert sorted(changed) == sorted(int(r) for i in good for r in sp.head_rows(ids, off, i, 13)[10:])


# ---- tg_copy_pages ----

@pytest.mark.parametrize("kind,D", [("bf16", 128), ("bf16", 64), ("int8", 128), ("int4", 128), ("int4", 64), ("bf16", 512)])
@pytest.mark.parametrize("partial", [False, True])
def test_copy_pages(kind, D, partial):
    rng = np.random.default_rng(D + partial)
    pages, m = 200, 61
    g = torch.Generator(device="cuda").manual_seed(1)
    if kind == "bf16":
        k, v = (sp.bf16(rng, pages, 16, D).cuda() for _ in range(2))
        ks = vs = None
    else:
        k, v = (torch.randint(0, 100, (pages, 16, D if kind == "int8" else D // 2), generator=g, device="cuda",
                              dtype=torch.int8 if kind == "int8" else torch.uint8) for _ in range(2))
        ks, vs = (torch.rand(pages, 16, generator=g, device="cuda") for _ in range(2))
    perm = rng.permutation(pages).astype(np.int32)
    dst, src = perm[:m], rng.choice(perm[m:], size=m)
    rows = rng.integers(0, 17, size=m).astype(np.int32) if partial else np.full(m, 16, np.int32)
    exp = [None if t is None else t.cpu().clone() for t in (k, v, ks, vs)]
    for t in exp:
        if t is not None:
            old = t.clone()
            for a, b, r in zip(src, dst, rows):
                t[b, :r] = old[a, :r]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    tg.tg_copy_pages(cu(src), cu(dst), cu(rows) if partial else None, k, v, bad, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    for t, e in zip((k, v, ks, vs), exp):
        assert t is None or torch.equal(t.cpu(), e)
    assert int(bad) == 0


def test_copy_pages_refusals():
    k = torch.arange(8 * 16 * 64, device="cuda").to(torch.bfloat16).view(8, 16, 64)
    v, k0 = k.clone(), k.clone()
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    src, dst = cu([0, 8, -1, 1, 2, 3, 4], np.int32), cu([5, 5, 5, 8, -7, 6, 4], np.int32)
    rows = cu([17, 1, 1, 1, 1, -1, 3], np.int32)
    tg.tg_copy_pages(src, dst, rows, k, v, bad)
    assert int(bad) == 6 and torch.equal(k, k0)
    for kw in (dict(v=v.float()), dict(v=v[:4]), dict(rows=rows[:3]), dict(src=src.long()), dict(k=k.transpose(0, 2)),
               dict(k_scale=torch.zeros(3, device="cuda"))):
        a = dict(src=src, dst=dst, rows=rows, k=k, v=v, k_scale=None)
        a.update(kw)
        with pytest.raises(ValueError):
            tg.tg_copy_pages(a["src"], a["dst"], a["rows"], a["k"], a["v"], bad, k_scale=a["k_scale"])
    odd = torch.zeros(4, 16, 12, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tg.TGError) as e:
        tg.tg_copy_pages(src, dst, rows, odd, odd.clone(), bad)
    assert e.value.status == tg.TG_EUNSUPPORTED
    tg.tg_copy_pages(src[:0], dst[:0], None, k, v, bad)


# ---- tg_compact_kv ----

@pytest.mark.parametrize("D,B,Hkv", [(128, 3, 4), (64, 1, 1), (72, 5, 2), (8, 2, 3), (256, 2, 2)])
def test_compact(D, B, Hkv):
    """Budgets of 0 to all tokens, lists in any order with repeats, fewer tokens than the budget."""
    rng = np.random.default_rng(D + B)
    BH = B * Hkv
    full = np.repeat(rng.integers(1, 400, size=B), Hkv)
    budget = np.array([rng.choice([0, 1, 16, 17, int(x)]) for x in full], np.int32)
    count = np.array([rng.integers(0, b + 1) if rng.random() < .3 else b for b in budget])
    sids, soff, spool = sp.tables(rng, -(-full // 16))
    ids, off, pool = sp.tables(rng, -(-budget.astype(np.int64) // 16))
    keep = [rng.integers(0, f, size=c) for f, c in zip(full, count)]
    koff = np.concatenate([[0], np.cumsum(count)]).astype(np.int64)
    ks, vs = (sp.bf16(rng, spool, 16, D).cuda() for _ in range(2))
    kd, vd = (sp.bf16(rng, pool, 16, D).cuda() for _ in range(2))
    exp = [kd.cpu().view(-1, D).clone(), vd.cpu().view(-1, D).clone()]
    for i in range(BH):
        to = sp.head_rows(ids, off, i, int(count[i]))
        frm = sp.head_rows(sids, soff, i, int(full[i]))[keep[i]]
        for e, s in zip(exp, (ks, vs)):
            e[to] = s.cpu().view(-1, D)[frm]
    n, bad = torch.full((BH,), 9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    flat = np.concatenate(keep) if koff[-1] else np.zeros(0)
    table = cu(ids if ids.size else np.zeros(1, np.int32))
    tg.tg_compact_kv(tg.make_shape(B, Hkv, Hkv, D, pool), ks, vs, cu(sids), cu(soff), cu(full, np.int32), cu(koff),
                     cu(flat, np.int32), kd, vd, table, cu(off), cu(budget), n, bad)
    torch.cuda.synchronize()
    assert int(bad) == 0 and np.array_equal(n.cpu().numpy(), count)
    assert torch.equal(kd.cpu().view(-1, D), exp[0]) and torch.equal(vd.cpu().view(-1, D), exp[1])


def test_compact_within_one_pool_and_bad_rows():
    """Source and destination pages of one pool; tokens and pages out of bounds are counted and left,
    a list above its budget or out of order refuses its head."""
    rng = np.random.default_rng(8)
    D, B, Hkv = 64, 1, 4
    ids, off, pool = sp.tables(rng, [7, 7, 7, 7, 3, 3, 3, 3])
    k, v = (sp.bf16(rng, pool, 16, D).cuda() for _ in range(2))
    k0 = k.cpu().view(-1, D).clone()
    table = ids.copy()
    table[off[3]] = pool + 1      # head 3: its first source page is outside the pool
    keep = np.array([3, 100, 111, 112, 1, 2, 2, 3, 0, 20], np.int32)   # 112 >= 112 tokens: bad
    koff = np.array([0, 4, 4, 8, 10], np.int64)
    budget = np.array([40, 40, 3, 40], np.int32)                       # head 2 keeps 4 > 3
    n, bad = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = lambda ko: (tg.make_shape(B, Hkv, Hkv, D, pool), k, v, cu(table), cu(off[:4]), cu(np.full(4, 112), np.int32),
                       cu(ko), cu(keep), k, v, cu(table), cu(off[4:]), cu(budget), n, bad)
    tg.tg_compact_kv(*args(koff))
    torch.cuda.synchronize()
    assert n.cpu().tolist() == [4, 0, 0, 2] and int(bad) == 3
    exp = k0.clone()
    src = sp.head_rows(ids, off, 0, 112)
    to = sp.head_rows(ids, off, 4, 4)
    exp[to[:3]] = k0[src[[3, 100, 111]]]
    exp[sp.head_rows(ids, off, 7, 2)[1]] = k0[sp.head_rows(ids, off, 3, 112)[20]]
    assert torch.equal(k.cpu().view(-1, D), exp)
    bad.zero_()
    tg.tg_compact_kv(*args(np.array([0, 4, 2, 50, 50], np.int64)))     # decreasing, then past the list
    torch.cuda.synchronize()
    assert n.cpu().tolist() == [4, 0, 0, 0] and int(bad) >= 2


# ---- together ----

@pytest.mark.parametrize("D,G", [(128, 4), (64, 1)])
def test_speculative_steps(D, G):
    """Prompt rows compacted to their budgets; then steps of norm + rotary, tree attention and path
    append; a fork with its page copies; and the ordinary decode over the resulting cache of each."""
    rng = np.random.default_rng(D)
    B, Hkv, P, sink = 3, 2, 4, 4
    Hq, BH = G * Hkv, 3 * 2
    full = np.repeat([90, 200, 33], Hkv)
    budget = np.array([20, 90, 64, 150, 33, 7], np.int32)
    count = np.minimum(budget, np.array([20, 70, 64, 150, 30, 7])).astype(np.int64)
    alloc = tg.tg_alloc_create(200, 16, 3)
    lists, counts = zip(*(tg.tg_reserve(alloc, b, budget[b * Hkv:(b + 1) * Hkv], with_counts=True) for b in range(B)))
    goh = np.array([0, 1], np.int32)
    table, off, goff = tg.tg_build_group_tables(np.stack(counts), goh, 2, np.concatenate(lists))
    off = off.reshape(-1)
    sids, soff, spool = sp.tables(rng, -(-full // 16))
    ks, vs = (sp.bf16(rng, spool, 16, D).cuda() for _ in range(2))
    kp, vp = (torch.full((200, 16, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    keep = [np.sort(rng.permutation(f)[:c]) for f, c in zip(full, count)]
    kv, bad = torch.zeros(BH, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    shape = tg.make_shape(B, Hq, Hkv, D, 200)
    tg.tg_compact_kv(shape, ks, vs, cu(sids), cu(soff), cu(full, np.int32),
                     cu(np.concatenate([[0], np.cumsum(count)]), np.int64), cu(np.concatenate(keep), np.int32), kp, vp,
                     cu(table), cu(off), cu(budget), kv, bad)
    # the expected cache: slot -> (k row, v row) per head
    cache = []
    for i in range(BH):
        rows = torch.from_numpy(sp.head_rows(sids, soff, i, int(full[i]))[keep[i]])
        cache.append([ks.cpu().view(-1, D)[rows].clone(), vs.cpu().view(-1, D)[rows].clone()])
    plan = tg.tg_tree_plan_create(shape, budget, 8, goh, goff)
    inv, rs = tg.tg_rope_frequencies(D, 10000.0, tg.TG_ROPE_LINEAR, 2.0)
    w = sp.bf16(rng, D).cuda()
    cursor = torch.zeros(BH, dtype=torch.int32, device="cuda")
    n_ref, c_ref = count.copy(), np.zeros(BH, np.int64)
    scale = 1 / math.sqrt(D)
    for step in range(4):
        nd = rng.integers(1, 9, size=B)
        doff = np.concatenate([[0], np.cumsum(nd)]).astype(np.int32)
        N = int(doff[-1])
        qkv = sp.bf16(rng, N, Hq + 2 * Hkv, D).cuda()
        q, k = (torch.empty(N, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
        v = qkv[:, Hq + Hkv:]
        pos = cu(rng.integers(0, 100000, size=N), np.int32)
        tg.tg_qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], w, w, 1e-6, pos, cu(inv), q, k, rot_scale=rs)
        parent = np.concatenate([[rng.integers(-1, j) if j else -1 for j in range(m)] for m in nd]).astype(np.int32)
        mask = tg.tg_tree_masks(doff, parent)
        out, lse = torch.empty_like(q), torch.empty(N, Hq, device="cuda")
        tg.tg_tree_decode(plan, cu(doff), q, k, v, cu(mask.view(np.int64)), kp, vp, cu(table), cu(off), kv, scale, 0.0,
                          out, lse)
        ro, rl, to, tl = sp.tree_reference(q.cpu(), k.cpu(), v.cpu(), mask, doff, [c[0] for c in cache],
                                           [c[1] for c in cache], G, scale, 0.0)
        assert bool(((out.double().cpu() - ro).abs() <= to).all()) and bool(((lse.double().cpu() - rl).abs() <= tl).all())
        plen = np.minimum(nd, rng.integers(0, P + 1, size=B)).astype(np.int32)
        path = np.stack([np.resize(np.sort(rng.permutation(m)[:P]), P) for m in nd]).astype(np.int32)
        kept, n_ref, c_ref, slots = sp.path_reference(sink, doff, path, plen, budget, n_ref, c_ref, Hkv)
        slot_out = torch.empty(BH, P, dtype=torch.int32, device="cuda")
        tg.tg_append_path_sink_recent(shape, sink, cu(doff), cu(path), cu(plen), k, v, kp, vp, cu(table), cu(off),
                                      cu(budget), kv, cursor, kv, cursor, slot_out)
        for i in range(BH):
            for side, new in ((0, k), (1, v)):
                rows = cache[i][side]
                grown = torch.zeros(int(n_ref[i]), D, dtype=torch.bfloat16)
                grown[:rows.shape[0]] = rows
                for slot, tok in kept[i].items():
                    grown[slot] = new[tok, i % Hkv].cpu()
                cache[i][side] = grown
        assert np.array_equal(kv.cpu().numpy(), n_ref) and np.array_equal(slot_out.cpu().numpy(), slots)
    assert tg.tg_tree_plan_status(plan) == tg.TG_OK and int(bad) == 0

    # fork sequence 1 (nothing shared under an eviction rule), then decode parent and child
    held = n_ref[Hkv:2 * Hkv].astype(np.int32)
    ids, cnt, src, dst, rows = tg.tg_fork(alloc, 1, 9, held, budget[Hkv:2 * Hkv], [0, 0])
    tg.tg_copy_pages(cu(src), cu(dst), cu(rows), kp, vp, bad)
    for seqs, page_lists, cnts in (([0, 1, 2], np.concatenate(lists), np.stack(counts)), ([1], ids, cnt[None])):
        heads = [b * Hkv + h for b in seqs for h in range(Hkv)]
        tb, of, go = tg.tg_build_group_tables(cnts, goh, 2, page_lists)
        sh = tg.make_shape(len(seqs), Hq, Hkv, D, 200)
        n = n_ref[heads].astype(np.int32)
        dp = tg.tg_plan_create(sh, n, goh, go)
        q = sp.bf16(rng, len(seqs), Hq, D).cuda()
        out, lse = torch.empty_like(q), torch.empty(len(seqs), Hq, device="cuda")
        tg.tg_ragged_paged_decode(dp, q, kp, vp, cu(tb), cu(of.reshape(-1)), cu(n), cu(goh), scale, out, lse)
        empty = torch.zeros(len(seqs), Hkv, D)
        ro, rl, to, tl = sp.tree_reference(q.cpu(), empty, empty, np.zeros(len(seqs), np.uint64),
                                           np.arange(len(seqs) + 1), [cache[i][0] for i in heads],
                                           [cache[i][1] for i in heads], G, scale, 0.0)
        assert bool(((out.double().cpu() - ro).abs() <= to).all()) and bool(((lse.double().cpu() - rl).abs() <= tl).all())
        assert tg.tg_plan_status(dp) == tg.TG_OK
    tg.tg_alloc_destroy(alloc)
